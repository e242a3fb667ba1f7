// Attention of one token per request over the cache in 4 bits.
//
// A value is low + scale code, with a pair (scale, low) for 32 values, a group,
// so with codes c
//     q k = sum over groups g of  scale_g (q c)_g + low_g sum(q)_g,
//     sum over keys of p v = sum (p scale_g) c + sum p low_g:
// products of codes, which need no arithmetic to become operands: a code at the
// lowest bits of a half is that many times 2^-24, four bits further that many
// times 2^-20, and the MMA takes subnormal halves as they are.  An AND makes two
// operands, a shift four.  Keys are the 16 rows of the first product (queries its
// columns, held as halves with the power of two taken out of each head), so that
// nothing is spent on heads that a group does not have; a key's scale is applied
// to the product of each group in fp32.  Values are the rows of the second,
// transposed by the cache's layout; there the scale belongs to what is summed
// over, so it goes into the probabilities.  The lows are one more MMA each.
//
// A unit of work is (request, K/V head, split of `chunk` positions).  Splits lie at
// fixed positions, so a result's bits do not depend on the batch.  A unit is one
// warp's: it takes units from a counter, keeps a ring of stages of 32 keys in
// flight across them by bulk copies of its own, and shares nothing with other
// warps, so there is no barrier but the one that a stage's copies complete.
// Partial results are joined in order by a kernel of its own.  A part that all
// requests share is units of its own, whose columns are the heads of several requests;
// a long one is first turned into halves and then the prompt kernel's work, as over a
// cache of 16 bits.
//
// Roundings: queries to halves after the power of two (exact but for elements below
// 2^-24 of the head's largest); probabilities, and these times a scale, to halves, by
// 2^-11, where results are bf16, and to two halves, by 2^-21, where they are fp16; both no
// finer than halves' smallest step lets them (see kSmall).
//
// What bounds it: instructions and their latency, not the memory.  A tile of 16 keys and
// values of 128 takes 247 instructions (80 make operands of codes, 18 are MMAs), a unit
// 910 more, and accumulators and operands leave room for 12 warps an SM, which use 42 %
// of the issue slots: 64 requests of 2,000 positions (32 / 8 heads of 128) 49 us, 3.4
// TB/s; 64 of 750 (16 heads of 64) 31 us.  256 of 500 to 4,000 behind 8,192: 161 us,
// where 16 bits take 277.  Measured and slower: one tile at a time and four CTAs (184 us
// against 164), four CTAs at width 64 (34.6 against 31.8), the next unit's blocks or
// queries asked for ahead (170; registers spill), each request's last chunk in quarters
// (170: a unit costs its warp about 6 us), results joined in this kernel (spills).
#include <algorithm>
#include <type_traits>

#include "lm.h"
#include "lm_join.cuh"
#include "lm_q4.cuh"
#include "tc_ptx.cuh"

namespace codec {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTiles = 2;                   // of a stage, of keys and as many of values
constexpr int kKeys = 16 * kTiles;
constexpr int kMaxStages = 6;
template <int D, int NT> constexpr int kCtas = D == 128 && NT == 2 ? 2 : 3;    // per SM, what the registers allow
// A probability of the reference is 2^kLift; the reference follows when a score
// passes it by more than kSlack (both log2), so that a probability times a scale
// below 2 stays below 2^15.
constexpr float kLift = 6.f, kSlack = 8.f;
// Halves' steps do not get finer below 2^-14, so where a split's scales all lie below
// 2^(kSmall - 15) they are taken times the power of two that brings the largest to 1 .. 2
// (2^15 at most, a multiplication without rounding).  A probability is off by 2^-31 of the
// row's largest at most, its product with a scale by 2^-31 of the largest's with the
// split's largest scale, 2^-25 with scales at that border.
constexpr int kSmall = 9;

struct Params {
    LmShape sh;
    int B, bf16;
    const void* q;
    long long qs;
    const uint8_t *k, *v;
    const uint8_t* zeros;               // a tile that stands for zero
    const int* tables;
    const int* kv_len;
    int table_blocks, bs_shift, n_blocks;
    const int* lead;                    // blocks of the first lead_len positions of every request
    int lead_len;
    int shared_len;                     // positions of them worked on apart from the requests' own
    int n_pre;                          // partial results of these from another kernel (in pre), or
    int n_shared, sets;                 // splits of these among the units, and sets of columns
    int chunk, max_splits;
    int stages;
    int after_shared;                   // the shared part's kernel is running: nothing here needs its results
    float c;                            // scale x log2 e
    float* part;                        // [B][max_splits + 1][hq][D], a request's own behind the shared ones
    float* part_lse;
    const float* pre;                   // [n_pre][B][hq][D]
    const float* pre_lse;
    int* taken;                         // units taken (null: unit = blockIdx, + gridDim, ..); zero between calls
    void* o;
    long long os;
    float* lse;
};

// d += a b, and d = a b.
__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_new(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float log2_fast(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float low_half(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)w)); }
__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b)
{
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// What rounding a and b to the halves of ab left off.
__device__ __forceinline__ uint32_t left_off(float a, float b, uint32_t ab)
{
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&ab));
    return pack(a - v.x, b - v.y);
}
// (a + e) s - as, with as the rounded a s.
__device__ __forceinline__ uint32_t times_left(uint32_t a, uint32_t e, uint32_t s, uint32_t as)
{
    auto half2 = [](const uint32_t& x) { return *reinterpret_cast<const __half2*>(&x); };
    const __half2 v = __hfma2(half2(e), half2(s), __hfma2(half2(a), half2(s), __hneg2(half2(as))));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// N words at a shared address (a multiple of 4 N bytes) and kOff bytes.
template <int N, int kOff>
__device__ __forceinline__ void lds(uint32_t at, uint32_t* w)
{
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at), "n"(kOff)
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2 + %3];" : "=r"(w[0]), "=r"(w[1]) : "r"(at), "n"(kOff) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1 + %2];" : "=r"(w[0]) : "r"(at), "n"(kOff) : "memory");
}

// f(0), .. f(N - 1) with constants.
template <int N, typename F>
__device__ __forceinline__ void each(F f)
{
    f(std::integral_constant<int, 0>());
    if constexpr (N == 2) f(std::integral_constant<int, 1>());
}

// Splits of the shared part among the units that a request of len positions takes
// results of.  One that ends inside that part reads its own positions of it, so that
// what lies behind them never touches it.
__device__ __forceinline__ int shared_of(const Params& p, int len)
{
    return len >= p.shared_len ? p.n_shared : 0;
}

// Positions before a request's own units, and how many of these it has: one at least.
__device__ __forceinline__ int start_of(const Params& p, int len)
{
    return p.n_shared > 0 && len < p.shared_len ? 0 : p.shared_len;
}
__device__ __forceinline__ int splits_of(const Params& p, int len)
{
    return max(1, (max(0, len - start_of(p, len)) + p.chunk - 1) / p.chunk);
}

// A unit in shared memory: x the request, or the set of columns of all requests with
// kShared (kEmpty: the request has no position at all; -1: no more units), y the K/V
// head, z the place of its results among the request's and how many these are << 16,
// w positions.
constexpr int kEmpty = 1 << 30, kShared = 1 << 29;

__device__ __forceinline__ int request_of(int4 unit) { return unit.x & (kShared - 1); }

// The unit of index u and its first position: units run over the requests' splits,
// K/V heads innermost.  first, lens: the requests' first units and lengths.  A whole
// warp: 32 places are looked at at once.
__device__ __forceinline__ int4 unit_at(const Params& p, const int* first, const int* lens, int u, int& key0)
{
    int x = u / p.sh.hk;
    const int hk = u - x * p.sh.hk;
    if (x < p.n_shared * p.sets) {
        const int split = x / p.sets;
        key0 = split * p.chunk;
        return make_int4((x - split * p.sets) | kShared, hk, split | (p.n_shared + 1) << 16, min(p.shared_len - key0, p.chunk));
    }
    x -= p.n_shared * p.sets;
    const int lane = threadIdx.x & 31;
    int b = 0;
    for (int step = p.B <= 32 ? 1 : p.B <= 1024 ? 32 : 1024; step > 0; step >>= 5) {
        const int at = b + lane * step;
        b += (__popc(__ballot_sync(0xffffffffu, at < p.B && first[at] <= x)) - 1) * step;
    }
    const int len = lens[b], split = x - first[b], before = shared_of(p, len);
    key0 = start_of(p, len) + split * p.chunk;
    return make_int4(b | (len == 0 ? kEmpty : 0), hk, (before + split) | (before + first[b + 1] - first[b]) << 16,
                     min(max(len - key0, 0), p.chunk));
}

// The warps' stages, the stages' units and barriers, a unit of each warp, flags, the requests' first units and lengths.
template <int D>
size_t smem_bytes(int stages, int B)
{
    return 128 + (size_t)kWarps * stages * (2 * kTiles * Q4Tile<D>::kBytes + 16 + 8) + kWarps * 16 + 16 + (2 * (size_t)B + 1) * 4;
}

__device__ __forceinline__ void store2(const Params& p, void* row, int i, float a, float b)
{
    if (p.bf16)
        reinterpret_cast<__nv_bfloat162*>(row)[i] = __floats2bfloat162_rn(a, b);
    else
        reinterpret_cast<__half2*>(row)[i] = __floats2half2_rn(a, b);
}

// Joins the partial results of (request, head), the shared part's first, in
// order.  One warp; empty: the request has no position at all.
template <int D, int kAhead>
__device__ __forceinline__ void join_parts(const Params& p, int b, int h, int n_splits, bool empty, int lane)
{
    constexpr int kE = D / 32;
    const int parts = empty ? 0 : p.n_pre + n_splits;
    const long long shared_row = (long long)b * p.sh.hq + h, own_row = (long long)b * (p.max_splits + 1) * p.sh.hq + h;
    auto row_of = [&](int i) {
        return i < p.n_pre ? (long long)i * p.B * p.sh.hq + shared_row : (long long)(i - p.n_pre) * p.sh.hq + own_row;
    };
    float v[kE], lse;
    join_row<kE, kAhead, true>(
        parts, empty, [&](int i) { return __ldcg((i < p.n_pre ? p.pre_lse : p.part_lse) + row_of(i)); },
        [&](int i, float* x) { row_part<kE>((i < p.n_pre ? p.pre : p.part) + row_of(i) * D, x); }, v, lse);
    uint16_t* row = static_cast<uint16_t*>(p.o) + b * p.os + (long long)h * D;
#pragma unroll
    for (int e = 0; e < kE; e += 2) store2(p, row, (lane * kE + e) / 2, v[e], v[e + 1]);
    if (p.lse && lane == 0) p.lse[(long long)b * p.sh.hq + h] = lse;
}

// A warp per (request, head) whose result is in parts.
constexpr int kJoinThreads = 128;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) lm_join_q4_kernel(const __grid_constant__ Params p)
{
    // A length was complete before the units' kernel passed its own wait, so it need not
    // wait for that kernel's end; from L2, as there.
    const long long w = blockIdx.x * (kJoinThreads / 32LL) + (threadIdx.x >> 5);
    const int b = (int)(w / p.sh.hq), h = (int)(w - (long long)b * p.sh.hq);
    int len = b < p.B ? __ldcg(p.kv_len + b) : 0;
    lm_clamp_len(len, (long long)p.table_blocks << p.bs_shift);
    const int n = shared_of(p, len) + splits_of(p, len);
    pdl_wait();
    pdl_launch();
    if (p.taken && blockIdx.x == 0 && threadIdx.x == 0) *p.taken = 0;
    if (b >= p.B) return;
    if (n == 1 && p.n_pre == 0) return;         // written by its unit
    join_parts<D, 16>(p, b, h, n, len == 0, threadIdx.x & 31);
}

// NT: sets of eight columns.  kFine: a probability, and its product with a scale, is two
// halves, what is rounded and what that leaves off (2^-21 in all).  Rounded to one half
// each they put a result off by 0.0003 of it, where its own rounding to fp16 does by 0.0002
// and to bf16 by 0.0017: fp16 results have it, for 15 % more instructions.
template <int D, int NT, bool kFine>
__global__ void __launch_bounds__(kThreads, kCtas<D, NT>) lm_step_q4_kernel(const __grid_constant__ Params p)
{
    using Tile = Q4Tile<D>;
    constexpr int G = Tile::G, kAt = NT == 1 ? 2 : 1;       // tiles worked on at once
    constexpr uint32_t kTile = Tile::kBytes, kM0 = 0x000f000fu, kM1 = 0x00f000f0u;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, S = p.stages;
    constexpr uint32_t kStage = 2 * kTiles * kTile;
    uint8_t* ring = smem + (size_t)warp * S * kStage;
    int4* units_of = reinterpret_cast<int4*>(smem + (size_t)kWarps * S * kStage);
    int4* unit_of = units_of + warp * S;                        // the unit whose first keys a stage holds
    int4* now = units_of + kWarps * S + warp;                   // the unit that is worked on
    uint64_t* full = reinterpret_cast<uint64_t*>(units_of + kWarps * (S + 1)) + warp * S;
    int* flags = reinterpret_cast<int*>(reinterpret_cast<uint64_t*>(units_of + kWarps * (S + 1)) + kWarps * S);  // abort
    uint64_t* never = reinterpret_cast<uint64_t*>(flags + 2);   // nothing arrives (see LmShape::unarrived)
    int* first = flags + 4;
    int* lens = first + p.B + 1;
    volatile int* abort_flag = flags;

    if (lane == 0)
        for (int i = 0; i < S; i++) mbar_init(&full[i], 1);
    if (tid == 0) {
        mbar_init(never, 1);
        flags[0] = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // Behind the shared part's kernel there is nothing to wait for: what this one
    // reads was complete when that one passed its own wait.  It has to come from L2
    // all the same: lengths, tables and queries by __ldcg, the rest by bulk copies.
    if (!p.after_shared) pdl_wait();
    pdl_launch();
    int next = blockIdx.x * kWarps + warp;      // lane 0's: the unit after this one
    if (p.taken && lane == 0) next = atomicAdd(p.taken, 1);
    {
        // units before each request: at least one per request, so that something writes its row
        if (warp == 0) {
            int before = 0;
            for (int base = 0; base < p.B; base += 32) {
                const int b = base + lane;
                int n = 0;
                if (b < p.B) {
                    int len = __ldcg(p.kv_len + b);
                    if (!lm_clamp_len(len, (long long)p.table_blocks << p.bs_shift) && blockIdx.x == 0)
                        atomicOr(p.sh.err, CODEC_LM_ERR_LENGTH);
                    n = splits_of(p, len);
                    lens[b] = len;
                }
                int incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                if (b < p.B) first[b] = before + incl - n;
                before += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) first[p.B] = before;
        }
        __syncthreads();
    }
    const int units = (p.n_shared * p.sets + first[p.B]) * p.sh.hk;

    // ---- copies ----
    // Lane i has what stage i of the next 32 of a unit takes, and issues it.
    int from = 0, end = 0, turn = 0, issued = 0;    // positions; the lane whose stage is next
    int tile[kTiles] = {-1, -1};                // the two tiles in the cache; -1: zeros
    int copied = 0;                             // the request, and the K/V head << 16
    bool last_out = false;                      // the stage that says so is out
    auto issue = [&](int st) {
        if (last_out) return;
        issued++;
        if (from >= end) {
            const int u = __shfl_sync(0xffffffffu, next, 0);
            if (u >= units) {
                if (lane == 0) {
                    unit_of[st].x = -1;
                    mbar_arrive(&full[st]);
                }
                last_out = true;
                return;
            }
            if (!p.taken)
                next += gridDim.x * kWarps;
            else if (lane == 0)
                next = atomicAdd(p.taken, 1);   // needed when this unit's copies are out
            const int4 unit = unit_at(p, first, lens, u, from);
            end = from + unit.w;
            turn = 32;
            copied = (unit.x & 0xffff) | unit.y << 16;          // (a set's tables are not looked at)
            if (lane == 0) unit_of[st] = unit;
            if (unit.w == 0) {                  // takes a stage without copies
                if (lane == 0) mbar_arrive(&full[st]);
                return;
            }
        }
        if (turn == 32) {
            turn = 0;
            const int* table = p.tables + (long long)(copied & 0xffff) * p.table_blocks;
#pragma unroll
            for (int i = 0; i < kTiles; i++) {
                const int pos = from + lane * kKeys + i * 16, j = pos >> p.bs_shift;
                tile[i] = -1;
                if (pos < end) {
                    const int id = __ldcg((pos < p.lead_len ? p.lead : table) + j);
                    if (id >= 0 && id < p.n_blocks)
                        tile[i] = ((id * p.sh.hk + (copied >> 16)) << (p.bs_shift - 4)) + ((pos & ((1 << p.bs_shift) - 1)) >> 4);
                    else
                        atomicOr(p.sh.err, CODEC_LM_ERR_BLOCK);
                }
            }
        }
        // (by one lane that the compiler knows to be one: the copies' operands are uniform)
        const int first_tile = __shfl_sync(0xffffffffu, tile[0], turn);
        const bool both = end - from > 16, apart = both && p.bs_shift == 4;
        const int second = apart ? __shfl_sync(0xffffffffu, tile[1], turn) : -1;
        if (elect_one()) {
            uint8_t* dst = ring + st * kStage;
            const uint32_t bytes = both && !apart ? 2 * kTile : kTile;
            mbar_expect_tx(&full[st], both ? 4 * kTile : 2 * kTile);
            const long long at = first_tile * (long long)kTile;
            bulk_load(dst, first_tile >= 0 ? p.k + at : p.zeros, &full[st], bytes);
            bulk_load(dst + kTiles * kTile, first_tile >= 0 ? p.v + at : p.zeros, &full[st], bytes);
            if (apart) {
                const long long at1 = second * (long long)kTile;
                bulk_load(dst + kTile, second >= 0 ? p.k + at1 : p.zeros, &full[st], kTile);
                bulk_load(dst + (kTiles + 1) * kTile, second >= 0 ? p.v + at1 : p.zeros, &full[st], kTile);
            }
        }
        turn++;
        from += kKeys;
    };
    for (int i = 0; i < S; i++) issue(i);

    // Request and head of its group of a unit's column c; a head behind the last for one that
    // nobody reads.
    auto column = [&](int4 unit, int c) {
        if (!(unit.x & kShared)) return make_int2(request_of(unit), c);
        const int j = request_of(unit) * 8 * NT + c, b = j / p.sh.group;
        return b < p.B && lens[b] >= p.shared_len ? make_int2(b, j - b * p.sh.group) : make_int2(min(b, p.B - 1), p.sh.group);
    };

    // ---- products ----
    const int r = lane >> 2, t = lane & 3;      // row (and + 8) and column pair of a fragment
    const int c0 = 2 * t;                       // first of this lane's two columns of a set
    const uint32_t base = smem_u32(ring);
    // this lane's places in a tile: a key's codes and (scale, low), the low of group t, values' codes,
    // their scales, and their lows of group r
    const uint32_t k_at = r * (D / 2) + t * 4 * G, kp_at = r * 4 * G, kl_at = (r * G + min(t, G - 1)) * 4;
    const uint32_t v_at = lane * 4 * G, vs_at = t * 8 * G, vl_at = (t * G + min(r, G - 1)) * 8;
    int st = 0, done = 0;
    uint32_t ph = 0;
    bool gave_up = false;
    while (true) {
        gave_up = !__all_sync(0xffffffffu, mbar_wait(&full[st], ph, abort_flag, kLmPolls));
        if (gave_up) break;
        const int4 unit = unit_of[st];
        if (unit.x < 0) {
            done++;
            break;
        }
        __syncwarp();
        if (lane == 0) *now = unit;
        const int keys = unit.w;
        uint32_t qf[NT][G][4], ql[NT];          // queries and their groups' sums
        float cf[NT][2];                        // of this lane's columns: what makes a score (log2) of an accumulator
        float acc[NT][G][2][4], low[NT][4];
        // A probability is 2^(score + bias); past `most` (an accumulator) the reference moves.
        float bias[NT][2], most[NT][2], l[NT][2];
#pragma unroll
        for (int x = 0; x < NT; x++) {
#pragma unroll
            for (int g = 0; g < G; g++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[x][g][0][e] = acc[x][g][1][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; e++) low[x][e] = 0.f;
            most[x][0] = most[x][1] = -INFINITY;
            bias[x][0] = bias[x][1] = 0.f;
            l[x][0] = l[x][1] = 0.f;
        }
        // Column r of each set, elements 8 t .. 8 t + 7 of each group, as halves times a
        // power of two.  Columns behind the last repeat it: nobody reads them.
#pragma unroll
        for (int x = 0; x < NT; x++) {
            const int2 col = column(unit, 8 * x + r);
            const uint16_t* row = static_cast<const uint16_t*>(p.q) + col.x * p.qs +
                                  ((long long)unit.y * p.sh.group + min(col.y, p.sh.group - 1)) * D + t * 8;
            uint4 w[G];
#pragma unroll
            for (int g = 0; g < G; g++) w[g] = __ldcg(reinterpret_cast<const uint4*>(row + g * 32));
            float f[G][8], top = 0.f;
#pragma unroll
            for (int g = 0; g < G; g++) {
                const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float2 y = kFine ? __half22float2(*reinterpret_cast<const __half2*>(&u[e]))
                                           : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[e]));
                    f[g][2 * e] = y.x;
                    f[g][2 * e + 1] = y.y;
                    top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int lift = q4_query_lift(top);
            const float m = __int_as_float((127 + lift) << 23), m16 = m * 0.0625f;
            float mine = 0.f;
#pragma unroll
            for (int g = 0; g < G; g++) {
#pragma unroll
                for (int e = 0; e < 8; e++) f[g][e] *= e & 1 ? m16 : m;
                float sum = fmaf(16.f, (f[g][1] + f[g][3]) + (f[g][5] + f[g][7]), (f[g][0] + f[g][2]) + (f[g][4] + f[g][6]));
                qf[x][g][0] = pack(f[g][0], f[g][4]);
                qf[x][g][1] = pack(f[g][2], f[g][6]);
                qf[x][g][2] = pack(f[g][1], f[g][5]);
                qf[x][g][3] = pack(f[g][3], f[g][7]);
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (g == t) mine = sum;
            }
            mine *= 0x1p-6f;
            const float hi = __half2float(__float2half_rn(mine));
            ql[x] = pack(hi, mine - hi);
            const float back = q4_query_factor(p.c, lift) * 0x1p24f;        // sums of codes are 2^-24 of what they stand for
            cf[x][0] = __shfl_sync(0xffffffffu, back, c0 * 4);
            cf[x][1] = __shfl_sync(0xffffffffu, back, c0 * 4 + 4);
        }
        // Scales are below 2^(1 + grown).  Beyond 0 the reference is lowered by it; below 0
        // scales are taken times 2^-grown.
        int grown = -15;
#pragma unroll 1
        for (int at = 0; at == 0 || at < keys; at += kKeys) {
            if (at > 0) {
                // (unarrived: one warp's second stage of a unit of more than 64 positions never comes)
                gave_up = !__all_sync(0xffffffffu, p.sh.unarrived && warp == 0 && keys > 64
                                                       ? mbar_wait(never, 0, abort_flag, p.sh.unarrived)
                                                       : mbar_wait(&full[st], ph, abort_flag, kLmPolls));
                if (gave_up) break;
            }
            if (keys > 0) {
#pragma unroll 1
                for (int w = 0; w < kTiles && at + 16 * w < keys; w += kAt) {
                    const int here = at + 16 * w;
                    const uint32_t kt = base + (uint32_t)st * kStage + w * kTile;
                    float s[kAt][NT][4];
                    // scores
                    each<kAt>([&](auto I) {
                        constexpr int i = I, kOff = i * kTile, kP = kOff + Tile::kParams;
                        uint32_t ka[G], kb[G], pa[G], pb[G], la, lb;
                        lds<G, kOff>(kt + k_at, ka);
                        lds<G, kOff + 4 * D>(kt + k_at, kb);
                        lds<1, kP>(kt + kl_at, &la);
                        lds<1, kP + 32 * G>(kt + kl_at, &lb);
                        lds<G, kP>(kt + kp_at, pa);
                        lds<G, kP + 32 * G>(kt + kp_at, pb);
                        if (G < 4 && t >= G) la = lb = 0u;
                        la = __byte_perm(la, 0, 0x3232);
                        lb = __byte_perm(lb, 0, 0x3232);
#pragma unroll
                        for (int x = 0; x < NT; x++) {
                            mma_new(s[i][x], la, lb, 0u, 0u, ql[x], 0u);
#pragma unroll
                            for (int e = 0; e < 4; e++) s[i][x][e] *= 0x1p-18f;
                        }
#pragma unroll
                        for (int g = 0; g < G; g++) {
                            const uint32_t a0 = ka[g] & kM0, a1 = ka[g] & kM1, a2 = ka[g] >> 8 & kM0, a3 = ka[g] >> 8 & kM1;
                            const uint32_t b0 = kb[g] & kM0, b1 = kb[g] & kM1, b2 = kb[g] >> 8 & kM0, b3 = kb[g] >> 8 & kM1;
                            const float sa = low_half(pa[g]), sb = low_half(pb[g]);
#pragma unroll
                            for (int x = 0; x < NT; x++) {
                                float d[4];
                                mma_new(d, a0, b0, a2, b2, qf[x][g][0], qf[x][g][1]);
                                mma(d, a1, b1, a3, b3, qf[x][g][2], qf[x][g][3]);
                                s[i][x][0] = fmaf(sa, d[0], s[i][x][0]);
                                s[i][x][1] = fmaf(sa, d[1], s[i][x][1]);
                                s[i][x][2] = fmaf(sb, d[2], s[i][x][2]);
                                s[i][x][3] = fmaf(sb, d[3], s[i][x][3]);
                            }
                        }
                    });
                    // values: scales and lows of keys 2 t, 2 t + 1 and of those 8 further
                    uint32_t sc[kAt][2 * G], vl[kAt][2];
                    each<kAt>([&](auto I) {
                        constexpr int i = I, kP = (kTiles + i) * kTile + Tile::kParams;
                        lds<4, kP>(kt + vs_at, sc[i]);
                        if constexpr (G == 4) lds<4, kP + 16>(kt + vs_at, sc[i] + 4);
                        lds<2, kP + D>(kt + vl_at, vl[i]);
                        if (r >= G) vl[i][0] = vl[i][1] = 0u;
                    });
                    if (here + 16 * kAt > keys) {
                        // what lies behind the last key may be anything
#pragma unroll
                        for (int i = 0; i < kAt; i++) {
                            const int left = keys - here - 16 * i;
#pragma unroll
                            for (int x = 0; x < NT; x++)
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    if (r + (e >> 1) * 8 >= left) s[i][x][e] = -INFINITY;
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const int k0 = c0 + 8 * h;
                                const uint32_t keep = (k0 < left ? 0xffffu : 0u) | (k0 + 1 < left ? 0xffff0000u : 0u);
#pragma unroll
                                for (int g = 0; g < G; g++) sc[i][2 * g + h] &= keep;
                                vl[i][h] &= keep;
                            }
                        }
                    }
                    uint32_t or_of = 0u;
#pragma unroll
                    for (int i = 0; i < kAt; i++)
#pragma unroll
                        for (int g = 0; g < 2 * G; g++) or_of |= sc[i][g];
                    or_of &= 0x7fff7fffu;
                    bool move = max(or_of & 0xffffu, or_of >> 16) >= (uint32_t)(16 + grown) << 10;
#pragma unroll
                    for (int i = 0; i < kAt; i++)
#pragma unroll
                        for (int x = 0; x < NT; x++)
#pragma unroll
                            for (int e = 0; e < 4; e++) move |= s[i][x][e] > most[x][e & 1];
                    if (__any_sync(0xffffffffu, move)) {
                        // the largest exponent among the scales (31: not finite, nothing follows from it)
                        int e = 0;
#pragma unroll
                        for (int i = 0; i < kAt; i++)
#pragma unroll
                            for (int g = 0; g < 2 * G; g++) {
                                const int lo = sc[i][g] >> 10 & 31, hi = sc[i][g] >> 26 & 31;
                                e = max(e, max(lo == 31 ? 0 : lo, hi == 31 ? 0 : hi));
                            }
                        e = (int)__reduce_max_sync(0xffffffffu, e);
                        const int to = max(grown, e >= kSmall ? max(e - 15, 0) : e - 15);
                        const int more = max(to, 0) - max(grown, 0);
                        const float shrink = __int_as_float((127 - more) << 23);
                        const float less = __int_as_float((127 + more - (to - grown)) << 23);   // of the scales
                        grown = to;
                        // a column's reference moves for its own scores alone (times 1 changes nothing)
#pragma unroll
                        for (int x = 0; x < NT; x++)
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                float m = fmaxf(s[0][x][h], s[0][x][2 + h]);
                                if constexpr (kAt == 2) m = fmaxf(m, fmaxf(s[1][x][h], s[1][x][2 + h]));
                                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                                float f = shrink;
                                bias[x][h] -= (float)more;
                                if (m > most[x][h]) {
                                    const float now = fmaf(-m, cf[x][h], kLift - (float)max(grown, 0));
                                    f = most[x][h] == -INFINITY ? 0.f : shrink * exp2_fast(now - bias[x][h]);
                                    bias[x][h] = now;
                                    most[x][h] = m + kSlack / cf[x][h];
                                }
                                if (here == 0) continue;        // nothing is summed yet
                                l[x][h] *= f;
                                low[x][h] *= f;
                                f *= less;
#pragma unroll
                                for (int g = 0; g < G; g++)
#pragma unroll
                                    for (int i = 0; i < 2; i++) {
                                        acc[x][g][i][h] *= f;
                                        acc[x][g][i][2 + h] *= f;
                                    }
                            }
                    }
                    if (grown < 0) {
                        const uint32_t up = (uint32_t)(15 - grown) * 0x04000400u;
#pragma unroll
                        for (int i = 0; i < kAt; i++)
#pragma unroll
                            for (int g = 0; g < 2 * G; g++) sc[i][g] = times(sc[i][g], up);
                    }
                    each<kAt>([&](auto I) {
                        constexpr int i = I, kOff = (kTiles + i) * kTile;
                        uint32_t va[G], vb[G], f0[NT], f1[NT], e0[NT], e1[NT];
                        lds<G, kOff>(kt + v_at, va);
                        lds<G, kOff + 4 * D>(kt + v_at, vb);
#pragma unroll
                        for (int x = 0; x < NT; x++) {
                            const float p0 = exp2_fast(fmaf(s[i][x][0], cf[x][0], bias[x][0])),
                                        p1 = exp2_fast(fmaf(s[i][x][1], cf[x][1], bias[x][1]));
                            const float p2 = exp2_fast(fmaf(s[i][x][2], cf[x][0], bias[x][0])),
                                        p3 = exp2_fast(fmaf(s[i][x][3], cf[x][1], bias[x][1]));
                            l[x][0] += p0 + p2;
                            l[x][1] += p1 + p3;
                            f0[x] = pack(p0, p1);
                            f1[x] = pack(p2, p3);
                            if constexpr (kFine) {
                                e0[x] = transposed(left_off(p0, p1, f0[x]));
                                e1[x] = transposed(left_off(p2, p3, f1[x]));
                            }
                            f0[x] = transposed(f0[x]);
                            f1[x] = transposed(f1[x]);
                            mma(low[x], vl[i][0], 0u, vl[i][1], 0u, f0[x], f1[x]);
                            if constexpr (kFine) mma(low[x], vl[i][0], 0u, vl[i][1], 0u, e0[x], e1[x]);
                        }
#pragma unroll
                        for (int g = 0; g < G; g++) {
                            const uint32_t a0 = va[g] & kM0, a1 = va[g] & kM1, a2 = va[g] >> 8 & kM0, a3 = va[g] >> 8 & kM1;
                            const uint32_t b0 = vb[g] & kM0, b1 = vb[g] & kM1, b2 = vb[g] >> 8 & kM0, b3 = vb[g] >> 8 & kM1;
#pragma unroll
                            for (int x = 0; x < NT; x++) {
                                const uint32_t g0 = times(f0[x], sc[i][2 * g]), g1 = times(f1[x], sc[i][2 * g + 1]);
                                mma(acc[x][g][0], a0, a1, b0, b1, g0, g1);
                                mma(acc[x][g][1], a2, a3, b2, b3, g0, g1);
                                if constexpr (kFine) {
                                    const uint32_t h0 = times_left(f0[x], e0[x], sc[i][2 * g], g0),
                                                   h1 = times_left(f1[x], e1[x], sc[i][2 * g + 1], g1);
                                    mma(acc[x][g][0], a0, a1, b0, b1, h0, h1);
                                    mma(acc[x][g][1], a2, a3, b2, b3, h0, h1);
                                }
                            }
                        }
                    });
                }
            }
            __syncwarp();
            issue(st);
            done++;
            if (++st == S) {
                st = 0;
                ph ^= 1u;
            }
        }
        if (gave_up) break;
        // Results: sums of codes are 2^-24 of what they stand for, and 2^-20 for a
        // group's elements 1 and 3 of four; this lane has elements 4 r .. of each group.
        const int4 was = *now;
        const bool alone = was.z >> 16 == 1 && p.n_pre == 0;
#pragma unroll
        for (int x = 0; x < NT; x++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                float sum = l[x][h];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int2 col = column(was, 8 * x + c0 + h);
                const int b = col.x, head = was.y * p.sh.group + col.y;
                const bool there = col.y < p.sh.group, none = keys == 0;
                // (both to 2^-22: the sum is 2^-9 at least)
                const float inv = none ? 0.f : reciprocal(sum),
                            lse = none ? -INFINITY : (log2_fast(sum) - bias[x][h]) * 0.6931471805599453f;
                const float down = inv * __int_as_float((127 + min(grown, 0)) << 23);
                const float inv24 = down * 0x1p24f, inv20 = down * 0x1p20f;
                const long long at = ((long long)b * (p.max_splits + 1) + (was.z & 0xffff)) * p.sh.hq + head;
#pragma unroll
                for (int g = 0; g < G; g++) {
                    const float add = __shfl_sync(0xffffffffu, low[x][h], g * 4 + t) * inv;
                    const float4 v = make_float4(fmaf(acc[x][g][0][h], inv24, add), fmaf(acc[x][g][0][2 + h], inv20, add),
                                                 fmaf(acc[x][g][1][h], inv24, add), fmaf(acc[x][g][1][2 + h], inv20, add));
                    if (!there) continue;
                    if (alone) {
                        uint16_t* row = static_cast<uint16_t*>(p.o) + b * p.os + (long long)head * D + g * 32 + r * 4;
                        store2(p, row, 0, v.x, v.y);
                        store2(p, row, 1, v.z, v.w);
                    } else {
                        __stcg(reinterpret_cast<float4*>(p.part + at * D + g * 32 + r * 4), v);
                    }
                }
                if (there && r == 0) {
                    if (!alone)
                        __stcg(p.part_lse + at, lse);
                    else if (p.lse)
                        p.lse[(long long)b * p.sh.hq + head] = lse;
                }
            }
    }
    // every copy that is out has landed before the CTA can end
    for (int i = done; i < issued; i++) mbar_drain(&full[i % S], (uint32_t)(i / S) & 1u);
    __syncthreads();
    if (tid == 0 && flags[0]) atomicOr(p.sh.err, CODEC_LM_ERR_TIMEOUT);
    // this kernel's end is its predecessors' too
    if (p.after_shared) pdl_wait();
}

// Stages and CTAs per SM: as many CTAs as registers allow, with three stages at least.
template <int D>
void fit(Params& p, int most_per_sm, int& per_sm)
{
    constexpr size_t kSm = 228 * 1024, kOne = 227 * 1024;
    for (per_sm = most_per_sm; per_sm >= 1; per_sm--)
        for (p.stages = kMaxStages; p.stages >= 3; p.stages--) {
            const size_t n = smem_bytes<D>(p.stages, p.B);
            if (n <= kOne && per_sm * (n + 1024) <= kSm) return;
        }
    per_sm = 1;
    p.stages = 3;
}

template <int D>
cudaError_t launch(const LmShape& sh, const LmStepArgs& a, cudaStream_t s)
{
    const LmKeys& ks = a.keys;
    Params p{};
    p.sh = sh;
    p.B = a.B;
    p.bf16 = sh.type == CODEC_LM_BF16;
    p.q = a.q;
    p.qs = a.qs;
    p.k = static_cast<const uint8_t*>(ks.k);
    p.v = static_cast<const uint8_t*>(ks.v);
    p.zeros = a.ws.zeros;
    p.tables = ks.tables;
    p.kv_len = ks.kv_len;
    p.table_blocks = ks.table_blocks;
    p.bs_shift = ks.bs_shift;
    p.n_blocks = ks.n_blocks;
    p.shared_len = a.shared_blocks << ks.bs_shift;
    p.chunk = a.ws.chunk_q4;
    p.max_splits = a.ws.max_splits_q4;
    p.c = (float)(sh.scale * 1.4426950408889634);
    p.part = a.ws.part;
    p.part_lse = a.ws.part_lse;
    p.pre = a.ws.pre;
    p.pre_lse = a.ws.pre_lse;
    p.o = a.o;
    p.os = a.os;
    p.lse = a.lse;
    p.lead = a.shared_table;
    p.lead_len = p.shared_len;
    // The shared part, by its length and the largest batch, so that the actual one changes
    // no bits.  Up to 64 positions every request reads it in front of its own (32 before
    // 64 x 16 heads of 64: 18.7 us, as units 23.4, by the prompt kernel 30.4; 128: 27.5,
    // 24.0, 30.9).  Up to 16,384 tiles of 16 keys x 8 columns (16 in groups beyond 8) it is
    // units of this kernel, whose columns are the heads of eight requests and more (64 of
    // 500 to 4,000 behind 1,024, 32 / 8 of 128, 16,384 tiles: 65.5, 55.7, 62.4 us; 256 of
    // 1 to 500 behind 256, as many: 53.3, 44.8, 49.5).  Beyond, it is turned into halves
    // and the prompt kernel's (behind 4,096, 64 x 16 heads, 32,768 tiles: 113, 39.4, 36.7;
    // 256 behind 8,192: 484, 269, 82.4); what of it does not fit the workspace every
    // request reads.  As units and as halves in front of 1 to 500 positions, by thousands of
    // tiles: 64 x 32 / 8, 12 21.5, 25.1; 16 21.8, 25.2; 20 28.0, 26.0; 25 34.8, 26.4; 64 x 16 / 16
    // of 64, 12 25.7, 26.7; 16 28.1, 26.9; 20 29.5, 26.4; 33 30.4, 28.3; 256 x 32 / 8, 16 42.0,
    // 47.2; 20 46.8, 47.1; 25 48.8, 47.2; 33 51.5, 49.2; 32 x 16 / 8, 16 22.3, 25.0; 33 38.4, 31.8.
    // Not for fp16: keys rounded to halves put its results off by 0.00054 of them, where they
    // are by 0.0002 when they are rounded alone.
    const int wide = lm_sets_q4(sh.group), most = (int)(a.ws.heads / sh.hk);
    if (most == 1 || p.shared_len <= 64) p.shared_len = 0;
    if (p.shared_len > 0 && !lm_halves_q4(sh.type, most, a.ws.heads, sh.group, p.shared_len)) {
        p.n_shared = (p.shared_len + p.chunk - 1) / p.chunk;
        p.sets = (a.B * sh.group + 8 * wide - 1) / (8 * wide);
    } else if (p.shared_len > 0) {
        p.shared_len = std::min(p.shared_len, a.ws.shared_q4);
        const int blocks = p.shared_len >> ks.bs_shift;
        const LmHalvesArgs h{ks.k, ks.v, a.shared_table, blocks, ks.bs_shift, ks.n_blocks, a.q, a.qs, a.B, a.ws.k16, a.ws.v16,
                             a.ws.q16, a.ws.row_c};
        cudaError_t e = launch_lm_halves_q4(sh, h, s);
        if (e != cudaSuccess) return e;
        LmShape halves = sh;
        halves.type = CODEC_LM_FP16;
        LmKeys in = ks;
        in.k = a.ws.k16;
        in.v = a.ws.v16;
        in.n_blocks = blocks;
        LmSharedArgs c{a.ws.q16, (long long)sh.hq * D, a.B, in, a.ws.count, p.shared_len, 0, a.ws.pre, a.ws.pre_lse, a.ws.row_c};
        // splits by the object's shape and the shared length alone
        const int n = lm_shared_splits(a.ws.shared_ctas, p.shared_len);
        c.split_len = ((p.shared_len + n - 1) / n + 127) & ~127;
        p.n_pre = (p.shared_len + c.split_len - 1) / c.split_len;
        // beside the shared part only while that one's CTAs all fit the GPU at once
        p.after_shared = lm_shared_ctas(halves, c) <= 152;
        e = launch_lm_shared(halves, c, s);
        if (e != cudaSuccess) return e;
    }
    int per_sm = 1;
    fit<D>(p, wide == 2 ? kCtas<D, 2> : kCtas<D, 1>, per_sm);
    // a unit per request and head at least, and no more CTAs than the SMs hold at once
    const long long units = ((long long)a.B * p.max_splits + (long long)p.n_shared * p.sets) * sh.hk;
    const unsigned ctas = (unsigned)std::min<long long>(152 * per_sm, (units + kWarps - 1) / kWarps);
    const bool two = p.n_pre + p.n_shared > 0 || p.max_splits > 1;
    // from the counter where a warp has more than one
    p.taken = two && units > (long long)ctas * kWarps ? a.ws.taken : nullptr;
    auto kernel = p.bf16 ? (wide == 2 ? lm_step_q4_kernel<D, 2, false> : lm_step_q4_kernel<D, 1, false>)
                         : (wide == 2 ? lm_step_q4_kernel<D, 2, true> : lm_step_q4_kernel<D, 1, true>);
    const cudaError_t e = launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem_bytes<D>(p.stages, a.B), s, p);
    if (e != cudaSuccess || !two) return e;
    return launch_pdl(lm_join_q4_kernel<D>, dim3((unsigned)(((long long)a.B * sh.hq + kJoinThreads / 32 - 1) / (kJoinThreads / 32))),
                      dim3(kJoinThreads), 0, s, p);
}

template <int D>
cudaError_t configure()
{
    const void* kernels[] = {(const void*)lm_step_q4_kernel<D, 1, false>, (const void*)lm_step_q4_kernel<D, 2, false>,
                             (const void*)lm_step_q4_kernel<D, 1, true>, (const void*)lm_step_q4_kernel<D, 2, true>};
    for (const void* k : kernels) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t configure_lm_step_q4()
{
    const cudaError_t e = configure<64>();
    return e != cudaSuccess ? e : configure<128>();
}

cudaError_t launch_lm_step_q4(const LmShape& sh, const LmStepArgs& a, cudaStream_t s)
{
    return sh.D == 128 ? launch<128>(sh, a, s) : launch<64>(sh, a, s);
}

}  // namespace codec
