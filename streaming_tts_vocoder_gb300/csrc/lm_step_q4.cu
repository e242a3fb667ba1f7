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
// A unit of work is (request, K/V head, split of `chunk` positions), or of the
// part that all requests share (the heads of as many requests as fill 16
// columns, K/V head, split).  Splits lie at fixed positions, so a result's bits do
// not depend on the batch.  A CTA's copy warp takes units one after the other and
// keeps a ring of stages of 64 keys in flight across them; four warps take a tile
// of 16 keys of each, with running softmaxes of their own that are joined at the
// unit's end.  Partial results are joined in order: by the CTA that finishes the
// last unit of a (request, head) where no CTA has more than one unit, else by a
// kernel of its own.
#include <algorithm>

#include "lm.h"
#include "lm_join.cuh"
#include "lm_q4.cuh"
#include "tc_ptx.cuh"

namespace codec {

namespace {

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kKeys = 16 * kConsumers;      // keys of a stage
constexpr int kMaxStages = 6;
// A probability of the reference is 2^kLift; the reference follows when a score
// passes it by more than kSlack (both log2), so that a probability times a scale
// below 2 stays below 2^15.
constexpr float kLift = 6.f, kSlack = 8.f;

struct Params {
    LmShape sh;
    int B, bf16;
    const void* q;
    long long qs;
    const uint8_t *k, *v;
    const uint8_t* zeros;               // a stage's keys that stand for zero
    const int* tables;
    const int* kv_len;
    int table_blocks, bs_shift, n_blocks;
    const int* lead;                    // blocks of the first lead_len positions of every request
    int lead_len;
    int shared_len, n_pre;              // part of its own: length, partial results of it
    int chunk, max_splits;              // shared part: chunk its splits' length
    int per, columns;                   // requests and columns of a unit
    int stages;
    int after_shared;                   // the shared part's kernel is running: nothing here needs its results
    float c;                            // scale x log2 e
    float* part;                        // [B][max_splits][hq][D]
    float* part_lse;
    float* pre;                         // [n_pre][B][hq][D]
    float* pre_lse;
    int* done;                          // [B][hk] finished units; zero between calls
    int* taken;                         // units taken (null: unit = blockIdx, + gridDim, ..); zero between calls
    int* taken_shared;
    void* o;
    long long os;
    float* lse;
};

__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                    const float* c)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// G words at shared address p (8 or 16 bytes).
template <int G>
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t* w)
{
    if constexpr (G == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    }
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"r"(32 * kConsumers) : "memory"); }

__device__ __forceinline__ bool consumers_all(bool ok)
{
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)ok), "n"(32 * kConsumers)
        : "memory");
    return all != 0;
}

struct Unit {
    int b, hk, split, n_splits;     // shared part: first request, -, split, -
    int key0, keys;                 // first position, positions of the split
    bool empty;                     // the request has no position at all
};

// The unit of index u: units run over the requests' splits, K/V heads innermost.
// first, lens: the requests' first units and lengths.  A whole warp: 32 places
// are looked at at once.
__device__ __forceinline__ Unit unit_at(const Params& p, const int* first, const int* lens, int u)
{
    Unit n;
    const int x = u / p.sh.hk;
    n.hk = u - x * p.sh.hk;
    const int lane = threadIdx.x & 31;
    int lo = 0;
    for (int step = p.B <= 32 ? 1 : p.B <= 1024 ? 32 : 1024; step > 0; step >>= 5) {
        const int at = lo + lane * step;
        lo += (__popc(__ballot_sync(0xffffffffu, at < p.B && first[at] <= x)) - 1) * step;
    }
    n.b = lo;
    n.split = x - first[lo];
    n.n_splits = first[lo + 1] - first[lo];
    const int len = lens[lo];
    n.empty = len == 0;
    n.key0 = p.shared_len + n.split * p.chunk;
    n.keys = min(max(len - n.key0, 0), p.chunk);
    return n;
}

// The same of the shared part: requests innermost, then K/V heads, so that the
// units of a split's keys run at about the same time.
__device__ __forceinline__ Unit shared_unit_at(const Params& p, int u)
{
    Unit n;
    const int sets = (p.B + p.per - 1) / p.per, x = u / sets;
    n.b = (u - x * sets) * p.per;
    n.split = x / p.sh.hk;
    n.hk = x - n.split * p.sh.hk;
    n.n_splits = 1;
    n.key0 = n.split * p.chunk;
    n.keys = min(p.shared_len - n.key0, p.chunk);
    n.empty = false;
    return n;
}

__device__ __forceinline__ int splits_of(const Params& p, int len)
{
    return max(1, (max(0, len - p.shared_len) + p.chunk - 1) / p.chunk);
}

template <int D>
__host__ __device__ constexpr uint32_t stage_bytes(int columns)
{
    return 2 * kConsumers * Q4Tile<D>::kBytes + columns * D * 2;
}
// A consumer's results lie [column][D + 4].
template <int D> constexpr int kPitch = D + 4;

// [stages], the consumers' results and their references and sums [4][16][2], the
// barriers, the stages' units and lengths, the requests' first units and lengths.
template <int D>
size_t smem_bytes(int stages, int columns, int B, bool shared)
{
    return 128 + (size_t)stages * stage_bytes<D>(columns) + (size_t)kConsumers * columns * kPitch<D> * 4 +
           kConsumers * 16 * 8 + 2 * kMaxStages * 8 + 16 + kMaxStages * 16 + kMaxStages * 64 +
           (shared ? 0 : (2 * (size_t)B + 1) * 4);
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
    const long long shared_row = (long long)b * p.sh.hq + h, own_row = (long long)b * p.max_splits * p.sh.hq + h;
    auto row_of = [&](int i) {
        return i < p.n_pre ? (long long)i * p.B * p.sh.hq + shared_row : (long long)(i - p.n_pre) * p.sh.hq + own_row;
    };
    float v[kE], lse;
    join_row<kE, kAhead>(
        parts, empty, [&](int i) { return __ldcg((i < p.n_pre ? p.pre_lse : p.part_lse) + row_of(i)); },
        [&](int i, float* x) { row_part<kE>((i < p.n_pre ? p.pre : p.part) + row_of(i) * D, x); }, v, lse);
    uint16_t* row = static_cast<uint16_t*>(p.o) + b * p.os + (long long)h * D;
#pragma unroll
    for (int e = 0; e < kE; e += 2) store2(p, row, (lane * kE + e) / 2, v[e], v[e + 1]);
    if (p.lse && lane == 0) p.lse[(long long)b * p.sh.hq + h] = lse;
}

// A warp per (request, head) whose result is in parts.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) lm_join_q4_kernel(const __grid_constant__ Params p)
{
    pdl_wait();
    pdl_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (p.taken) *p.taken = 0;
        *p.taken_shared = 0;
    }
    const long long w = blockIdx.x * (kJoinThreads / 32LL) + (threadIdx.x >> 5);
    const int b = (int)(w / p.sh.hq), h = (int)(w - (long long)b * p.sh.hq);
    if (b >= p.B) return;
    int len = __ldg(p.kv_len + b);
    lm_clamp_len(len, (long long)p.table_blocks << p.bs_shift);
    const int n = splits_of(p, len);
    if (n == 1 && p.n_pre == 0) return;         // written by its unit
    join_parts<D, 4>(p, b, h, n, len == 0, threadIdx.x & 31);
}

// NT: sets of eight columns.  kShared: units of the shared part, partial results
// to pre.  kJoin: partial results are joined here.
template <int D, int NT, bool kShared, bool kJoin>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) lm_step_q4_kernel(const __grid_constant__ Params p)
{
    using Tile = Q4Tile<D>;
    constexpr int G = Tile::G;
    constexpr uint32_t kTile = Tile::kBytes, kM0 = 0x000f000fu, kM1 = 0x00f000f0u;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
    const uint32_t pitch = stage_bytes<D>(p.columns);
    float* res = reinterpret_cast<float*>(smem + (size_t)p.stages * pitch);
    float* ml = res + kConsumers * p.columns * kPitch<D>;
    uint64_t* full = reinterpret_cast<uint64_t*>(ml + kConsumers * 16 * 2);
    uint64_t* empty = full + kMaxStages;
    int* flags = reinterpret_cast<int*>(empty + kMaxStages);    // abort, last one of a (request, head)
    uint64_t* never = reinterpret_cast<uint64_t*>(flags + 2);   // nothing arrives (see LmShape::unarrived)
    // the unit whose first keys a stage holds: request (-1: no more), K/V head, split and splits << 16, positions
    int4* unit_of = reinterpret_cast<int4*>(flags + 4);
    int* sees = reinterpret_cast<int*>(unit_of + kMaxStages);   // [stage][request of the unit] positions of the split (kShared)
    int* first = sees + kMaxStages * 16;
    int* lens = first + p.B + 1;
    volatile int* abort_flag = flags;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < p.stages; i++) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kConsumers);
        }
        mbar_init(never, 1);
        flags[0] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // Behind the shared part's kernel there is nothing to wait for: what this one
    // reads was complete when that one passed its own wait.  It has to come from L2
    // all the same: lengths and tables by __ldcg, the rest by bulk copies.
    if (!p.after_shared) pdl_wait();
    pdl_launch();
    int* taken = kShared ? p.taken_shared : p.taken;
    int unit0 = blockIdx.x;                 // of the copy warp's lane 0
    if (taken && warp == kConsumers && lane == 0) unit0 = atomicAdd(taken, 1);
    int units;
    if constexpr (kShared) {
        units = p.n_pre * p.sh.hk * ((p.B + p.per - 1) / p.per);
        __syncthreads();
    } else {
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
        units = first[p.B] * p.sh.hk;
    }

    if (warp == kConsumers) {
        // -------------------------------------------------------- copies --
        int st = 0, loads = 0;
        uint32_t ph = 0;
        bool ok = true;
        const int box_tiles = min(1 << (p.bs_shift - 4), kConsumers);   // tiles per box: a block, or half of one of 128
        const int box_shift = box_tiles == 1 ? 4 : box_tiles == 2 ? 5 : 6;
        const int per = kKeys >> box_shift;
        int u = __shfl_sync(0xffffffffu, unit0, 0);
        while (ok) {
            int next = u + gridDim.x;
            if (taken && lane == 0 && u < units) next = atomicAdd(taken, 1);    // needed when this unit's copies are out
            if (u >= units) u = -1;
            Unit n{};
            if (u >= 0) {
                if constexpr (kShared) n = shared_unit_at(p, u);
                else n = unit_at(p, first, lens, u);
            }
            const int* table = kShared ? p.lead : p.tables + (long long)n.b * p.table_blocks;
            const int reqs = kShared ? min(p.per, p.B - n.b) : 1;
            int see = 0;
            if constexpr (kShared) {
                if (u >= 0 && lane < reqs) {
                    int len = __ldcg(p.kv_len + n.b + lane);
                    lm_clamp_len(len, (long long)p.table_blocks << p.bs_shift);
                    // one without any position: its result is not used, so it need not be cut out
                    see = len == 0 ? n.keys : min(max(len - n.key0, 0), n.keys);
                }
            }
            auto tiles_at = [&](int j) { return (n.keys - j * kKeys + 15) >> 4; };      // tiles from stage j on
            auto boxes = [&](int j) { return max(0, min(per, (tiles_at(j) + box_tiles - 1) / box_tiles)); };
            auto position = [&](int j) { return n.key0 + j * kKeys + (lane << box_shift); };
            auto block = [&](int j) {
                const int pos = position(j);
                return lane < boxes(j) ? __ldcg((!kShared && pos < p.lead_len ? p.lead : table) + (pos >> p.bs_shift)) : 0;
            };
            int id_ahead = block(0);
            // a unit without keys, and the end, take a stage without copies
            for (int j = 0; j == 0 || j * kKeys < n.keys; j++) {
                const int here = boxes(j), id = id_ahead;
                id_ahead = block(j + 1);
                long long tile = -1;            // of the cache, -1: none
                if (lane < here) {
                    if (id < 0 || id >= p.n_blocks)
                        atomicOr(p.sh.err, CODEC_LM_ERR_BLOCK);
                    else
                        tile = (((long long)id * p.sh.hk + n.hk) << (p.bs_shift - 4)) +
                               ((position(j) & ((1 << p.bs_shift) - 1)) >> 4);
                }
                ok = mbar_wait(&empty[st], ph ^ 1u, abort_flag, kLmPolls);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t* dst = smem + (size_t)st * pitch;
                if constexpr (kShared)
                    if (j == 0 && lane < 16) sees[st * 16 + lane] = lane < reqs ? see : n.keys;
                // one thread issues them all
                long long tiles[4];
#pragma unroll
                for (int b = 0; b < 4; b++) tiles[b] = __shfl_sync(0xffffffffu, tile, b);
                __syncwarp();
                if (elect_one()) {
                    const bool with_q = j == 0 && here > 0;
                    const int count = min(kConsumers, max(0, tiles_at(j)));
                    const uint32_t q_bytes = p.sh.group * D * 2;
                    if (j == 0)
                        unit_of[st] = make_int4(u < 0 ? -1 : n.b | (n.empty ? 1 << 30 : 0), n.hk, n.split | n.n_splits << 16, n.keys);
                    mbar_expect_tx(&full[st], count * 2 * kTile + (with_q ? reqs * q_bytes : 0));
                    if (with_q)
                        for (int i = 0; i < reqs; i++)
                            bulk_load(dst + 2 * kConsumers * kTile + i * q_bytes,
                                      static_cast<const uint16_t*>(p.q) + (n.b + i) * p.qs + (long long)n.hk * p.sh.group * D,
                                      &full[st], q_bytes);
#pragma unroll
                    for (int b = 0; b < 4; b++)
                        if (b < here) {
                            const int at = b * box_tiles;
                            const uint32_t bytes = min(box_tiles, count - at) * kTile;
                            const bool good = tiles[b] >= 0;
                            bulk_load(dst + at * kTile, good ? p.k + tiles[b] * kTile : p.zeros, &full[st], bytes);
                            bulk_load(dst + (kConsumers + at) * kTile, good ? p.v + tiles[b] * kTile : p.zeros, &full[st], bytes);
                        }
                }
                __syncwarp();
                loads++;
                if (++st == p.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (u < 0) break;
            u = __shfl_sync(0xffffffffu, next, 0);
        }
        // every stage's last load has landed before the CTA can end
        for (int q = 0; q < p.stages && q < loads; q++) {
            const int last = q + ((loads - 1 - q) / p.stages) * p.stages;
            mbar_drain(&full[q], (uint32_t)(last / p.stages) & 1u);
        }
    } else {
        // ------------------------------------------------------ consumers --
        const int r = lane >> 2, t = lane & 3;      // row (and + 8) and column pair of a fragment
        const int c0 = 2 * t;                       // first of this lane's two columns of a set
        int st = 0;
        uint32_t ph = 0;
        // When a wait gives up inside a unit its warps still meet at the unit's
        // barriers; at the next unit they all leave, whatever has landed by then.
        bool gave_up = false;
        while (true) {
            if (!consumers_all(!gave_up && mbar_wait(&full[st], ph, abort_flag, kLmPolls))) break;
            const int4 unit = unit_of[st];
            if (unit.x < 0) break;
            Unit n;
            n.b = unit.x & 0xffff;
            n.hk = unit.y;
            n.split = unit.z & 0xffff;
            n.n_splits = unit.z >> 16;
            n.keys = unit.w;
            n.empty = unit.x >> 30;
            const int group = p.sh.group;
            // positions that this lane's columns see, and the one whose row it is when transposed
            int sees2[NT][2], sees_t[NT], all_see = n.keys, some_see = n.keys;
#pragma unroll
            for (int x = 0; x < NT; x++) {
                sees2[x][0] = sees2[x][1] = sees_t[x] = n.keys;
                if constexpr (kShared) {
                    auto of = [&](int col) { return sees[st * 16 + min(col, p.columns - 1) / group]; };
                    sees2[x][0] = of(8 * x + c0);
                    sees2[x][1] = of(8 * x + c0 + 1);
                    sees_t[x] = of(8 * x + r);
                    const int lo = __reduce_min_sync(0xffffffffu, sees_t[x]), hi = __reduce_max_sync(0xffffffffu, sees_t[x]);
                    all_see = min(all_see, lo);
                    some_see = x == 0 ? hi : max(some_see, hi);
                }
            }
            uint32_t qf[NT][G][4], ql[NT];          // queries and their groups' sums
            float cf[NT][2];                        // of this lane's columns: what makes a score of an accumulator
            float acc[NT][G][2][4], low[NT][4];
            float ref[NT][2], l[NT][2];
#pragma unroll
            for (int x = 0; x < NT; x++) {
#pragma unroll
                for (int g = 0; g < G; g++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[x][g][0][e] = acc[x][g][1][e] = 0.f;
#pragma unroll
                for (int e = 0; e < 4; e++) low[x][e] = 0.f;
                ref[x][0] = ref[x][1] = -INFINITY;
                l[x][0] = l[x][1] = 0.f;
            }
            int grown = 0;                          // scales are below 2^(1 + grown)
            for (int j = 0; j == 0 || j * kKeys < n.keys; j++) {
                // (unarrived: one warp's second stage never comes)
                const bool ok = j == 0 || (p.sh.unarrived && warp == 0 && j == 1
                                               ? mbar_wait(never, 0, abort_flag, p.sh.unarrived)
                                               : mbar_wait(&full[st], ph, abort_flag, kLmPolls));
                gave_up = !__all_sync(0xffffffffu, ok);
                if (gave_up) break;
                const uint8_t* stage = smem + (size_t)st * pitch;
                if (j == 0 && n.keys > 0) {
                    // Column r of each set, elements 8 t .. 8 t + 7 of each group, times the power
                    // of two that brings its largest to 2^14 .. 2^15: exact as halves but for what
                    // lies 2^38 below.  Columns behind the last repeat it: nobody reads them.
#pragma unroll
                    for (int x = 0; x < NT; x++) {
                        const uint8_t* row = stage + 2 * kConsumers * kTile + min(8 * x + r, p.columns - 1) * D * 2 + t * 16;
                        float f[G][8], top = 0.f;
#pragma unroll
                        for (int g = 0; g < G; g++) {
                            uint32_t w[4];
                            lds<4>(row + g * 64, w);
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float2 y = p.bf16 ? __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w[e]))
                                                        : __half22float2(*reinterpret_cast<__half2*>(&w[e]));
                                f[g][2 * e] = y.x;
                                f[g][2 * e + 1] = y.y;
                                top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
                            }
                        }
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        const int e2 = (int)(__float_as_uint(top) >> 23);       // 255: not finite
                        const int lift = e2 == 255 ? 0 : min(127 + 14 - e2, 100);
                        const float m = __int_as_float((127 + lift) << 23);
                        float mine = 0.f;
#pragma unroll
                        for (int g = 0; g < G; g++) {
                            float sum = 0.f;
#pragma unroll
                            for (int e = 0; e < 8; e++) {
                                f[g][e] *= m;
                                sum += f[g][e];
                            }
                            qf[x][g][0] = pack(f[g][0], f[g][4]);
                            qf[x][g][1] = pack(f[g][2], f[g][6]);
                            qf[x][g][2] = pack(f[g][1] * 0.0625f, f[g][5] * 0.0625f);
                            qf[x][g][3] = pack(f[g][3] * 0.0625f, f[g][7] * 0.0625f);
                            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                            if (g == t) mine = sum;
                        }
                        mine *= 0x1p-6f;
                        const float hi = __half2float(__float2half_rn(mine));
                        ql[x] = pack(hi, mine - hi);
                        // an accumulator holds scores times 2^(lift - 24)
                        const float back = fminf(p.c * __int_as_float((127 - lift) << 23) * 0x1p24f, 3e38f);
                        cf[x][0] = __shfl_sync(0xffffffffu, back, c0 * 4);
                        cf[x][1] = __shfl_sync(0xffffffffu, back, c0 * 4 + 4);
                    }
                }
                const int at = j * kKeys + warp * 16;           // of the warp's tile in the split
                if (at < n.keys) {
                    const uint8_t *kt = stage + warp * kTile, *vt = kt + kConsumers * kTile;
                    float s[NT][4];
                    {
                        uint32_t ka[G], kb[G], pa[G], pb[G];
                        lds<G>(kt + r * (D / 2) + t * 4 * G, ka);
                        lds<G>(kt + (r + 8) * (D / 2) + t * 4 * G, kb);
                        lds<G>(kt + Tile::kParams + r * 4 * G, pa);
                        lds<G>(kt + Tile::kParams + (r + 8) * 4 * G, pb);
                        uint32_t la = 0, lb = 0;
                        if (G == 4 || t < G) {
                            la = __byte_perm(*reinterpret_cast<const uint32_t*>(kt + Tile::kParams + (r * G + t) * 4), 0, 0x3232);
                            lb = __byte_perm(*reinterpret_cast<const uint32_t*>(kt + Tile::kParams + ((r + 8) * G + t) * 4), 0, 0x3232);
                        }
                        const float zero[4] = {};
#pragma unroll
                        for (int x = 0; x < NT; x++) {
                            mma(s[x], la, lb, 0u, 0u, ql[x], 0u, zero);
#pragma unroll
                            for (int e = 0; e < 4; e++) s[x][e] *= 0x1p-18f;
                        }
#pragma unroll
                        for (int g = 0; g < G; g++) {
                            const uint32_t ha = ka[g] >> 8, hb = kb[g] >> 8;
                            const float sa = low_half(pa[g]), sb = low_half(pb[g]);
#pragma unroll
                            for (int x = 0; x < NT; x++) {
                                float d[4];
                                mma(d, ka[g] & kM0, kb[g] & kM0, ha & kM0, hb & kM0, qf[x][g][0], qf[x][g][1], zero);
                                mma(d, ka[g] & kM1, kb[g] & kM1, ha & kM1, hb & kM1, qf[x][g][2], qf[x][g][3], d);
                                s[x][0] = fmaf(sa, d[0], s[x][0]);
                                s[x][1] = fmaf(sa, d[1], s[x][1]);
                                s[x][2] = fmaf(sb, d[2], s[x][2]);
                                s[x][3] = fmaf(sb, d[3], s[x][3]);
                            }
                        }
                    }
                    // values: codes of keys 2 t, 2 t + 1 and of those 8 further; scales and lows of the same
                    uint32_t va[G], vb[G], sc[2 * G], vl[2] = {0u, 0u};
                    lds<G>(vt + lane * 4 * G, va);
                    lds<G>(vt + 4 * D + lane * 4 * G, vb);
                    lds<4>(vt + Tile::kParams + t * 8 * G, sc);
                    if constexpr (G == 4) lds<4>(vt + Tile::kParams + t * 8 * G + 16, sc + 4);
                    if (r < G) lds<2>(vt + Tile::kParams + D + (t * G + r) * 8, vl);
#pragma unroll
                    for (int x = 0; x < NT; x++)
#pragma unroll
                        for (int e = 0; e < 4; e++) s[x][e] *= cf[x][e & 1];
                    const bool cut = at + 16 > all_see;
                    if (cut) {
                        // what a column does not see may be anything
#pragma unroll
                        for (int x = 0; x < NT; x++)
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                if (at + r + (e >> 1) * 8 >= sees2[x][e & 1]) s[x][e] = -INFINITY;
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int k0 = at + c0 + 8 * h;
                            const uint32_t keep = (k0 < some_see ? 0xffffu : 0u) | (k0 + 1 < some_see ? 0xffff0000u : 0u);
#pragma unroll
                            for (int g = 0; g < G; g++) sc[2 * g + h] &= keep;
                            vl[h] &= keep;
                        }
                        // a low that is not finite would reach every column: it goes by its scale, as NaN
                        if constexpr (kShared) {
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const uint32_t wild = ((vl[h] & 0x7c00u) == 0x7c00u ? 0x0000ffffu : 0u) |
                                                      ((vl[h] & 0x7c000000u) == 0x7c000000u ? 0xffff0000u : 0u);
                                vl[h] &= ~wild;
#pragma unroll
                                for (int g = 0; g < G; g++) sc[2 * g + h] |= __shfl_sync(0xffffffffu, wild, g * 4 + t);
                            }
                        }
                    }
                    uint32_t or_of = sc[0] | sc[1] | sc[2];
#pragma unroll
                    for (int g = 3; g < 2 * G; g++) or_of |= sc[g];
                    or_of &= 0x7fff7fffu;
                    bool move = max(or_of & 0xffffu, or_of >> 16) >= (uint32_t)(16 + grown) << 10;
#pragma unroll
                    for (int x = 0; x < NT; x++)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            move |= s[x][e] - ref[x][e & 1] > kSlack;
                        }
                    if (__any_sync(0xffffffffu, move)) {
                        // the largest exponent among the scales (31: not finite, follows from nothing)
                        int e = 0;
#pragma unroll
                        for (int g = 0; g < 2 * G; g++) {
                            const int lo = sc[g] >> 10 & 31, hi = sc[g] >> 26 & 31;
                            e = max(e, max(lo == 31 ? 0 : lo, hi == 31 ? 0 : hi));
                        }
                        const int want = max(grown, (int)__reduce_max_sync(0xffffffffu, e) - 15);
                        const float shrink = __int_as_float((127 - (want - grown)) << 23);
                        grown = want;
                        // a column's reference moves for its own scores alone (times 1 changes nothing)
#pragma unroll
                        for (int x = 0; x < NT; x++)
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                float m = fmaxf(s[x][h], s[x][2 + h]);
                                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                                const bool up = m - ref[x][h] > kSlack;
                                const float f = (!up ? 1.f : ref[x][h] == -INFINITY ? 0.f : exp2_fast(ref[x][h] - m)) * shrink;
                                ref[x][h] = up ? m : ref[x][h];
                                l[x][h] *= f;
#pragma unroll
                                for (int g = 0; g < G; g++)
#pragma unroll
                                    for (int i = 0; i < 2; i++) {
                                        acc[x][g][i][h] *= f;
                                        acc[x][g][i][2 + h] *= f;
                                    }
                                low[x][h] *= f;
                            }
                    }
                    const float lift = kLift - (float)grown;
#pragma unroll
                    for (int x = 0; x < NT; x++) {
                        const float b0 = ref[x][0] == -INFINITY ? 0.f : lift - ref[x][0];
                        const float b1 = ref[x][1] == -INFINITY ? 0.f : lift - ref[x][1];
                        const float p0 = exp2_fast(s[x][0] + b0), p1 = exp2_fast(s[x][1] + b1);
                        const float p2 = exp2_fast(s[x][2] + b0), p3 = exp2_fast(s[x][3] + b1);
                        l[x][0] += p0 + p2;
                        l[x][1] += p1 + p3;
                        const uint32_t f0 = transposed(pack(p0, p1)), f1 = transposed(pack(p2, p3));
                        mma(low[x], vl[0], 0u, vl[1], 0u, f0, f1, low[x]);
                        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                        if (cut) {
                            const int k0 = at + c0;
                            keep0 = (k0 < sees_t[x] ? 0xffffu : 0u) | (k0 + 1 < sees_t[x] ? 0xffff0000u : 0u);
                            keep1 = (k0 + 8 < sees_t[x] ? 0xffffu : 0u) | (k0 + 9 < sees_t[x] ? 0xffff0000u : 0u);
                        }
#pragma unroll
                        for (int g = 0; g < G; g++) {
                            const uint32_t g0 = times(f0, sc[2 * g]) & keep0, g1 = times(f1, sc[2 * g + 1]) & keep1;
                            const uint32_t ha = va[g] >> 8, hb = vb[g] >> 8;
                            mma(acc[x][g][0], va[g] & kM0, va[g] & kM1, vb[g] & kM0, vb[g] & kM1, g0, g1, acc[x][g][0]);
                            mma(acc[x][g][1], ha & kM0, ha & kM1, hb & kM0, hb & kM1, g0, g1, acc[x][g][1]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
                if (++st == p.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            // results of the warp: sums of codes are 2^-24 of what they stand for, and 2^-20 for
            // a group's elements 1 and 3 of four
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    l[x][h] += __shfl_xor_sync(0xffffffffu, l[x][h], 4);
                    l[x][h] += __shfl_xor_sync(0xffffffffu, l[x][h], 8);
                    l[x][h] += __shfl_xor_sync(0xffffffffu, l[x][h], 16);
                    const int col = 8 * x + c0 + h;
                    float* dst = res + (warp * p.columns + min(col, p.columns - 1)) * kPitch<D> + r * 4;
#pragma unroll
                    for (int g = 0; g < G; g++) {
                        const float add = __shfl_sync(0xffffffffu, low[x][h], g * 4 + t);
                        const float4 v = make_float4(fmaf(acc[x][g][0][h], 0x1p24f, add), fmaf(acc[x][g][0][2 + h], 0x1p20f, add),
                                                     fmaf(acc[x][g][1][h], 0x1p24f, add), fmaf(acc[x][g][1][2 + h], 0x1p20f, add));
                        if (col < p.columns) *reinterpret_cast<float4*>(dst + g * 32) = v;
                    }
                    if (r == 0 && col < p.columns) {
                        // the exponent that a probability of 1 has
                        ml[(warp * 16 + col) * 2] = ref[x][h] == -INFINITY ? -INFINITY : ref[x][h] - kLift + (float)grown;
                        ml[(warp * 16 + col) * 2 + 1] = l[x][h];
                    }
                }
            consumers_sync();
            const bool alone = !kShared && n.n_splits == 1 && p.n_pre == 0;
            for (int e = tid; e < p.columns * (D / 4); e += 32 * kConsumers) {
                const int col = e / (D / 4), d = (e - col * (D / 4)) * 4;
                const int b = kShared ? n.b + col / group : n.b, h = n.hk * group + (kShared ? col % group : col);
                if (kShared && b >= p.B) continue;
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < kConsumers; w++) m = fmaxf(m, ml[(w * 16 + col) * 2]);
                float sum = 0.f;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kConsumers; w++) {
                    const float mw = ml[(w * 16 + col) * 2], lw = ml[(w * 16 + col) * 2 + 1];
                    // a warp without keys has a sum of 0; one whose scores are all NaN has no reference and a sum of NaN
                    const float f = mw == -INFINITY ? (lw == 0.f ? 0.f : 1.f) : exp2_fast(mw - m);
                    const float4 y = *reinterpret_cast<const float4*>(res + (w * p.columns + col) * kPitch<D> + d);
                    if (f != 0.f) {
                        sum = fmaf(f, lw, sum);
                        v.x = fmaf(f, y.x, v.x);
                        v.y = fmaf(f, y.y, v.y);
                        v.z = fmaf(f, y.z, v.z);
                        v.w = fmaf(f, y.w, v.w);
                    }
                }
                const bool none = sum == 0.f;           // no key, or none that it sees
                const float inv = none ? 0.f : 1.f / sum;
                v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                const float lse = none ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(sum)) * 0.6931471805599453f;
                if (alone) {
                    uint16_t* row = static_cast<uint16_t*>(p.o) + b * p.os + (long long)h * D;
                    store2(p, row, d / 2, v.x, v.y);
                    store2(p, row, d / 2 + 1, v.z, v.w);
                    if (p.lse && d == 0) p.lse[(long long)b * p.sh.hq + h] = lse;
                } else {
                    const long long at = kShared ? ((long long)n.split * p.B + b) * p.sh.hq + h
                                                 : ((long long)b * p.max_splits + n.split) * p.sh.hq + h;
                    __stcg(reinterpret_cast<float4*>((kShared ? p.pre : p.part) + at * D + d), v);
                    if (d == 0) __stcg((kShared ? p.pre_lse : p.part_lse) + at, lse);
                }
            }
            consumers_sync();                   // res is written again
            if constexpr (kJoin) {
                if (alone) continue;
                if (tid == 0) {
                    // releases the CTA's results (ordered before it by the barrier) and
                    // acquires those of the others
                    int* done = p.done + (long long)n.b * p.sh.hk + n.hk;
                    int was = 0;
                    if (n.n_splits > 1)
                        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(was) : "l"(done) : "memory");
                    flags[1] = was == n.n_splits - 1;
                    if (flags[1] && n.n_splits > 1) *done = 0;
                }
                consumers_sync();
                if (!flags[1]) continue;
                for (int g = warp; g < group; g += kConsumers)
                    join_parts<D, 12>(p, n.b, n.hk * group + g, n.n_splits, n.empty, lane);
            }
        }
    }
    __syncthreads();
    if (tid == 0 && flags[0]) atomicOr(p.sh.err, CODEC_LM_ERR_TIMEOUT);
    // this kernel's end is its predecessors' too
    if (p.after_shared) pdl_wait();
}

// Stages and CTAs per SM: as many CTAs as registers allow, with two stages at least.
template <int D>
void fit(Params& p, int most_per_sm, bool shared, int& per_sm)
{
    constexpr size_t kSm = 228 * 1024, kOne = 227 * 1024;
    for (per_sm = most_per_sm; per_sm >= 1; per_sm--) {
        p.stages = kMaxStages;
        auto fits = [&] {
            const size_t n = smem_bytes<D>(p.stages, p.columns, p.B, shared);
            return n <= kOne && per_sm * (n + 1024) <= kSm;
        };
        while (p.stages > 2 && !fits()) p.stages--;
        if (fits()) return;
    }
    per_sm = 1;
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
    p.chunk = a.ws.chunk;
    p.max_splits = a.ws.max_splits;
    p.c = (float)(sh.scale * 1.4426950408889634);
    p.part = a.ws.part;
    p.part_lse = a.ws.part_lse;
    p.pre = a.ws.pre;
    p.pre_lse = a.ws.pre_lse;
    p.done = a.ws.done;
    p.taken_shared = a.ws.taken + 1;
    p.o = a.o;
    p.os = a.os;
    p.lse = a.lse;
    p.per = 1;
    p.columns = sh.group;
    p.lead = a.shared_table;
    const bool wide = sh.group > 8;
    // A short shared part is read by every request.
    const long long most_short = p.shared_len <= 256 ? 65536 : p.shared_len <= 1024 ? 32768 : 0;
    if (a.ws.heads == sh.hk || a.ws.heads * p.shared_len <= most_short) {
        p.lead_len = p.shared_len;
        p.shared_len = 0;
    }
    int per_sm = 1;
    if (p.shared_len > 0) {
        Params c = p;
        c.per = 16 / sh.group;
        c.columns = c.per * sh.group;
        // splits by the object's shape and the shared length alone
        const int n = lm_shared_splits_q4(a.ws.heads / sh.hk, sh.hk, sh.group, p.shared_len);
        c.chunk = ((p.shared_len + n - 1) / n + kKeys - 1) / kKeys * kKeys;
        p.n_pre = c.n_pre = (p.shared_len + c.chunk - 1) / c.chunk;
        fit<D>(c, 2, true, per_sm);
        const long long units = (long long)c.n_pre * sh.hk * ((a.B + c.per - 1) / c.per);
        const cudaError_t e = launch_pdl(lm_step_q4_kernel<D, 2, true, false>, dim3((unsigned)std::min<long long>(152 * per_sm, units)),
                                         dim3(kThreads), smem_bytes<D>(c.stages, c.columns, c.B, true), s, c);
        if (e != cudaSuccess) return e;
        p.after_shared = 1;
    }
    fit<D>(p, wide ? 2 : 3, false, per_sm);
    // a unit per request and head at least, and no more CTAs than the SMs hold at once
    const long long most = (long long)a.B * p.max_splits * sh.hk;
    const unsigned ctas = (unsigned)std::min<long long>(152 * per_sm, most);
    // joined in this kernel where a CTA has one unit at most and needs no other kernel's results
    const bool join = most <= ctas && p.n_pre == 0, two = !join && (p.n_pre > 0 || p.max_splits > 1);
    p.taken = two ? a.ws.taken : nullptr;
    auto kernel = wide ? (join ? lm_step_q4_kernel<D, 2, false, true> : lm_step_q4_kernel<D, 2, false, false>)
                       : (join ? lm_step_q4_kernel<D, 1, false, true> : lm_step_q4_kernel<D, 1, false, false>);
    const cudaError_t e = launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem_bytes<D>(p.stages, p.columns, a.B, false), s, p);
    if (e != cudaSuccess || !two) return e;
    return launch_pdl(lm_join_q4_kernel<D>, dim3((unsigned)(((long long)a.B * sh.hq + kJoinThreads / 32 - 1) / (kJoinThreads / 32))),
                      dim3(kJoinThreads), 0, s, p);
}

template <int D>
cudaError_t configure()
{
    const void* kernels[] = {(const void*)lm_step_q4_kernel<D, 1, false, false>, (const void*)lm_step_q4_kernel<D, 1, false, true>,
                             (const void*)lm_step_q4_kernel<D, 2, false, false>, (const void*)lm_step_q4_kernel<D, 2, false, true>,
                             (const void*)lm_step_q4_kernel<D, 2, true, false>};
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
