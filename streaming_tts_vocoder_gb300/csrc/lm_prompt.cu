// Attention of many query rows over the same keys, on the tensor cores: whole
// prompts (packed or behind a cached context) and, for single tokens, the part
// of the context that all requests share.
//
// o = softmax(scale q K^T) V in one pass over the keys, 128 at a time.  With
// the scores in log2 units (c = scale log2 e) a row keeps a reference r >= its
// maximum - 8 and l = sum 2^(c s - c r); when a tile's maximum passes r by more
// than 8, l and the output accumulator are scaled down once and r moves up.
// (r need not be the maximum: it cancels in o / l, and 2^8 is far from any
// overflow.)  Scores, r, l and the accumulator are fp32; the probabilities are
// rounded to the operands' type for the second product, as every 16-bit
// tensor-core attention must, and l sums them before that rounding.
//
// Rows of a tile are (token, query head) pairs of one K/V head, so grouped
// heads share every K/V tile that is loaded: 128 / group tokens per tile, two
// tiles per CTA.  Per 128 keys a tile is S = Q K^T (K-major operands in shared
// memory), a softmax of one row per thread, and O += P V with P read from TMEM
// (it overwrites its scores there) and V in its natural layout as the MN-major
// operand.  TMEM: two score tiles of 128 columns and two accumulators of D.
//
// Roles (384 threads, one CTA per SM):
//   warp 0      copies: Q once, then K and V tiles through a ring of stages;
//               paged keys one box per cache block, one block per lane
//   warp 1      TMEM and MMA issue: the MMAs of one tile run while the
//               softmax of the other does
//   warps 2, 3  V tiles that hold keys some row may not see: rows nobody sees
//               are zeroed, and so is what is not finite (0 x NaN is NaN, so a
//               probability of zero would not keep it out); where it was is
//               noted, and the rows that do see it get it back at the end
//   warps 4-11  softmax, four warps per tile; they also rescale the
//               accumulator and write the result
// Every wait is bounded: when one expires the CTA raises the error bit, stops,
// drains its copies and MMAs, frees TMEM and returns.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "lm.h"
#include "tc_ptx.cuh"

namespace codec {

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;                  // rows of a query tile, keys of a K/V tile
constexpr uint32_t kHalfBytes = kTile * 128;    // 64 columns of a tile: 128 rows of 128 bytes
constexpr int kMaxStages = 8;
constexpr uint32_t kPolls = 1u << 22;
constexpr int kNone = 0x7fffffff;

struct Params {
    LmShape sh;
    int rows;                   // query rows (requests, for a shared part)
    const int* row_start;       // null: a shared part, query row t is request t
    int B;
    const int* tables;          // null: packed keys
    const int* kv_len;
    int table_blocks, bs_shift, n_blocks;
    int shared_len, split_len;  // shared part: its length, and keys per blockIdx.z
    int tokens;                 // tokens per query tile: 128 / group
    float c;                    // scale x log2 e
    uint32_t idesc_s, idesc_o;
    void* o;
    long long os;
    float* lse;
    float* part;                // shared part: [split][rows][hq][D], normalised, fp32
    float* part_lse;            // [split][rows][hq]
};

// What the CTA works on; filled once.
struct Item {
    int b;                      // request
    int q0;                     // first query row
    int ntok;                   // tokens of the two tiles that exist
    int key0;                   // packed: row of key 0; else key 0's position
    int end;                    // keys at or behind it: seen by no row
    int free_from;              // keys below it: seen by every row that sees any
    int n[2];                   // K/V tiles of each query tile
};

// MN-major operand with 128-byte swizzle: 64 elements of N in a 128-byte row
// per k; 8-row groups 1024 bytes apart (stride byte offset), the next 64
// elements of N one half tile further (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kHalfBytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// D[tmem] (+)= A[tmem] x B[shared]
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations per instruction, on register pairs.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(*reinterpret_cast<uint64_t*>(&d))
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
          "l"(*reinterpret_cast<const uint64_t*>(&c)));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<uint64_t*>(&d))
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> {
    static constexpr uint32_t kFormat = 1;              // MMA operand format
    static constexpr uint32_t kExp = 0x7f807f80u, kOne = 0x00800080u;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float one(uint32_t h) { return __uint_as_float(h << 16); }
};
template <> struct Two<__half> {
    static constexpr uint32_t kFormat = 0;
    static constexpr uint32_t kExp = 0x7c007c00u, kOne = 0x04000400u;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float one(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)h)); }
};

// Which of a word's two values is not finite, as bits 15 and 31.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    return ((w & Two<T>::kExp) + Two<T>::kOne) & 0x80008000u;
}

template <int D> constexpr int stages() { return D == 128 ? 5 : 8; }

struct Shared {
    uint64_t q_full, drain;
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t raw[kMaxStages], clean[kMaxStages];    // V tiles that are cleaned before use: landed, cleaned
    uint64_t s_full[2], p_full[2][2], o_full[2];
    uint32_t tmem;
    int abort;
    Item item;
    int any_bad;
    int scan[kThreads / 32];
    int found;
    int lim[2 * kTile];         // keys each token sees
    int bad[3][128];            // first key whose value in this column is NaN, +inf, -inf
};

template <int D> constexpr uint32_t tile_bytes() { return kTile * D * 2; }
static_assert(sizeof(Shared) <= 227 * 1024 - 7 * 32768, "five stages of 32 KB beside two query tiles");
template <int D> constexpr size_t smem_bytes()
{
    return (size_t)(2 + stages<D>()) * tile_bytes<D>() + sizeof(Shared);
}

// Finds the CTA's request and query rows: item x of the requests' tile pairs,
// in request order, each request's last (longest) pair first.  All threads.
__device__ bool find_item(const Params& p, Shared& s)
{
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int pair = 2 * p.tokens;
    const bool report = blockIdx.x == 0 && blockIdx.y == 0;
    int before = 0;
    for (int base = 0; base < p.B; base += kThreads) {
        const int b = base + tid;
        int first = 0, n = 0, tiles = 0;
        if (b < p.B) {
            if (!lm_rows(p.row_start, b, p.rows, first, n) && report) atomicOr(p.sh.err, CODEC_LM_ERR_LENGTH);
            tiles = (n + pair - 1) / pair;
        }
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) s.scan[w] = incl;
        __syncthreads();
        int at = before, total = 0;
        for (int i = 0; i < kThreads / 32; i++) {
            if (i < w) at += s.scan[i];
            total += s.scan[i];
        }
        at += incl - tiles;
        const int x = (int)blockIdx.x - at;
        if (x >= 0 && x < tiles) {
            const int t = tiles - 1 - x;
            s.item.b = b;
            s.item.q0 = first + t * pair;
            s.item.ntok = min(pair, n - t * pair);
            s.item.key0 = p.tables ? 0 : first;
            int keys = n;
            if (p.tables) {
                keys = __ldg(p.kv_len + b);
                if (!lm_clamp_len(keys, (long long)p.table_blocks << p.bs_shift))
                    atomicOr(p.sh.err, CODEC_LM_ERR_LENGTH);
            }
            // the first token's keys (others see one more each), before the clamp at 0
            s.item.end = keys - n + t * pair + 1;
            s.found = 1;
        }
        before += total;
        __syncthreads();
        if (s.found && !report) break;
    }
    return s.found != 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) lm_prompt_kernel(const __grid_constant__ CUtensorMap mq,
                                                                const __grid_constant__ CUtensorMap mk,
                                                                const __grid_constant__ CUtensorMap mv,
                                                                const __grid_constant__ Params p)
{
    constexpr int kStages = stages<D>();
    constexpr uint32_t kBytes = tile_bytes<D>();
    constexpr int kHalves = D / 64;
    constexpr uint32_t kTmem = 512;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sq = smem;                                 // two query tiles
    uint8_t* skv = smem + 2 * kBytes;                   // ring: K tile, V tile, K tile, ...
    Shared& s = *reinterpret_cast<Shared*>(skv + (size_t)kStages * kBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hk = blockIdx.y;

    if (tid == 0) {
        mbar_init(&s.q_full, 1);
        mbar_init(&s.drain, 1);
        for (int i = 0; i < kStages; i++) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
            mbar_init(&s.raw[i], 1);
            mbar_init(&s.clean[i], 2);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i][0], 4);
            mbar_init(&s.p_full[i][1], 4);
            mbar_init(&s.o_full[i], 1);
        }
        s.abort = 0;
        s.any_bad = 0;
        s.found = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < 3 * 128; i += kThreads) (&s.bad[0][0])[i] = kNone;
    __syncthreads();
    pdl_wait();
    pdl_launch();

    // ---- what to work on ----
    if (p.row_start) {
        if (!find_item(p, s)) return;       // the same for all threads, and before TMEM is taken
        const int first = s.item.end;
        __syncthreads();
        for (int t = tid; t < 2 * kTile; t += kThreads)
            s.lim[t] = t < s.item.ntok ? max(0, first + t) : 0;
    } else {
        const int q0 = blockIdx.x * 2 * p.tokens, k0 = blockIdx.z * p.split_len;
        const int ntok = min(2 * p.tokens, p.rows - q0);
        for (int t = tid; t < 2 * kTile; t += kThreads) {
            int n = 0;
            if (t < ntok) {
                n = __ldg(p.kv_len + q0 + t);
                lm_clamp_len(n, (long long)p.table_blocks << p.bs_shift);
                n = min(max(min(n, p.shared_len) - k0, 0), p.split_len);
            }
            s.lim[t] = n;
        }
        if (tid == 0) {
            s.item.b = 0;
            s.item.q0 = q0;
            s.item.ntok = ntok;
            s.item.key0 = k0;
        }
    }
    __syncthreads();
    if (warp == 0) {                        // the largest and the smallest number of keys but none
        int most[2] = {0, 0}, least = kNone;
        for (int t = lane; t < s.item.ntok; t += 32) {
            const int n = s.lim[t], i = t >= p.tokens;
            most[i] = max(most[i], n);
            if (n > 0) least = min(least, n);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            most[0] = max(most[0], __shfl_xor_sync(0xffffffffu, most[0], o));
            most[1] = max(most[1], __shfl_xor_sync(0xffffffffu, most[1], o));
            least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        }
        if (lane == 0) {
            s.item.end = max(most[0], most[1]);
            s.item.free_from = least;
            s.item.n[0] = (most[0] + kTile - 1) / kTile;
            s.item.n[1] = (most[1] + kTile - 1) / kTile;
        }
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Item it = s.item;
    const uint32_t tmem = s.tmem;
    volatile int* abort_flag = &s.abort;
    const int n_max = max(it.n[0], it.n[1]);
    // tiles from here on hold keys that some row does not see
    const int first_masked = it.free_from / kTile;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
        if (warp == 0) {
            // ------------------------------------------------------ copies --
            int st = 0;
            uint32_t ph = 0;
            uint32_t full_n = 0, raw_n = 0, full_any = 0, raw_any = 0;  // uses of each stage's barriers: parity, any
            bool ok = true;
            if (n_max > 0 && lane == 0) {
                prefetch_tensormap(&mq);
                prefetch_tensormap(&mk);
                prefetch_tensormap(&mv);
                const int tiles = it.n[1] > 0 ? 2 : 1;
                const int g = p.sh.group;
                mbar_expect_tx(&s.q_full, (uint32_t)(tiles * p.tokens * g * D * 2));
                for (int i = 0; i < tiles; i++)
                    for (int h = 0; h < kHalves; h++)
                        tma_load_3d(sq + i * kBytes + h * kHalfBytes, &mq, &s.q_full, h * 64, hk * g,
                                    it.q0 + i * p.tokens);
            }
            const int per = kTile >> p.bs_shift;        // cache blocks per tile
            const int* table = p.tables + (p.row_start ? (long long)it.b * p.table_blocks : 0LL) +
                               (it.key0 >> p.bs_shift);
            const int blocks = (it.end + (1 << p.bs_shift) - 1) >> p.bs_shift;
            int next = 0;
            if (p.tables && lane < min(per, blocks)) next = __ldg(table + lane);
            for (int j = 0; j < n_max && ok; j++) {
                int id = next;
                const int here = p.tables ? min(per, blocks - j * per) : 1;
                if (p.tables) {
                    const int at = (j + 1) * per + lane;
                    if (lane < per && at < blocks) next = __ldg(table + at);
                    if (lane < here && (id < 0 || id >= p.n_blocks)) {
                        atomicOr(p.sh.err, CODEC_LM_ERR_BLOCK);
                        id = p.n_blocks;                // behind the last row: the copy writes zeros
                    }
                }
                for (int kv = 0; kv < 2; kv++) {
                    ok = mbar_wait(&s.empty[st], ph ^ 1u, abort_flag, kPolls);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint8_t* dst = skv + (size_t)st * kBytes;
                    const CUtensorMap* map = kv ? &mv : &mk;
                    const bool clean = kv && j >= first_masked;
                    uint64_t* bar = clean ? &s.raw[st] : &s.full[st];
                    if (clean) {
                        raw_n ^= 1u << st;
                        raw_any |= 1u << st;
                    } else {
                        full_n ^= 1u << st;
                        full_any |= 1u << st;
                    }
                    if (lane == 0)
                        mbar_expect_tx(bar, p.tables ? (uint32_t)(here << p.bs_shift) * D * 2 : kBytes);
                    __syncwarp();
                    if (p.tables) {
                        if (lane < here)
                            for (int h = 0; h < kHalves; h++)
                                tma_load_3d(dst + h * kHalfBytes + ((uint32_t)lane << p.bs_shift) * 128, map,
                                            bar, h * 64, hk, id << p.bs_shift);
                    } else if (lane == 0) {
                        for (int h = 0; h < kHalves; h++)
                            tma_load_3d(dst + h * kHalfBytes, map, bar, h * 64, hk, it.key0 + j * kTile);
                    }
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            // every stage's last load has landed before the CTA can end
            for (int q = 0; q < kStages; q++) {
                if (full_any >> q & 1u) mbar_drain(&s.full[q], (full_n >> q & 1u) ^ 1u);
                if (raw_any >> q & 1u) mbar_drain(&s.raw[q], (raw_n >> q & 1u) ^ 1u);
            }
            if (n_max > 0) mbar_drain(&s.q_full, 0);
        } else if (warp == 1) {
            // -------------------------------------------------------- MMAs --
            if (n_max > 0 && elect_one()) {
                const uint32_t q_addr = smem_u32(sq), kv_addr = smem_u32(skv);
                uint32_t full_ph = 0, clean_ph = 0;     // parity of each stage's barriers
                auto landed = [&](int st) {
                    const bool in = mbar_wait(&s.full[st], full_ph >> st & 1u, abort_flag, kPolls);
                    full_ph ^= 1u << st;
                    return in;
                };
                auto score = [&](int i, int st) {       // S_i = Q_i K^T
                    const uint64_t a0 = sdesc_sw128(q_addr + i * kBytes), b0 = sdesc_sw128(kv_addr + st * kBytes);
#pragma unroll
                    for (int k = 0; k < D / 16; k++) {
                        const uint64_t off = (uint64_t)(((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4);
                        mma_f16(tmem + i * 128, a0 + off, b0 + off, p.idesc_s, k > 0);
                    }
                    mma_commit(&s.s_full[i]);
                };
                auto value = [&](int i, int st, int half, bool more) {  // O_i += P_i V over 64 keys
                    const uint64_t b0 = sdesc_mn_sw128(kv_addr + st * kBytes);
#pragma unroll
                    for (int k = half * 4; k < half * 4 + 4; k++)
                        mma_f16_ta(tmem + 256 + i * 128, tmem + i * 128 + k * 8, b0 + (uint64_t)((k * 2048) >> 4),
                                   p.idesc_o, more || k > 0);
                };
                bool ok = mbar_wait(&s.q_full, 0, abort_flag, kPolls) && landed(0);
                if (ok) {
                    tc_fence_after();
                    for (int i = 0; i < 2; i++)
                        if (it.n[i] > 0) score(i, 0);
                    mma_commit(&s.empty[0]);
                }
                int st = 1;                             // stage of V_j; K_{j+1} is in the one after it
                for (int j = 0; j < n_max && ok; j++) {
                    const int sv = st;
                    if (j < first_masked) {
                        ok = landed(sv);
                    } else {
                        ok = mbar_wait(&s.clean[sv], clean_ph >> sv & 1u, abort_flag, kPolls);
                        clean_ph ^= 1u << sv;
                    }
                    if (!ok) break;
                    if (++st == kStages) st = 0;
                    const int sk = st;
                    if (j + 1 < n_max) {
                        if (!(ok = landed(sk))) break;
                        if (++st == kStages) st = 0;
                    }
                    for (int i = 0; i < 2 && ok; i++) {
                        if (j < it.n[i]) {
                            if (!(ok = mbar_wait(&s.p_full[i][0], j & 1, abort_flag, kPolls))) break;
                            tc_fence_after();
                            value(i, sv, 0, j > 0);
                            if (!(ok = mbar_wait(&s.p_full[i][1], j & 1, abort_flag, kPolls))) break;
                            tc_fence_after();
                            value(i, sv, 1, true);
                            if (j + 1 == it.n[i]) mma_commit(&s.o_full[i]);
                        }
                        if (j + 1 < it.n[i]) score(i, sk);
                    }
                    if (!ok) break;
                    mma_commit(&s.empty[sv]);
                    if (j + 1 < n_max) mma_commit(&s.empty[sk]);
                }
                mma_commit(&s.drain);
                mbar_drain(&s.drain, 0);
            }
            __syncwarp();
        } else {
            // ------------------------------- values that not every row sees --
            const int t = (warp - 2) * 32 + lane;
            uint32_t raw_ph = 0;                        // parity of each stage's raw barrier
            for (int j = first_masked; j < n_max; j++) {
                const int st = (2 * j + 1) % kStages;
                const bool ok = mbar_wait(&s.raw[st], raw_ph >> st & 1u, abort_flag, kPolls);
                raw_ph ^= 1u << st;
                if (!__all_sync(0xffffffffu, ok)) break;
                uint8_t* v = skv + (size_t)st * kBytes;
                const int live = min(kTile, it.end - j * kTile);
                for (int e = t; e < kTile * D / 8; e += 64) {       // 16 bytes: 8 values of a key
                    const int r = (e >> 3) & (kTile - 1), h = e / (8 * kTile);
                    uint4* at = reinterpret_cast<uint4*>(v + e * 16);
                    if (r >= live) {
                        *at = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    uint4 w = *at;
                    uint32_t u[4] = {w.x, w.y, w.z, w.w};
                    if (not_finite<T>(u[0]) | not_finite<T>(u[1]) | not_finite<T>(u[2]) | not_finite<T>(u[3])) {
                        const int col = h * 64 + (((e & 7) ^ (r & 7)) << 3), key = j * kTile + r;
                        for (int i = 0; i < 8; i++) {
                            const uint32_t bits = (u[i >> 1] >> (16 * (i & 1))) & 0xffffu;
                            if (not_finite<T>(bits) == 0) continue;
                            const float f = Two<T>::one(bits);
                            atomicMin(&s.bad[f != f ? 0 : f > 0.f ? 1 : 2][col + i], key);
                            u[i >> 1] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
                        }
                        *at = make_uint4(u[0], u[1], u[2], u[3]);
                        s.any_bad = 1;
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.clean[st]);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;" ::: "memory");
        // ----------------------------------------------------------- softmax --
        const int i = (warp >> 2) - 1;                  // query tile
        const int r = (warp & 3) * 32 + lane;           // row of it
        const int g = r % p.sh.group, tok = i * p.tokens + r / p.sh.group;
        const bool live = r < p.tokens * p.sh.group && tok < it.ntok;
        const int lim = live ? s.lim[tok] : 0;
        const int n = it.n[i];
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lane_base + i * 128, to = lane_base + 256 + i * 128;
        float ref = 0.f, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n; j++) {
            ok = mbar_wait(&s.s_full[i], j & 1, abort_flag, kPolls);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            float x[kTile];
#pragma unroll
            for (int q = 0; q < kTile; q += 32) tmem_ld32_async(ts + q, reinterpret_cast<uint32_t*>(x) + q);
            tmem_wait_ld();
            if (j >= first_masked) {
                const int see = lim - j * kTile;
#pragma unroll
                for (int q = 0; q < kTile; q++) x[q] = q < see ? x[q] : -INFINITY;
            }
            float m0 = max3(x[0], x[1], x[2]), m1 = max3(x[3], x[4], x[5]), m2 = max3(x[6], x[7], x[8]),
                  m3 = max3(x[9], x[10], x[11]);
#pragma unroll
            for (int q = 12; q < 124; q += 8) {
                m0 = max3(m0, x[q], x[q + 1]);
                m1 = max3(m1, x[q + 2], x[q + 3]);
                m2 = max3(m2, x[q + 4], x[q + 5]);
                m3 = max3(m3, x[q + 6], x[q + 7]);
            }
            m0 = max3(m0, x[124], x[125]);
            m1 = max3(m1, x[126], x[127]);
            const float m = max3(fmaxf(m0, m1), m2, m3);
            if (j == 0) {
                ref = m == -INFINITY ? 0.f : m;
            } else if (__any_sync(0xffffffffu, (m - ref) * p.c > 8.f)) {
                // the accumulator rests: its last product ran before these scores
                const float to_ref = fmaxf(ref, m), f = exp2_fast((ref - to_ref) * p.c);
                l *= f;
                ref = to_ref;
#pragma unroll
                for (int q = 0; q < D; q += 32) {
                    uint32_t a[32];
                    tmem_ld32_async(to + q, a);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e++) a[e] = __float_as_uint(__uint_as_float(a[e]) * f);
                    tmem_st32(to + q, a);
                }
            }
            const float2 c2 = make_float2(p.c, p.c), base = make_float2(-ref * p.c, -ref * p.c);
            float2 l0 = make_float2(0.f, 0.f), l1 = l0;
#pragma unroll
            for (int q = 0; q < kTile; q += 64) {
                uint32_t w[32];
#pragma unroll
                for (int e = 0; e < 64; e += 4) {
                    float2 a = fma2(make_float2(x[q + e], x[q + e + 1]), c2, base);
                    float2 b = fma2(make_float2(x[q + e + 2], x[q + e + 3]), c2, base);
                    a = make_float2(exp2_fast(a.x), exp2_fast(a.y));
                    b = make_float2(exp2_fast(b.x), exp2_fast(b.y));
                    l0 = add2(l0, a);
                    l1 = add2(l1, b);
                    w[e / 2] = Two<T>::pack(a.x, a.y);
                    w[e / 2 + 1] = Two<T>::pack(b.x, b.y);
                }
                // half of the keys: their products start while the other half is worked on
                tmem_st32(ts + q / 2, w);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_full[i][q / 64]);
            }
            l0 = add2(l0, l1);
            l += l0.x + l0.y;
        }
        if (ok && n > 0) {
            ok = mbar_wait(&s.o_full[i], 0, abort_flag, kPolls);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        }
        if (ok) {
            const float inv = lim > 0 ? 1.f / l : 0.f;
            const int h = hk * p.sh.group + g;
            const long long row = it.q0 + tok;
            const bool fix = s.any_bad != 0 && lim > 0;
            const float lse = lim > 0 ? ref * p.sh.scale + logf(l) : -INFINITY;
            if (live) {
                if (p.part)
                    p.part_lse[((long long)blockIdx.z * p.rows + row) * p.sh.hq + h] = lse;
                else if (p.lse)
                    p.lse[row * p.sh.hq + h] = lse;
            }
#pragma unroll
            for (int q = 0; q < D; q += 32) {
                uint32_t a[32] = {};
                if (n > 0) {                            // the same for the warp
                    tmem_ld32_async(to + q, a);
                    tmem_wait_ld();
                }
                float f[32];
#pragma unroll
                for (int e = 0; e < 32; e++) f[e] = lim > 0 ? __uint_as_float(a[e]) * inv : 0.f;
                if (fix) {
                    for (int e = 0; e < 32; e++) {
                        const bool nan = s.bad[0][q + e] < lim, up = s.bad[1][q + e] < lim, down = s.bad[2][q + e] < lim;
                        if (nan || (up && down)) f[e] = NAN;
                        else if (up || down) f[e] += up ? INFINITY : -INFINITY;
                    }
                }
                if (!live) continue;
                if (p.part) {
                    float4* dst = reinterpret_cast<float4*>(
                        p.part + (((long long)blockIdx.z * p.rows + row) * p.sh.hq + h) * D + q);
#pragma unroll
                    for (int e = 0; e < 8; e++) dst[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.o) + row * p.os + (long long)h * D + q);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        dst[e] = make_uint4(Two<T>::pack(f[8 * e], f[8 * e + 1]), Two<T>::pack(f[8 * e + 2], f[8 * e + 3]),
                                            Two<T>::pack(f[8 * e + 4], f[8 * e + 5]),
                                            Two<T>::pack(f[8 * e + 6], f[8 * e + 7]));
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (tid == 0 && s.abort) atomicOr(p.sh.err, CODEC_LM_ERR_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem));
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

}  // namespace

// [rows][heads][D] with rows `stride` elements apart; boxes of 64 elements x
// box_heads x box_rows, 128-byte swizzle; out-of-range rows read as zero.
bool lm_make_map(CUtensorMap* map, int type, const void* base, int D, int heads, long long rows, long long stride,
              int box_heads, int box_rows)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(map, type == CODEC_LM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// Instruction descriptor: fp32 accumulator, both operands of the given format,
// M = 128; N columns; B MN-major or K-major.
uint32_t idesc(uint32_t format, int N, bool b_mn)
{
    return (1u << 4) | (format << 7) | (format << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(kTile >> 4) << 24);
}

template <typename T, int D>
cudaError_t launch(const LmShape& sh, const void* q, long long qs, const LmKeys& ks, Params& p, dim3 grid,
                   cudaStream_t s)
{
    p.sh = sh;
    p.tokens = kTile / sh.group;
    p.tables = ks.tables;
    p.kv_len = ks.kv_len;
    p.table_blocks = ks.table_blocks;
    p.bs_shift = ks.bs_shift;
    p.n_blocks = ks.n_blocks;
    p.c = (float)(sh.scale * 1.4426950408889634);
    p.idesc_s = idesc(Two<T>::kFormat, kTile, false);
    p.idesc_o = idesc(Two<T>::kFormat, D, true);
    const bool paged = ks.tables != nullptr;
    const long long key_rows = paged ? (long long)ks.n_blocks << ks.bs_shift : p.rows;
    const long long k_stride = paged ? (long long)sh.hk * D : ks.k_stride;
    const long long v_stride = paged ? (long long)sh.hk * D : ks.v_stride;
    const int box = paged ? 1 << ks.bs_shift : kTile;
    CUtensorMap mq, mk, mv;
    if (!lm_make_map(&mq, sh.type, q, D, sh.hq, p.rows, qs, sh.group, p.tokens) ||
        !lm_make_map(&mk, sh.type, ks.k, D, sh.hk, key_rows, k_stride, 1, box) ||
        !lm_make_map(&mv, sh.type, ks.v, D, sh.hk, key_rows, v_stride, 1, box))
        return cudaErrorInvalidValue;
    return launch_pdl(lm_prompt_kernel<T, D>, grid, dim3(kThreads), smem_bytes<D>(), s, mq, mk, mv, p);
}

cudaError_t launch_any(const LmShape& sh, const void* q, long long qs, const LmKeys& ks, Params& p, dim3 grid,
                       cudaStream_t s)
{
    if (sh.type == CODEC_LM_BF16)
        return sh.D == 128 ? launch<__nv_bfloat16, 128>(sh, q, qs, ks, p, grid, s)
                           : launch<__nv_bfloat16, 64>(sh, q, qs, ks, p, grid, s);
    return sh.D == 128 ? launch<__half, 128>(sh, q, qs, ks, p, grid, s) : launch<__half, 64>(sh, q, qs, ks, p, grid, s);
}

}  // namespace

cudaError_t configure_lm_prompt()
{
    const std::pair<const void*, size_t> kernels[] = {{(const void*)lm_prompt_kernel<__nv_bfloat16, 128>, smem_bytes<128>()},
                                                      {(const void*)lm_prompt_kernel<__nv_bfloat16, 64>, smem_bytes<64>()},
                                                      {(const void*)lm_prompt_kernel<__half, 128>, smem_bytes<128>()},
                                                      {(const void*)lm_prompt_kernel<__half, 64>, smem_bytes<64>()}};
    for (const auto& k : kernels) {
        const cudaError_t e = cudaFuncSetAttribute(k.first, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.second);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_lm_prompt(const LmShape& sh, const LmPromptArgs& a, cudaStream_t s)
{
    Params p{};
    p.rows = a.rows;
    p.row_start = a.row_start;
    p.B = a.B;
    p.o = a.o;
    p.os = a.os;
    p.lse = a.lse;
    // pairs of query tiles: at most one partly filled pair per request
    const int pair = 2 * (kTile / sh.group);
    const long long items = a.rows / pair + std::min(a.rows, a.B);
    return launch_any(sh, a.q, a.qs, a.keys, p, dim3((unsigned)items, (unsigned)sh.hk), s);
}

cudaError_t launch_lm_shared(const LmShape& sh, const LmSharedArgs& a, cudaStream_t s)
{
    Params p{};
    p.rows = a.B;
    p.shared_len = a.shared_len;
    p.split_len = a.split_len;
    p.part = a.part;
    p.part_lse = a.part_lse;
    LmKeys ks = a.keys;
    ks.tables = a.shared_table;
    const int pair = 2 * (kTile / sh.group);
    const dim3 grid((a.B + pair - 1) / pair, sh.hk, (a.shared_len + a.split_len - 1) / a.split_len);
    return launch_any(sh, a.q, a.qs, ks, p, grid, s);
}

}  // namespace codec
