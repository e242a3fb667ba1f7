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
// Work: an item is a pair of query tiles of one request and K/V head.  Few
// items: one CTA each.  More than there are SMs: one CTA per SM walks a list
// of them, longest first, that a small kernel makes from the lengths; copies
// and MMAs of the next item then run while the last one is written.  Where the
// longest items would keep a few SMs busy long after the others, they are cut
// along the keys: the pieces leave partial results in fp32, which a third
// kernel joins in order.
//
// Roles (384 threads, one CTA per SM):
//   warp 0      takes the items from a counter; copies: Q, then K and V tiles through a ring of stages; paged
//               keys one box per cache block, one block per lane
//   warp 1      TMEM and MMA issue: the MMAs of one tile run while the
//               softmax of the other does
//   warps 2, 3  V tiles that hold keys some row may not see: rows nobody sees
//               are zeroed, and so is what is not finite (0 x NaN is NaN, so a
//               probability of zero would not keep it out); the rows that do
//               see it get it back at the end
//   warps 4-11  softmax, four warps per tile; they also rescale the
//               accumulator and write the result
// Every wait is bounded: when one expires the CTA raises the error bit, stops,
// drains its copies and MMAs, frees TMEM and returns.
//
// What bounds it.  Long prompts: a pair of tiles takes about 2,800 cycles per 128
// keys where its MMAs need 2,048; 6,904 and 9,000 tokens of 32 / 8 heads of 128 in
// bf16 take 711 us, 1,480 TFLOP/s (79 % of a large library GEMM), the tensor pipe
// 70 % active.  A warp's softmax of a tile is 1,100 cycles, and a tile's scores
// cannot be made before its last probabilities have been used, as these lie over
// them: two tiles in turn hide most of that.  Ragged and short ones: an item costs
// 8,000 cycles besides its tiles - the last product with V 2,400, the result 4,900
// while the other tile's warps share the SM.  Behind a cached context one tile's
// 64 KB of K and V per 128 keys and SM add up to 4 TB/s, and blocks of 16 positions
// to 32 copies per tile.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "lm.h"
#include "lm_join.cuh"
#include "tc_ptx.cuh"

namespace codec {

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;                  // rows of a query tile, keys of a K/V tile
constexpr uint32_t kHalfBytes = kTile * 128;    // 64 columns of a tile: 128 rows of 128 bytes
constexpr int kMaxStages = 8;
constexpr int kNone = 0x7fffffff;
constexpr int kSms = 152;

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
    const void* v;              // values, for what is not finite
    long long v_stride;
    const int4* list;           // items, two each (see Entry); null: by blockIdx
    int* counts;                // items of the list, items taken from it, items to join
    int4* joins;                // of each: first query row, tokens, first slot and pieces << 16, keys of the first token
    int split;                  // items may be cut along the keys
    int most_cut;               // so many of them at most (with their K/V heads)
    float* piece;               // pieces' results: [slot][2 x 128 rows][D], normalised, fp32
    float* piece_lse;
    float c;                    // scale x log2 e
    uint32_t idesc_s, idesc_o;
    void* o;
    long long os;
    float* lse;
    float* part;                // shared part: [split][rows][hq][D], normalised, fp32
    float* part_lse;            // [split][rows][hq]
    const float* row_c;         // shared part: c of each (row, head) instead (kRowScale)
};

// An item as the list holds it.
struct Entry {
    int4 rows;                  // request, first query row, tokens, keys of the first token
    int4 keys;                  // first K/V tile, tiles, first slot of the piece (of K/V head 0; -1: whole)
};

// A pair of query tiles, or a piece of one along the keys.
struct Item {
    int b, hk;                  // request, K/V head
    int q0;                     // first query row
    int ntok;                   // tokens of the two tiles that exist
    int first;                  // prompts: keys of the first token, each later one sees one more (may be < 1)
    int key0;                   // packed: row of key 0; else key 0's position
    int cap;                    // keys of the piece at most
    int slot;                   // where a piece's result goes; -1: the item is whole
    int end;                    // keys at or behind it: seen by no row
    int free_from;              // keys below it: seen by every row that sees any
    int n[2];                   // K/V tiles of each query tile
};

// Operand descriptors, low words (address and leading byte offset; the high
// word is the same for all: 8-row groups 1024 bytes apart, descriptor version,
// 128-byte swizzle).  K-major: as sdesc_sw128.  MN-major: 64 elements of N in a
// 128-byte row per k, the next 64 one half tile further (leading byte offset).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr) { return (saddr >> 4) | ((kHalfBytes >> 4) << 16); }

// D[tmem] (+)= A[shared] x B[shared]
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
        : "memory");
}

// D[tmem] (+)= A[tmem] x B[shared]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
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

// Eight columns of this warp's lanes times f (few registers: the scores are live around it).
__device__ __forceinline__ void tmem_scale8(uint32_t taddr, float f)
{
    float a[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int e = 0; e < 8; e++) a[e] *= f;
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(a[0]), "f"(a[1]),
                 "f"(a[2]), "f"(a[3]), "f"(a[4]), "f"(a[5]), "f"(a[6]), "f"(a[7]), "r"(taddr)
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
};
template <> struct Two<__half> {
    static constexpr uint32_t kFormat = 0;
    static constexpr uint32_t kExp = 0x7c007c00u, kOne = 0x04000400u;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};

// Which of a word's two values is not finite, as bits 15 and 31.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    return ((w & Two<T>::kExp) + Two<T>::kOne) & 0x80008000u;
}

template <int D> constexpr int stages() { return D == 128 ? 4 : 7; }
constexpr int kWork = 4;                // items handed out ahead
constexpr uint32_t kStageOut = 4096;    // per softmax warp: 32 rows of 128 bytes on their way out

struct Shared {
    uint64_t drain;
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t raw[kMaxStages], clean[kMaxStages];    // V tiles that are cleaned before use: landed, cleaned
    uint64_t never;             // nothing arrives (see LmShape::unarrived)
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], o_empty[2];
    uint64_t work_full[kWork], work_empty[kWork];
    Item work[kWork];           // hk -1: no more
    uint32_t tmem;
    int abort;
    int scan[kThreads / 32];
    int found;
    Item item;                  // without a list
    int written[2];             // softmax warps of each query tile that are done with an item, summed
    int dirty[2];               // 1 + the last even / odd item with a value that is not finite in a cleaned tile
};

template <int D> constexpr uint32_t tile_bytes() { return kTile * D * 2; }
template <int D> constexpr size_t smem_bytes()
{
    return (size_t)(2 + stages<D>()) * tile_bytes<D>() + 8 * kStageOut + sizeof(Shared);
}
static_assert(smem_bytes<128>() <= 227 * 1024 && smem_bytes<64>() <= 227 * 1024, "shared memory");

// Finds the CTA's request and query rows: item x of the requests' tile pairs,
// in request order, each request's last (longest) pair first.  All threads.
__device__ void find_item(const Params& p, Shared& s)
{
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int pair = 2 * p.tokens;
    const bool report = blockIdx.x == 0 && blockIdx.y == 0;
    int before = 0;
    for (int base = 0; base < p.B; base += kThreads) {
        const int b = base + tid;
        int first = 0, n = 0, tiles = 0;
        if (b < p.B) {
            bool good = lm_rows(p.row_start, b, p.rows, first, n);
            if (report && p.tables) {
                int keys = __ldg(p.kv_len + b);
                good &= lm_clamp_len(keys, (long long)p.table_blocks << p.bs_shift);
            }
            if (report && !good) atomicOr(p.sh.err, CODEC_LM_ERR_LENGTH);
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
            int keys = n;
            if (p.tables) {
                keys = __ldg(p.kv_len + b);
                lm_clamp_len(keys, (long long)p.table_blocks << p.bs_shift);
            }
            s.item.first = keys - n + t * pair + 1;
            s.found = 1;
        }
        before += total;
        __syncthreads();
        if (s.found && !report) break;
    }
}

// Keys that token t of an item sees, from key0 on.
__device__ __forceinline__ int keys_of(const Params& p, const Item& it, int t)
{
    if (p.row_start) return min(it.cap, max(0, it.first + t));
    int n = __ldg(p.kv_len + it.q0 + t);
    lm_clamp_len(n, (long long)p.table_blocks << p.bs_shift);
    return min(max(min(n, p.shared_len) - it.key0, 0), p.split_len);
}

// What follows from a prompt item's rows and its first token's keys.
__device__ __forceinline__ void derive(const Params& p, Item& it, int4 keys)
{
    const int skip = keys.x * kTile;
    it.key0 = (p.tables ? 0 : it.q0 - (it.first - 1)) + skip;
    it.first -= skip;
    it.cap = keys.y < kNone / kTile ? keys.y * kTile : kNone;
    it.slot = keys.z < 0 ? -1 : keys.z + it.hk;
    const int most0 = min(it.cap, max(0, it.first + min(it.ntok, p.tokens) - 1));
    const int most1 = it.ntok > p.tokens ? min(it.cap, max(0, it.first + it.ntok - 1)) : 0;
    it.end = max(most0, most1);
    it.free_from = it.end > 0 ? min(it.cap, max(1, it.first)) : kNone;
    it.n[0] = (most0 + kTile - 1) / kTile;
    it.n[1] = (most1 + kTile - 1) / kTile;
}

// The CTA's items, one after the other.  The copy warp takes them from a
// counter and hands them on in shared memory (few registers: each role reads
// what it needs); each other role waits for them by itself.
struct Walk {
    int k = 0;                  // items so far

    // The copy warp hands out (e, hk); null: that was the end.
    __device__ __forceinline__ const Item* hand_out(const Params& p, Shared& s, const Entry& e, int hk, int lane)
    {
        if (!p.list) return k++ || !s.found ? nullptr : &s.item;
        const int slot = k % kWork;
        const bool ok = mbar_wait(&s.work_empty[slot], (uint32_t)(k / kWork & 1) ^ 1u, &s.abort, kLmPolls);
        k++;
        if (!__all_sync(0xffffffffu, ok)) return nullptr;
        Item& it = s.work[slot];
        if (lane == 0) {
            it.hk = hk;
            it.b = e.rows.x;
            it.q0 = e.rows.y;
            it.ntok = e.rows.z;
            it.first = e.rows.w;
            derive(p, it, e.keys);
            mbar_arrive(&s.work_full[slot]);
        }
        __syncwarp();
        return hk < 0 ? nullptr : &it;
    }
    // Every other role.
    __device__ __forceinline__ const Item* next(const Params& p, Shared& s)
    {
        if (!p.list) return k++ || !s.found ? nullptr : &s.item;
        const int slot = k % kWork;
        const bool ok = mbar_wait(&s.work_full[slot], (uint32_t)(k / kWork & 1), &s.abort, kLmPolls);
        k++;
        return !ok || s.work[slot].hk < 0 ? nullptr : &s.work[slot];
    }
    // and when it needs the item no longer: one thread of each waiting warp.
    __device__ __forceinline__ void done(const Params& p, Shared& s)
    {
        if (p.list) mbar_arrive(&s.work_empty[(k - 1) % kWork]);
    }
};

// Adds to a warp's rows (dst: this lane's, T or fp32; lim: the keys it sees) the values
// that are not finite of its keys lo .. lim - 1 of an item.  Rare, and read from
// global memory: once for the warp, D / 32 columns per lane, each row taking the
// sum where its last key is in.  One infinity a head among 8,192 shared positions,
// 64 requests: 0.3 ms on top (48 with a column at a time, every row reading its keys anew).
template <typename T, int D>
__device__ __noinline__ void add_not_finite(const Params& p, const Item& it, int lo, int lim, unsigned long long dst,
                                            bool fp32)
{
    constexpr int kE = D / 32;
    const int col = (threadIdx.x & 31) * kE;
    const T* v = static_cast<const T*>(p.v) + (long long)it.hk * D + col;
    const int* table = p.tables ? p.tables + (p.row_start ? (long long)it.b * p.table_blocks : 0LL) : nullptr;
    float sum[kE] = {};
    for (int k = lo;;) {
        const int next = __reduce_min_sync(0xffffffffu, lim > k ? lim : kNone);
        if (next == kNone) break;
#pragma unroll 8
        for (int x = k; x < next; x++) {
            long long row = it.key0 + x;
            bool in = true;
            if (table) {
                const int id = __ldg(table + (row >> p.bs_shift));
                in = id >= 0 && id < p.n_blocks;
                row = ((long long)id << p.bs_shift) + (row & ((1 << p.bs_shift) - 1));
            }
            alignas(8) T y[kE] = {};
            if constexpr (kE == 4) {
                if (in) *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(v + row * p.v_stride);
            } else {
                if (in) *reinterpret_cast<uint32_t*>(y) = *reinterpret_cast<const uint32_t*>(v + row * p.v_stride);
            }
#pragma unroll
            for (int e = 0; e < kE; e++) sum[e] += isfinite((float)y[e]) ? 0.f : (float)y[e];
        }
        k = next;
        unsigned rows = __ballot_sync(0xffffffffu, lim == next);
        while (rows) {
            const unsigned long long to = __shfl_sync(0xffffffffu, dst, __ffs(rows) - 1);
            rows &= rows - 1;
#pragma unroll
            for (int e = 0; e < kE; e++) {
                if (sum[e] == 0.f) continue;
                if (fp32)
                    reinterpret_cast<float*>(to)[col + e] += sum[e];
                else
                    reinterpret_cast<T*>(to)[col + e] = (T)((float)reinterpret_cast<T*>(to)[col + e] + sum[e]);
            }
        }
    }
}

// kRowScale: queries are times a power of two of their own, which row_c undoes (an
// instance of its own: a register more).
template <typename T, int D, bool kRowScale = false>
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
    uint8_t* sout = skv + (size_t)kStages * kBytes;     // rows on their way out
    Shared& s = *reinterpret_cast<Shared*>(sout + 8 * kStageOut);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(&s.drain, 1);
        mbar_init(&s.never, 1);
        for (int i = 0; i < kStages; i++) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
            mbar_init(&s.raw[i], 1);
            mbar_init(&s.clean[i], 2);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i][0], 4);
            mbar_init(&s.p_full[i][1], 4);
            mbar_init(&s.o_full[i], 1);
            mbar_init(&s.o_empty[i], 4);
            s.dirty[i] = 0;
        }
        for (int i = 0; i < kWork; i++) {
            mbar_init(&s.work_full[i], 1);
            mbar_init(&s.work_empty[i], 11);            // MMA thread, 2 cleaning and 8 softmax warps
        }
        s.abort = 0;
        s.found = 0;
        s.written[0] = s.written[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tensormap(&mq);
        prefetch_tensormap(&mk);
        prefetch_tensormap(&mv);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    // the set-up above touches no global memory that an earlier kernel writes
    pdl_wait();
    pdl_launch();

    if (!p.list) {
        if (p.row_start) {
            find_item(p, s);
            if (tid == 0 && s.found) {
                s.item.hk = blockIdx.y;
                derive(p, s.item, make_int4(0, kNone, -1, 0));
            }
        } else if (warp == 0) {
            // a shared part: the largest and the smallest number of keys but none
            Item it;
            it.b = 0;
            it.hk = blockIdx.y;
            it.q0 = blockIdx.x * 2 * p.tokens;
            it.ntok = min(2 * p.tokens, p.rows - it.q0);
            it.key0 = blockIdx.z * p.split_len;
            it.first = 0;
            it.cap = kNone;
            it.slot = -1;
            int most[2] = {0, 0}, least = kNone;
            for (int t = lane; t < it.ntok; t += 32) {
                const int n = keys_of(p, it, t);
                if (t < p.tokens) most[0] = max(most[0], n); else most[1] = max(most[1], n);
                if (n > 0) least = min(least, n);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                most[0] = max(most[0], __shfl_xor_sync(0xffffffffu, most[0], o));
                most[1] = max(most[1], __shfl_xor_sync(0xffffffffu, most[1], o));
                least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
            }
            it.end = max(most[0], most[1]);
            it.free_from = least;
            it.n[0] = (most[0] + kTile - 1) / kTile;
            it.n[1] = (most[1] + kTile - 1) / kTile;
            if (lane == 0) {
                s.item = it;
                s.found = 1;
            }
        }
        __syncthreads();
    }
    volatile int* abort_flag = &s.abort;
    Walk walk;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
        if (warp == 0) {
            // ------------------------------------------------------ copies --
            int st = 0;
            uint32_t ph = 0, q_n = 0;                   // stage and its round; uses of the query tiles (parity)
            uint32_t full_n = 0, raw_n = 0, full_any = 0, raw_any = 0, q_any = 0;  // uses of the barriers: parity, any
            const int per = kTile >> p.bs_shift;        // cache blocks per tile
            const int g = p.sh.group;
            bool ok = true;
            Entry entry{};
            int entry_hk = -1;
            int count = 0, taken = 0;                   // taken: lane 0's, from the counter
            auto fetch = [&](int w) {                   // the list has room for a grid of items
                entry_hk = w % p.sh.hk;
                entry.rows = __ldg(p.list + 2 * (w / p.sh.hk));
                entry.keys = __ldg(p.list + 2 * (w / p.sh.hk) + 1);
            };
            if (p.list) {
                count = __ldcg(p.counts) * p.sh.hk;
                fetch(blockIdx.x);
                if ((int)blockIdx.x >= count) entry_hk = -1;
            }
            while (ok) {
                const Item* const item = walk.hand_out(p, s, entry, entry_hk, lane);
                if (!item) break;
                const Item& it = *item;
                const int n_max = max(it.n[0], it.n[1]);
                const int first_masked = it.free_from / kTile;
                const int* table = nullptr;
                int blocks = 0, next = 0;
                if (p.tables) {
                    table = p.tables + (p.row_start ? (long long)it.b * p.table_blocks : 0LL) + (it.key0 >> p.bs_shift);
                    blocks = (it.end + (1 << p.bs_shift) - 1) >> p.bs_shift;
                    if (lane < min(per, blocks)) next = __ldg(table + lane);
                }
                for (int i = 0; i < 2 && ok; i++) {
                    if (it.n[i] == 0) continue;
                    ok = mbar_wait(&s.q_empty[i], (q_n >> i & 1u) ^ 1u, abort_flag, kLmPolls);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    q_n ^= 1u << i;
                    q_any |= 1u << i;
                    if (elect_one()) {
                        mbar_expect_tx(&s.q_full[i], (uint32_t)(p.tokens * g * D * 2));
                        for (int h = 0; h < kHalves; h++)
                            tma_load_3d(sq + i * kBytes + h * kHalfBytes, &mq, &s.q_full[i], h * 64, it.hk * g,
                                        it.q0 + i * p.tokens);
                    }
                    __syncwarp();
                }
                for (int j = 0; j < n_max && ok; j++) {
                    int id = next;
                    const int here = p.tables ? min(per, blocks - j * per) : 1;
                    if (p.tables) {
                        const int at = (j + 1) * per + lane;
                        if (lane < per && at < blocks) next = __ldg(table + at);
                        if (lane < here && (id < 0 || id >= p.n_blocks)) {
                            atomicOr(p.sh.err, CODEC_LM_ERR_BLOCK);
                            id = p.n_blocks;            // behind the last row: the copy writes zeros
                        }
                    }
                    for (int kv = 0; kv < 2; kv++) {
                        ok = mbar_wait(&s.empty[st], ph ^ 1u, abort_flag, kLmPolls);
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
                        if (p.tables) {
                            if (lane == 0) mbar_expect_tx(bar, (uint32_t)(here << p.bs_shift) * D * 2);
                            __syncwarp();
                            if (lane < here)
                                for (int h = 0; h < kHalves; h++)
                                    tma_load_3d(dst + h * kHalfBytes + ((uint32_t)lane << p.bs_shift) * 128, map, bar,
                                                h * 64, it.hk, id << p.bs_shift);
                        } else if (elect_one()) {
                            mbar_expect_tx(bar, kBytes);
                            for (int h = 0; h < kHalves; h++)
                                tma_load_3d(dst + h * kHalfBytes, map, bar, h * 64, it.hk, it.key0 + j * kTile);
                        }
                        __syncwarp();
                        if (++st == kStages) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
                }
                // The next item, two tiles ahead of its use.  No sooner: a CTA in the midst of
                // a long item would hold one that others could have begun.
                if (p.list) {
                    if (lane == 0) taken = atomicAdd(p.counts + 1, 1) + gridDim.x;
                    taken = __shfl_sync(0xffffffffu, taken, 0);
                    entry_hk = -1;
                    if (taken < count) fetch(taken);
                }
            }
            // every last load has landed before the CTA can end
            for (int q = 0; q < kStages; q++) {
                if (full_any >> q & 1u) mbar_drain(&s.full[q], (full_n >> q & 1u) ^ 1u);
                if (raw_any >> q & 1u) mbar_drain(&s.raw[q], (raw_n >> q & 1u) ^ 1u);
            }
            for (int i = 0; i < 2; i++)
                if (q_any >> i & 1u) mbar_drain(&s.q_full[i], (q_n >> i & 1u) ^ 1u);
        } else if (warp == 1) {
            // -------------------------------------------------------- MMAs --
            if (elect_one()) {
                const uint32_t q_addr = smem_u32(sq), kv_addr = smem_u32(skv);
                uint32_t full_ph = 0, clean_ph = 0;     // parity of each stage's barriers
                uint32_t tile_ph = 0, item_ph = 0;      // of each query tile's: per K/V tile, per item
                int st = 0;
                auto landed = [&](int stage) {
                    const bool in = mbar_wait(&s.full[stage], full_ph >> stage & 1u, abort_flag, kLmPolls);
                    full_ph ^= 1u << stage;
                    tc_fence_after();
                    return in;
                };
                auto score = [&](int i, int stage, bool last) {         // S_i = Q_i K^T
                    const uint32_t a0 = desc_k(q_addr + i * kBytes), b0 = desc_k(kv_addr + stage * kBytes);
#pragma unroll
                    for (int k = 0; k < D / 16; k++) {
                        const uint32_t off = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
                        mma_ss(tmem + i * 128, a0 + off, b0 + off, p.idesc_s, k > 0);
                    }
                    mma_commit(&s.s_full[i]);
                    if (last) mma_commit(&s.q_empty[i]);
                };
                auto value = [&](int i, int stage, int half, bool more) {   // O_i += P_i V over 64 keys
                    const uint32_t b0 = desc_mn(kv_addr + stage * kBytes);
#pragma unroll
                    for (int k = half * 4; k < half * 4 + 4; k++)
                        mma_ts(tmem + 256 + i * 128, tmem + i * 128 + k * 8, b0 + ((k * 2048) >> 4), p.idesc_o,
                               more || k > 0);
                };
                bool ok = true;
                while (ok) {
                    const Item* const item = walk.next(p, s);
                    if (!item) break;
                    const int n0 = item->n[0], n1 = item->n[1], first_masked = item->free_from / kTile;
                    walk.done(p, s);
                    const int n_max = max(n0, n1);
                    if (n_max == 0) continue;
                    const int sk0 = st;
                    if (++st == kStages) st = 0;
                    if (!(ok = landed(sk0))) break;
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        if ((i ? n1 : n0) == 0 || !ok) continue;
                        ok = mbar_wait(&s.q_full[i], item_ph >> i & 1u, abort_flag, kLmPolls);
                        tc_fence_after();
                        if (ok) score(i, sk0, (i ? n1 : n0) == 1);
                    }
                    if (!ok) break;
                    mma_commit(&s.empty[sk0]);
                    for (int j = 0; j < n_max && ok; j++) {
                        const int sv = st;
                        if (++st == kStages) st = 0;
                        if (j < first_masked) {
                            ok = landed(sv);
                        } else {
                            ok = mbar_wait(&s.clean[sv], clean_ph >> sv & 1u, abort_flag, kLmPolls);
                            clean_ph ^= 1u << sv;
                            tc_fence_after();
                        }
                        if (!ok) break;
                        const int sk = st;              // K_{j+1}
                        const bool more = j + 1 < n_max;
                        if (more && ++st == kStages) st = 0;
                        bool here = false;              // K_{j+1} has landed
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            if (!ok) break;
                            if (j < (i ? n1 : n0)) {
                                const uint32_t ph = tile_ph >> i & 1u;
                                ok = mbar_wait(&s.p_full[i][0], ph, abort_flag, kLmPolls);
                                // the last item's result has been read
                                if (ok && j == 0)
                                    ok = mbar_wait(&s.o_empty[i], (item_ph >> i & 1u) ^ 1u, abort_flag, kLmPolls);
                                if (!ok) break;
                                tc_fence_after();
                                value(i, sv, 0, j > 0);
                                if (!(ok = mbar_wait(&s.p_full[i][1], ph, abort_flag, kLmPolls))) break;
                                tc_fence_after();
                                value(i, sv, 1, true);
                                tile_ph ^= 1u << i;
                                if (j + 1 == (i ? n1 : n0)) mma_commit(&s.o_full[i]);
                            }
                            if (j + 1 < (i ? n1 : n0)) {
                                if (!here) {
                                    if (!(ok = landed(sk))) break;
                                    here = true;
                                }
                                score(i, sk, j + 2 == (i ? n1 : n0));
                            }
                        }
                        if (!ok) break;
                        mma_commit(&s.empty[sv]);
                        if (more) mma_commit(&s.empty[sk]);
                    }
                    for (int i = 0; i < 2; i++)
                        if ((i ? n1 : n0) > 0) item_ph ^= 1u << i;
                }
                // all issued MMAs complete before TMEM is released
                mma_commit(&s.drain);
                mbar_drain(&s.drain, 0);
            }
            __syncwarp();
        } else {
            // ------------------------------- values that not every row sees --
            const int t = (warp - 2) * 32 + lane;
            uint32_t raw_ph = 0;                        // parity of each stage's raw barrier
            int load0 = 0;                              // stage of the item's first load
            bool ok = true;
            while (ok) {
                const Item* const item = walk.next(p, s);
                if (!__all_sync(0xffffffffu, item != nullptr)) break;
                const int n_max = max(item->n[0], item->n[1]), first_masked = item->free_from / kTile, end = item->end;
                __syncwarp();
                if (lane == 0) walk.done(p, s);
                for (int j = first_masked; j < n_max; j++) {
                    const int st = (load0 + 2 * j + 1) % kStages;
                    ok = mbar_wait(&s.raw[st], raw_ph >> st & 1u, abort_flag, kLmPolls);
                    raw_ph ^= 1u << st;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint8_t* v = skv + (size_t)st * kBytes;
                    const int live = min(kTile, end - j * kTile);
                    for (int e = t; e < kTile * D / 8; e += 64) {       // 16 bytes: 8 values of a key
                        const int r = (e >> 3) & (kTile - 1);
                        uint4* at = reinterpret_cast<uint4*>(v + e * 16);
                        if (r >= live) {
                            *at = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        const uint4 w = *at;
                        const uint32_t b0 = not_finite<T>(w.x), b1 = not_finite<T>(w.y), b2 = not_finite<T>(w.z),
                                       b3 = not_finite<T>(w.w);
                        if (b0 | b1 | b2 | b3) {
                            auto keep = [](uint32_t x, uint32_t bad) {
                                return x & ((bad & 0x8000u ? 0u : 0xffffu) | (bad & 0x80000000u ? 0u : 0xffff0000u));
                            };
                            *at = make_uint4(keep(w.x, b0), keep(w.y, b1), keep(w.z, b2), keep(w.w, b3));
                            // the note of the item before the last one has been read by now, or soon is
                            volatile int* written = s.written;
                            for (uint32_t i = 0; min(written[0], written[1]) < 4 * (walk.k - 2) && !*abort_flag; i++)
                                if (i >= kLmPolls) *abort_flag = 1;
                            *reinterpret_cast<volatile int*>(&s.dirty[walk.k & 1]) = walk.k;
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.clean[st]);
                }
                load0 = (load0 + 2 * n_max) % kStages;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;" ::: "memory");
        // ----------------------------------------------------------- softmax --
        const int i = (warp >> 2) - 1;                  // query tile
        const int r = (warp & 3) * 32 + lane;           // row of it
        const int g = r % p.sh.group, tok = i * p.tokens + r / p.sh.group;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lane_base + i * 128, to = lane_base + 256 + i * 128;
        uint32_t tile_ph = 0, item_ph = 0;
        bool ok = !p.sh.unarrived || warp != 4 || mbar_wait(&s.never, 0, abort_flag, p.sh.unarrived);
        ok = __all_sync(0xffffffffu, ok);
        while (ok) {
            const Item* const item = walk.next(p, s);
            if (!__all_sync(0xffffffffu, item != nullptr)) break;
            const Item& it = *item;
            const bool live = r < p.tokens * p.sh.group && tok < it.ntok;
            const int lim = live ? keys_of(p, it, tok) : 0;
            const int n = it.n[i];
            // tiles from here on hold keys that some row does not see
            const int first_masked = it.free_from / kTile;
            float ref = 0.f, l = 0.f;
            float c = p.c;
            if constexpr (kRowScale)
                if (live) c = __ldcg(p.row_c + ((long long)it.q0 + tok) * p.sh.hq + it.hk * p.sh.group + g);
            for (int j = 0; j < n; j++) {
                ok = mbar_wait(&s.s_full[i], tile_ph, abort_flag, kLmPolls);
                tile_ph ^= 1u;
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
                    // scores of -inf alone so far: below whatever comes
                    ref = m == -INFINITY ? -1e30f : m;
                } else if (__any_sync(0xffffffffu, (m - ref) * c > 8.f)) {
                    // Only the rows that need it move (times 1 changes nothing): a row's bits
                    // do not depend on its neighbours.  The accumulator rests: its last
                    // product ran before these scores.
                    const float to_ref = (m - ref) * c > 8.f ? m : ref, f = exp2_fast((ref - to_ref) * c);
                    l *= f;
                    ref = to_ref;
#pragma unroll 1
                    for (int q = 0; q < D; q += 8) tmem_scale8(to + q, f);
                }
                const float2 c2 = make_float2(c, c), base = make_float2(-ref * c, -ref * c);
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
                ok = mbar_wait(&s.o_full[i], item_ph, abort_flag, kLmPolls);
                item_ph ^= 1u;
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
            }
            if (!ok) break;
            const float inv = lim > 0 ? 1.f / l : 0.f;
            const int h = it.hk * p.sh.group + g;
            const long long row = it.q0 + tok;
            const bool fix = *reinterpret_cast<volatile int*>(&s.dirty[walk.k & 1]) == walk.k && lim > 0;
            if (live) {
                const float lse = lim > 0 ? ref * (kRowScale ? c * 0.6931471805599453f : p.sh.scale) + logf(l) : -INFINITY;
                if (it.slot >= 0)
                    p.piece_lse[((long long)it.slot * 2 + i) * kTile + r] = lse;
                else if (p.part)
                    p.part_lse[((long long)blockIdx.z * p.rows + row) * p.sh.hq + h] = lse;
                else if (p.lse)
                    p.lse[row * p.sh.hq + h] = lse;
            }
            // A row per lane would touch 32 lines with every store; so 32 rows of 128
            // bytes go through shared memory (16-byte chunks swizzled by the row) and
            // leave as four whole rows per store.  Rolled loops: this runs once per
            // item, and unrolled it came from beyond the instruction cache each time.
            uint8_t* out = sout + (size_t)(warp - 4) * kStageOut;
            const unsigned rows = __ballot_sync(0xffffffffu, live);
            const bool fp32 = p.part || it.slot >= 0;
            const unsigned long long mine = reinterpret_cast<unsigned long long>(
                it.slot >= 0 ? static_cast<void*>(p.piece + (((long long)it.slot * 2 + i) * kTile + r) * D)
                : p.part ? static_cast<void*>(p.part + (((long long)blockIdx.z * p.rows + row) * p.sh.hq + h) * D)
                       : static_cast<void*>(static_cast<T*>(p.o) + row * p.os + (long long)h * D));
            auto flush = [&](int byte) {
                __syncwarp();
                uint4 v[8];
                unsigned long long dst[8];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int from = 4 * e + (lane >> 3);
                    v[e] = *reinterpret_cast<const uint4*>(out + from * 128 + (((lane & 7) ^ (from & 7)) << 4));
                    dst[e] = __shfl_sync(0xffffffffu, mine, from) + byte + (lane & 7) * 16;
                }
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (rows >> (4 * e + (lane >> 3)) & 1u) *reinterpret_cast<uint4*>(dst[e]) = v[e];
                __syncwarp();
            };
#pragma unroll 1
            for (int q = 0; q < D; q += 64) {
                uint32_t a[64] = {};
                if (n > 0) {                            // the same for the warp
                    tmem_ld32_async(to + q, a);
                    tmem_ld32_async(to + q + 32, a + 32);
                    tmem_wait_ld();
                    if (q + 64 == D) {                  // the accumulator is free for the next item
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s.o_empty[i]);
                    }
                }
                float f[64];
#pragma unroll
                for (int e = 0; e < 64; e++) f[e] = lim > 0 ? __uint_as_float(a[e]) * inv : 0.f;
                auto put = [&](int chunk, uint4 v) {
                    *reinterpret_cast<uint4*>(out + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = v;
                };
                if (fp32) {
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            put(e, make_uint4(__float_as_uint(f[c + 4 * e]), __float_as_uint(f[c + 4 * e + 1]),
                                              __float_as_uint(f[c + 4 * e + 2]), __float_as_uint(f[c + 4 * e + 3])));
                        flush((q + c) * 4);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        put(e, make_uint4(Two<T>::pack(f[8 * e], f[8 * e + 1]), Two<T>::pack(f[8 * e + 2], f[8 * e + 3]),
                                          Two<T>::pack(f[8 * e + 4], f[8 * e + 5]),
                                          Two<T>::pack(f[8 * e + 6], f[8 * e + 7])));
                    flush(q * 2);
                }
            }
            // added to what the other tiles and the row's statistics gave, which may be an infinity or NaN already
            if (__any_sync(0xffffffffu, fix)) add_not_finite<T, D>(p, it, first_masked * kTile, fix ? lim : 0, mine, fp32);
            __syncwarp();
            if (lane == 0) {
                atomicAdd(&s.written[i], 1);
                walk.done(p, s);
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

// The items of a call, from the device's lengths: requests by their keys,
// most first (in request order where there are many), each request's last pair
// of tiles first.  With p.split, items of more than 5/4 of an SM's share of the
// call's tiles are cut into pieces of about that share (at least kMinPiece
// tiles: an item costs as much as three tiles besides them; with six two requests of
// 64 tokens behind 1,936 positions take 24.0 us, with four 22.6).  One CTA.
constexpr int kListThreads = 512;
constexpr int kListSort = 512;          // requests that are sorted (by counting)
constexpr int kMinPiece = 4;

__global__ void __launch_bounds__(kListThreads) lm_list_kernel(const Params p, int4* list)
{
    __shared__ int keys[kListSort], row0[kListSort], nrow[kListSort];
    __shared__ unsigned short order[kLmMaxRequests];
    __shared__ int start[kLmMaxRequests + 1];
    __shared__ int warp_sum[3][kListThreads / 32];
    __shared__ int carry[3];
    __shared__ unsigned long long work;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int pair = 2 * p.tokens;
    pdl_wait();
    pdl_launch();
    auto rows_and_keys = [&](int b, int& first, int& n, bool report) {
        const bool good = lm_rows(p.row_start, b, p.rows, first, n);
        int k = n;
        bool len = true;
        if (p.tables) {
            k = __ldg(p.kv_len + b);
            len = lm_clamp_len(k, (long long)p.table_blocks << p.bs_shift);
        }
        if (report && !(good && len)) atomicOr(p.sh.err, CODEC_LM_ERR_LENGTH);
        return k;
    };
    // running sums over the block of up to three values, on top of carry (which grows)
    auto scan = [&](int* v, int count) {
        int incl[3];
        for (int c = 0; c < count; c++) {
            incl[c] = v[c];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl[c], o);
                if (lane >= o) incl[c] += up;
            }
            if (lane == 31) warp_sum[c][w] = incl[c];
        }
        __syncthreads();
        int total[3];
        for (int c = 0; c < count; c++) {
            int at = carry[c];
            total[c] = at;
            for (int i = 0; i < kListThreads / 32; i++) {
                if (i < w) at += warp_sum[c][i];
                total[c] += warp_sum[c][i];
            }
            v[c] = at + incl[c] - v[c];         // exclusive
        }
        __syncthreads();
        if (tid == 0)
            for (int c = 0; c < count; c++) carry[c] = total[c];
        __syncthreads();
    };
    const bool sorted = p.B <= kListSort;
    if (tid < 3) carry[tid] = 0;
    if (tid == 0) work = 0;
    for (int b = tid; b < p.B; b += kListThreads) {
        int first, n;
        const int k = rows_and_keys(b, first, n, true);
        if (sorted) {
            keys[b] = n > 0 ? k : -1;
            row0[b] = first;
            nrow[b] = n;
        } else {
            order[b] = (unsigned short)b;
        }
    }
    __syncthreads();
    if (sorted && tid < p.B) {
        int rank = 0;
        for (int c = 0; c < p.B; c++) rank += keys[c] > keys[tid] || (keys[c] == keys[tid] && c < tid);
        order[rank] = (unsigned short)tid;
    }
    __syncthreads();
    for (int base = 0; base < p.B; base += kListThreads) {
        const int x = base + tid;
        int tiles = 0, first, n;
        if (x < p.B) {
            if (sorted) n = nrow[order[x]]; else lm_rows(p.row_start, order[x], p.rows, first, n);
            tiles = (n + pair - 1) / pair;
        }
        scan(&tiles, 1);
        if (x < p.B) start[x] = tiles;
    }
    __syncthreads();                            // item() reads every warp's starts
    // row_starts that overlap could make more items than there is room for
    const int total = min(carry[0], (int)lm_list_items(p.rows, p.B, p.sh.group));
    // the item of number e, and its K/V tiles
    auto item = [&](int e, int4& rows) {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] <= e) lo = mid; else hi = mid - 1;
        }
        int first, n, k;
        const int b = order[lo];
        if (sorted) {
            first = row0[b];
            n = nrow[b];
            k = keys[b];
        } else {
            k = rows_and_keys(b, first, n, false);
        }
        const int t = (n + pair - 1) / pair - 1 - (e - start[lo]);
        rows = make_int4(b, first + t * pair, min(pair, n - t * pair), k - n + t * pair + 1);
        return (max(0, rows.w + rows.z - 1) + kTile - 1) / kTile;
    };
    if (!p.split) {
        for (int e = tid; e < total; e += kListThreads) {
            int4 rows;
            item(e, rows);
            list[2 * e] = rows;
            list[2 * e + 1] = make_int4(0, kNone, -1, 0);
        }
        if (tid == 0) {
            p.counts[0] = total;
            p.counts[1] = 0;
        }
        return;
    }
    // a call whose items may be cut has at most 2 kSms of them: one per thread
    int4 rows = make_int4(0, 0, 0, 0);
    const int tiles = tid < total ? item(tid, rows) : 0;
    unsigned long long sum = tiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0 && sum) atomicAdd(&work, sum);        // whole numbers: any order
    __syncthreads();                            // every thread has its total: carry begins anew
    if (tid < 3) carry[tid] = 0;
    __syncthreads();
    const int share = (int)min(max((work * p.sh.hk + kSms - 1) / kSms, (unsigned long long)kMinPiece),
                               1ull << 24);
    const int pieces = tid >= total ? 0 : tiles > share + share / 4 ? (tiles + share / 2) / share : 1;
    int v[3] = {pieces, pieces > 1 ? pieces * p.sh.hk : 0, pieces > 1 ? 1 : 0};
    scan(v, 3);
    if (tid == 0) {
        p.counts[0] = carry[0];
        p.counts[1] = 0;
        p.counts[2] = carry[2];
    }
    // the shares bound the slots; should they not, the item stays whole (and keeps its places)
    const bool cut = pieces > 1 && v[1] + pieces * p.sh.hk <= kLmSlots;
    const int len = cut ? (tiles + pieces - 1) / pieces : kNone;
    for (int c = 0; c < pieces; c++) {
        const bool live = cut ? c * len < tiles : c == 0;
        list[2 * (v[0] + c)] = live ? rows : make_int4(rows.x, rows.y, 0, 0);
        list[2 * (v[0] + c) + 1] = cut && live ? make_int4(c * len, len, v[1] + c * p.sh.hk, 0) : make_int4(0, kNone, -1, 0);
    }
    if (pieces > 1)
        p.joins[v[2]] = make_int4(rows.y, cut ? rows.z : 0, v[1] | (cut ? (tiles + len - 1) / len : 0) << 16, rows.w);
}
static_assert(2 * kSms <= kListThreads, "a thread per item that may be cut");

// Joins the pieces of items that were cut: a warp per row.
constexpr int kPieceThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kPieceThreads, 4) lm_pieces_kernel(const __grid_constant__ Params p)
{
    pdl_wait();
    pdl_launch();
    const int lane = threadIdx.x & 31, group = p.sh.group;
    const long long total = (long long)__ldcg(p.counts + 2) * p.sh.hk * 2 * kTile;
    const long long warps = gridDim.x * (kPieceThreads / 32LL);
    for (long long x = blockIdx.x * (kPieceThreads / 32LL) + (threadIdx.x >> 5); x < total; x += warps) {
        const int r = (int)(x % (2 * kTile));
        const int y = (int)(x / (2 * kTile)), hk = y % p.sh.hk;
        const int4 j = __ldcg(p.joins + y / p.sh.hk);
        const int i = r / kTile, in = r % kTile, tok = i * p.tokens + in / group;
        if (in >= p.tokens * group || tok >= j.y) continue;
        auto row_of = [&](int c) { return (long long)((j.z & 0xffff) + c * p.sh.hk + hk) * 2 * kTile + r; };
        constexpr int kE = D / 32;
        float v[kE], lse;
        join_row<kE, 4>(
            j.z >> 16, j.w + tok <= 0, [&](int c) { return __ldcg(p.piece_lse + row_of(c)); },
            [&](int c, float* f) { row_part<kE>(p.piece + row_of(c) * D, f); }, v, lse);
        const long long row = j.x + tok;
        const int h = hk * group + in % group;
        T* dst = static_cast<T*>(p.o) + row * p.os + (long long)h * D + lane * kE;
        if constexpr (kE == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(Two<T>::pack(v[0], v[1]), Two<T>::pack(v[2], v[3]));
        else
            *reinterpret_cast<uint32_t*>(dst) = Two<T>::pack(v[0], v[1]);
        if (p.lse && lane == 0) p.lse[row * p.sh.hq + h] = lse;
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

template <typename T, int D, bool kRowScale = false>
cudaError_t launch(const LmShape& sh, const void* q, long long qs, const LmKeys& ks, Params& p, dim3 grid,
                   cudaStream_t s, int4* list)
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
    p.v = ks.v;
    p.v_stride = v_stride;
    CUtensorMap mq, mk, mv;
    if (!lm_make_map(&mq, sh.type, q, D, sh.hq, p.rows, qs, sh.group, p.tokens) ||
        !lm_make_map(&mk, sh.type, ks.k, D, sh.hk, key_rows, k_stride, 1, box) ||
        !lm_make_map(&mv, sh.type, ks.v, D, sh.hk, key_rows, v_stride, 1, box))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    if (list) {
        e = launch_pdl(lm_list_kernel, dim3(1), dim3(kListThreads), 0, s, p, list);
        if (e != cudaSuccess) return e;
        p.list = list;
    }
    e = launch_pdl(lm_prompt_kernel<T, D, kRowScale>, grid, dim3(kThreads), smem_bytes<D>(), s, mq, mk, mv, p);
    if (e != cudaSuccess || !p.split) return e;
    // a row per warp where they fit: four rows per warp in turn, 608 CTAs less, took
    // 40 instead of 34 us for 670 tokens behind 6,000 positions, eight K/V heads
    const int ctas = std::min(8 * kSms, p.most_cut * 2 * kTile / (kPieceThreads / 32));
    return launch_pdl(lm_pieces_kernel<T, D>, dim3(ctas), dim3(kPieceThreads), 0, s, p);
}

cudaError_t launch_any(const LmShape& sh, const void* q, long long qs, const LmKeys& ks, Params& p, dim3 grid,
                       cudaStream_t s, int4* list = nullptr)
{
    if (sh.type == CODEC_LM_BF16)
        return sh.D == 128 ? launch<__nv_bfloat16, 128>(sh, q, qs, ks, p, grid, s, list)
                           : launch<__nv_bfloat16, 64>(sh, q, qs, ks, p, grid, s, list);
    return sh.D == 128 ? launch<__half, 128>(sh, q, qs, ks, p, grid, s, list)
                       : launch<__half, 64>(sh, q, qs, ks, p, grid, s, list);
}

}  // namespace

cudaError_t configure_lm_prompt()
{
    const std::pair<const void*, size_t> kernels[] = {{(const void*)lm_prompt_kernel<__nv_bfloat16, 128>, smem_bytes<128>()},
                                                      {(const void*)lm_prompt_kernel<__nv_bfloat16, 64>, smem_bytes<64>()},
                                                      {(const void*)lm_prompt_kernel<__half, 128>, smem_bytes<128>()},
                                                      {(const void*)lm_prompt_kernel<__half, 64>, smem_bytes<64>()},
                                                      {(const void*)lm_prompt_kernel<__half, 128, true>, smem_bytes<128>()},
                                                      {(const void*)lm_prompt_kernel<__half, 64, true>, smem_bytes<64>()}};
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
    // Pairs of query tiles: at most one partly filled pair per request.  Cutting
    // along the keys pays where items are few for the SMs and their keys may be
    // many: 64 tokens behind 32,768 positions, eight items, take 43 us cut and 373
    // whole.  It costs about 5 us: 20 requests of 18 tokens behind 300 to 3,150
    // positions, 160 items, take 48 us whole and 52 cut.  The fewer the items, the
    // sooner: tables of more than 1,280 positions where they are at most 48 (whole and
    // cut, 16 / 8 heads of 128: 1 token behind 1,299 positions 22.2 and 17.9 us, 4 of 60
    // behind 1,240 25.2 and 24.0; but 300 behind 730 23.2 and 27.8, 2 of 200 behind 890
    // 24.6 and 28.7, 60 behind 1,030 20.1 and 21.4), else of more than 2,048 (4 of 200
    // behind 1,800, 80 items, 34.2 and 35.5).
    const long long items = lm_list_items(a.rows, a.B, sh.group) * sh.hk;
    const bool cut = a.keys.tables ? items <= kSms && ((long long)a.keys.table_blocks << a.keys.bs_shift) >
                                                          (items <= 48 ? 1280 : 2048)
                                   : items <= 2 * kSms && a.rows > 2048;
    if (items <= kSms && !cut)
        return launch_any(sh, a.q, a.qs, a.keys, p, dim3((unsigned)(items / sh.hk), (unsigned)sh.hk), s);
    p.split = cut;
    p.most_cut = (int)std::min<long long>(items, kLmSlots / 2);
    p.counts = a.ws.counts;
    p.joins = static_cast<int4*>(a.ws.joins);
    p.piece = a.ws.piece;
    p.piece_lse = a.ws.piece_lse;
    return launch_any(sh, a.q, a.qs, a.keys, p, dim3(kSms), s, static_cast<int4*>(a.ws.list));
}

static dim3 shared_grid(const LmShape& sh, const LmSharedArgs& a)
{
    const int pair = 2 * (kTile / sh.group);
    return dim3((a.B + pair - 1) / pair, sh.hk, (a.shared_len + a.split_len - 1) / a.split_len);
}

long long lm_shared_ctas(const LmShape& sh, const LmSharedArgs& a)
{
    const dim3 g = shared_grid(sh, a);
    return (long long)g.x * g.y * g.z;
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
    const dim3 grid = shared_grid(sh, a);
    p.row_c = a.row_c;
    if (a.row_c)
        return sh.D == 128 ? launch<__half, 128, true>(sh, a.q, a.qs, ks, p, grid, s, nullptr)
                           : launch<__half, 64, true>(sh, a.q, a.qs, ks, p, grid, s, nullptr);
    return launch_any(sh, a.q, a.qs, ks, p, grid, s);
}

}  // namespace codec
