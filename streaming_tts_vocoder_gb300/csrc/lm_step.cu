// Attention of one token per request over the cache.
//
// The part of the context that all requests share is one problem with many
// query rows: lm_prompt.cu computes it, with partial results in fp32.  What
// each request has of its own is read here, once, and that is the bound:
// group x 4 flops per 4 bytes, far below the tensor pipe's balance.
//
// A unit of work is (request, K/V head, split of `chunk` positions).  The
// splits lie at fixed positions, so a result's bits do not depend on the
// batch.  The units' number is known on the device only: a CTA's producer warp
// takes one after the other, from a counter where that pays (CTAs start late
// where the shared part's kernel holds their SM), and keeps a ring of 64-key K and V tiles, the
// unit's queries with the first, in flight across units, so the copies never
// pause.
// Four warps take 16 keys of a tile each: scores and values by m16n8k16 MMAs
// with the group's heads as the 16 rows (padded; the instruction is not what
// bounds this), each warp with its own running softmax, joined at the unit's
// end.  Partial results are joined in split order: by the CTA that finishes
// the last unit of a (request, head) where no CTA has more than one unit, else
// by a kernel of its own - the fence, the counter and the join cost a CTA
// about 6,000 cycles, a third of a unit's time when one walks many.
//
// Long contexts: HBM.  256 requests of 32 / 8 heads of 128 in bf16 with 420,000
// positions of their own behind 8,192 shared ones take 277 to 282 us, 6.2 to 6.3
// TB/s (94 % of the rate of a copy); two CTAs per SM keep six stages of 32 KB in flight.  Short ones: the latency of a unit, about 3,300
// cycles of its consumers for a tile (its scores and sums half of that, the
// four warps' join the rest), and two launches where results are joined.
#include <algorithm>

#include "lm.h"
#include "lm_join.cuh"
#include "tc_ptx.cuh"

namespace codec {

namespace {

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kKeys = 64;               // keys of a tile, 16 per consumer warp
constexpr int kMaxStages = 6;
constexpr uint32_t kHalf = kKeys * 128; // 64 columns of a tile

struct Params {
    LmShape sh;
    int B;
    const void* q;
    long long qs;
    const int* tables;
    const int* kv_len;
    int table_blocks, bs_shift, n_blocks;
    const int* lead;                    // a short shared part: the blocks of the first lead_len positions
    int lead_len;
    int shared_len, n_pre;              // shared part: length, partial results of it
    int chunk, max_splits;
    int stages;
    int after_shared;                   // the shared part's kernel is running: nothing here needs its results
    float c;                            // scale x log2 e
    float* part;                        // [B][max_splits][hq][D]
    float* part_lse;
    const float* pre;                   // [n_pre][B][hq][D]
    const float* pre_lse;
    int* done;                          // [B][hk] finished units; zero between calls
    int* taken;                         // units taken from the counter (null: unit = blockIdx, + gridDim, ..); zero between calls
    void* o;
    long long os;
    float* lse;
};

template <typename T> struct Mma;
template <> struct Mma<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ void run(float* d, const uint32_t* a, uint32_t b0, uint32_t b1)
    {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Mma<__half> {
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ void run(float* d, const uint32_t* a, uint32_t b0, uint32_t b1)
    {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
    int b, hk, split, n_splits;
    int key0, keys;             // first position, positions of the split
    bool empty;                 // the request has no position at all
};

// The unit of index u: units run over the requests' splits, K/V heads innermost.
// first, lens: the requests' first units and lengths.  A whole warp: 32 places
// are looked at at once (halving took 1,100 cycles a unit for 500 requests).
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

// K tile, V tile, and the group's queries.
template <int D>
__host__ __device__ constexpr uint32_t stage_bytes(int group)
{
    return 2 * kKeys * D * 2 + ((group * D * 2 + 1023) & ~1023);
}
// A consumer's results lie [group][D + 8], so that the rows of a fragment fall into different banks.
template <int D> constexpr int kPitch = D + 8;

// [stages], then the consumers' results [4][group][pitch] fp32 and their
// maxima and sums [4][16][2], the barriers, the stages' units, and the requests'
// first units and lengths.
template <int D>
size_t smem_bytes(int stages, int group, int B)
{
    return 1024 + (size_t)stages * stage_bytes<D>(group) + (size_t)kConsumers * group * kPitch<D> * 4 + kConsumers * 16 * 8 +
           2 * kMaxStages * 8 + 16 + kMaxStages * 16 + (2 * (size_t)B + 1) * 4;
}

// Joins the partial results of (request, head), the shared part's first, in
// order.  One warp; empty: the request has no position at all.
template <typename T, int D, int kAhead>
__device__ __forceinline__ void join_parts(const Params& p, int b, int h, int n_splits, bool empty, int lane)
{
    const int parts = p.n_pre + n_splits;
    const long long shared_row = (long long)b * p.sh.hq + h, own_row = (long long)b * p.max_splits * p.sh.hq + h;
    auto row_of = [&](int i) {
        return i < p.n_pre ? (long long)i * p.B * p.sh.hq + shared_row : (long long)(i - p.n_pre) * p.sh.hq + own_row;
    };
    constexpr int kE = D / 32;
    float v[kE], lse;
    join_row<kE, kAhead>(
        parts, empty, [&](int i) { return __ldcg((i < p.n_pre ? p.pre_lse : p.part_lse) + row_of(i)); },
        [&](int i, float* x) { row_part<kE>((i < p.n_pre ? p.pre : p.part) + row_of(i) * D, x); }, v, lse);
    T* dst = static_cast<T*>(p.o) + b * p.os + (long long)h * D + lane * kE;
    if constexpr (kE == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(Mma<T>::pack(v[0], v[1]), Mma<T>::pack(v[2], v[3]));
    else
        *reinterpret_cast<uint32_t*>(dst) = Mma<T>::pack(v[0], v[1]);
    if (p.lse && lane == 0) p.lse[(long long)b * p.sh.hq + h] = lse;
}

__device__ __forceinline__ int splits_of(const Params& p, int len)
{
    return max(1, (max(0, len - p.shared_len) + p.chunk - 1) / p.chunk);
}

// A warp per (request, head) whose result is in parts.
constexpr int kJoinThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 4) lm_join_kernel(const __grid_constant__ Params p)
{
    pdl_wait();
    pdl_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.taken) *p.taken = 0;
    const long long w = blockIdx.x * (kJoinThreads / 32LL) + (threadIdx.x >> 5);
    const int b = (int)(w / p.sh.hq), h = (int)(w - (long long)b * p.sh.hq);
    if (b >= p.B) return;
    int len = __ldg(p.kv_len + b);
    lm_clamp_len(len, (long long)p.table_blocks << p.bs_shift);
    const int n = splits_of(p, len);
    if (n == 1 && p.n_pre == 0) return;         // written by its unit
    join_parts<T, D, 4>(p, b, h, n, len == 0, threadIdx.x & 31);
}

// kJoin: partial results are joined here (an instance of its own: the join's
// registers would make the main loop spill).
template <typename T, int D, bool kJoin>
__global__ void __launch_bounds__(kThreads, 2) lm_step_kernel(const __grid_constant__ CUtensorMap mk,
                                                           const __grid_constant__ CUtensorMap mv,
                                                           const __grid_constant__ Params p)
{
    constexpr uint32_t kTileBytes = kKeys * D * 2;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int group = p.sh.group;
    const uint32_t pitch = stage_bytes<D>(group);
    float* res = reinterpret_cast<float*>(smem + (size_t)p.stages * pitch);
    float* ml = res + kConsumers * group * kPitch<D>;
    uint64_t* full = reinterpret_cast<uint64_t*>(ml + kConsumers * 16 * 2);
    uint64_t* empty = full + kMaxStages;
    int* flags = reinterpret_cast<int*>(empty + kMaxStages);    // abort, last one of a (request, head)
    uint64_t* never = reinterpret_cast<uint64_t*>(flags + 2);   // nothing arrives (see LmShape::unarrived)
    // the unit whose first tile a stage holds: request (-1: no more), K/V head, split and splits << 16, positions
    int4* unit_of = reinterpret_cast<int4*>(flags + 4);
    int* first = reinterpret_cast<int*>(unit_of + kMaxStages);
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
    // all the same, as this SM's L1 may hold it from before: lengths and tables by
    // __ldcg, queries by bulk copies, keys and values by TMA, nothing by plain or
    // read-only loads.
    if (!p.after_shared) pdl_wait();
    pdl_launch();
    int unit0 = blockIdx.x;                 // of the copy warp's lane 0
    if (p.taken && warp == kConsumers && lane == 0) unit0 = atomicAdd(p.taken, 1);
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
    const int units = first[p.B] * p.sh.hk;

    if (warp == kConsumers) {
        // -------------------------------------------------------- copies --
        int st = 0, loads = 0;
        uint32_t ph = 0;
        bool ok = true;
        if (lane == 0) {
            prefetch_tensormap(&mk);
            prefetch_tensormap(&mv);
        }
        const int box_shift = min(p.bs_shift, 6);           // keys per box: a block, or half of one of 128
        const int per = kKeys >> box_shift;
        int u = __shfl_sync(0xffffffffu, unit0, 0);
        while (ok) {
            int next = u + gridDim.x;
            if (p.taken && lane == 0 && u < units) next = atomicAdd(p.taken, 1);    // needed when this unit's copies are out
            if (u >= units) u = -1;
            Unit n{};
            if (u >= 0) n = unit_at(p, first, lens, u);
            const int* table = p.tables + (long long)n.b * p.table_blocks;
            const T* q = static_cast<const T*>(p.q) + n.b * p.qs + (long long)n.hk * group * D;
            auto boxes = [&](int j) { return max(0, min(per, (n.keys - j * kKeys + (1 << box_shift) - 1) >> box_shift)); };
            auto position = [&](int j) { return n.key0 + j * kKeys + (lane << box_shift); };
            auto block = [&](int j) {
                const int pos = position(j);
                return lane < boxes(j) ? __ldcg((pos < p.lead_len ? p.lead : table) + (pos >> p.bs_shift)) : 0;
            };
            int id_ahead = block(0);
            // a unit without keys, and the end, take a stage without copies
            for (int j = 0; j == 0 || j * kKeys < n.keys; j++) {
                const int here = boxes(j), id = id_ahead;
                id_ahead = block(j + 1);
                int row = 0;
                if (lane < here) {
                    const int pos = position(j);
                    if (id < 0 || id >= p.n_blocks) {
                        atomicOr(p.sh.err, CODEC_LM_ERR_BLOCK);
                        row = p.n_blocks << p.bs_shift;     // behind the last row: the copy writes zeros
                    } else {
                        row = (id << p.bs_shift) + (pos & ((1 << p.bs_shift) - 1));
                    }
                }
                ok = mbar_wait(&empty[st], ph ^ 1u, abort_flag, kLmPolls);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t* dst = smem + (size_t)st * pitch;
                // one thread issues them all (lanes that each issue their own take turns)
                int rows[4];
#pragma unroll
                for (int b = 0; b < 4; b++) rows[b] = __shfl_sync(0xffffffffu, row, b);
                if (elect_one()) {
                    const uint32_t q_bytes = j == 0 && here > 0 ? group * D * 2 : 0;
                    if (j == 0)
                        unit_of[st] = make_int4(u < 0 ? -1 : n.b | (n.empty ? 1 << 30 : 0), n.hk, n.split | n.n_splits << 16, n.keys);
                    mbar_expect_tx(&full[st], (uint32_t)(here << box_shift) * D * 4 + q_bytes);
                    if (q_bytes) bulk_load(dst + 2 * kTileBytes, q, &full[st], q_bytes);
#pragma unroll
                    for (int b = 0; b < 4; b++)
                        if (b < here)
                            for (int h = 0; h < D / 64; h++) {
                                const uint32_t at = h * kHalf + ((uint32_t)b << box_shift) * 128;
                                tma_load_3d(dst + at, &mk, &full[st], h * 64, n.hk, rows[b]);
                                tma_load_3d(dst + kTileBytes + at, &mv, &full[st], h * 64, n.hk, rows[b]);
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
        const uint32_t base = smem_u32(smem);
        const int r0 = lane >> 2, cp = (lane & 3) * 2;      // row (and + 8) and column pair of a fragment
        const int m8 = lane >> 3, l8 = lane & 7;
        // this lane's row addresses for the K (keys x 16-byte chunks) and V fragments
        const int k_key = warp * 16 + (m8 >> 1) * 8 + l8, k_chunk = m8 & 1;
        const int v_key = warp * 16 + (m8 & 1) * 8 + l8, v_chunk = m8 >> 1;
        int st = 0;
        uint32_t ph = 0;
        // When a wait gives up inside a unit its warps still meet at the unit's
        // barriers; at the next unit they all leave, whatever has landed by then: the
        // warps may stand at different stages, and not each of those holds a unit's start.
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
            uint32_t qf[D / 16][4];
            float acc[D / 8][4];
#pragma unroll
            for (int i = 0; i < D / 8; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[i][e] = 0.f;
            float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            for (int j = 0; j == 0 || j * kKeys < n.keys; j++) {
                // (unarrived: one warp's second tile never comes)
                const bool ok = j == 0 || (p.sh.unarrived && warp == 0 && j == 1
                                               ? mbar_wait(never, 0, abort_flag, p.sh.unarrived)
                                               : mbar_wait(&full[st], ph, abort_flag, kLmPolls));
                gave_up = !__all_sync(0xffffffffu, ok);
                if (gave_up) break;
                const uint32_t kt = base + (uint32_t)st * pitch, vt = kt + kTileBytes;
                if (j == 0 && n.keys > 0) {     // rows behind the group's repeat its last: nobody reads them
                    const uint32_t qt = vt + kTileBytes + min((m8 & 1) * 8 + l8, group - 1) * D * 2 + (m8 >> 1) * 16;
#pragma unroll
                    for (int k = 0; k < D / 16; k++) ldsm4(qt + k * 32, qf[k]);
                }
                const int left = n.keys - j * kKeys - warp * 16;    // keys of the warp's 16 that exist
                if (left > 0) {
                    float s[2][4] = {};
#pragma unroll
                    for (int k = 0; k < D / 16; k++) {
                        const int c = k * 2 + k_chunk;
                        uint32_t f[4];
                        ldsm4(kt + (c >> 3) * kHalf + k_key * 128 + (((c & 7) ^ (k_key & 7)) << 4), f);
                        Mma<T>::run(s[0], qf[k], f[0], f[1]);
                        Mma<T>::run(s[1], qf[k], f[2], f[3]);
                    }
                    if (left < 16) {
#pragma unroll
                        for (int i = 0; i < 2; i++)
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                if (i * 8 + cp + (e & 1) >= left) s[i][e] = -INFINITY;
                    }
                    float m[2];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        m[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
                        m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 1));
                        m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 2));
                    }
                    // a row's reference moves up by more than 8 (in log2) or not at all, for its own
                    // scores alone, as for prompts (times 1 changes nothing)
                    if (__any_sync(0xffffffffu, (m[0] - ref[0]) * p.c > 8.f || (m[1] - ref[1]) * p.c > 8.f)) {
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const bool up = (m[h] - ref[h]) * p.c > 8.f;
                            const float f = !up ? 1.f : ref[h] == -INFINITY ? 0.f : exp2_fast((ref[h] - m[h]) * p.c);
                            ref[h] = up ? m[h] : ref[h];
                            l[h] *= f;
#pragma unroll
                            for (int i = 0; i < D / 8; i++) {
                                acc[i][2 * h] *= f;
                                acc[i][2 * h + 1] *= f;
                            }
                        }
                    }
                    const float b0 = ref[0] == -INFINITY ? 0.f : -ref[0] * p.c;
                    const float b1 = ref[1] == -INFINITY ? 0.f : -ref[1] * p.c;
                    uint32_t pf[4];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float x0 = exp2_fast(fmaf(s[i][0], p.c, b0)), x1 = exp2_fast(fmaf(s[i][1], p.c, b0));
                        const float y0 = exp2_fast(fmaf(s[i][2], p.c, b1)), y1 = exp2_fast(fmaf(s[i][3], p.c, b1));
                        l[0] += x0 + x1;
                        l[1] += y0 + y1;
                        pf[2 * i] = Mma<T>::pack(x0, x1);
                        pf[2 * i + 1] = Mma<T>::pack(y0, y1);
                    }
                    // values behind the last key may be anything: they are cut out
                    uint32_t mask[2] = {0xffffffffu, 0xffffffffu};
                    if (left < 16) {
#pragma unroll
                        for (int i = 0; i < 2; i++)
                            mask[i] = (i * 8 + cp < left ? 0x0000ffffu : 0u) | (i * 8 + cp + 1 < left ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        const int c = i * 2 + v_chunk;
                        uint32_t f[4];
                        ldsm4_t(vt + (c >> 3) * kHalf + v_key * 128 + (((c & 7) ^ (v_key & 7)) << 4), f);
                        if (left < 16) {
                            f[0] &= mask[0];
                            f[1] &= mask[1];
                            f[2] &= mask[0];
                            f[3] &= mask[1];
                        }
                        Mma<T>::run(acc[2 * i], pf, f[0], f[1]);
                        Mma<T>::run(acc[2 * i + 1], pf, f[2], f[3]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
                if (++st == p.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            // join the four warps
#pragma unroll
            for (int h = 0; h < 2; h++) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                const int r = r0 + 8 * h;
                if (r < group) {
                    float* dst = res + (warp * group + r) * kPitch<D>;
#pragma unroll
                    for (int i = 0; i < D / 8; i++)
                        *reinterpret_cast<float2*>(dst + i * 8 + cp) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
                    if ((lane & 3) == 0) {
                        ml[(warp * 16 + r) * 2] = ref[h];
                        ml[(warp * 16 + r) * 2 + 1] = l[h];
                    }
                }
            }
            consumers_sync();
            const bool alone = n.n_splits == 1 && p.n_pre == 0;
            const long long at = ((long long)n.b * p.max_splits + n.split) * p.sh.hq + n.hk * group;
            for (int e = tid; e < group * (D / 4); e += 32 * kConsumers) {
                const int g = e / (D / 4), d = (e - g * (D / 4)) * 4;
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < kConsumers; w++) m = fmaxf(m, ml[(w * 16 + g) * 2]);
                float sum = 0.f;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (n.keys > 0) {
#pragma unroll
                    for (int w = 0; w < kConsumers; w++) {
                        const float mw = ml[(w * 16 + g) * 2];
                        // a warp without keys has a sum of 0 and an accumulator of 0
                        const float f = mw == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : exp2_fast((mw - m) * p.c);
                        const float4 x = *reinterpret_cast<const float4*>(res + (w * group + g) * kPitch<D> + d);
                        sum = fmaf(f, ml[(w * 16 + g) * 2 + 1], sum);
                        v.x = fmaf(f, x.x, v.x);
                        v.y = fmaf(f, x.y, v.y);
                        v.z = fmaf(f, x.z, v.z);
                        v.w = fmaf(f, x.w, v.w);
                    }
                    const float inv = 1.f / sum;
                    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                }
                const float lse = n.keys > 0 ? m * p.sh.scale + logf(sum) : -INFINITY;
                if (alone) {
                    const long long h = n.hk * group + g;
                    *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + n.b * p.os + h * D + d) =
                        make_uint2(Mma<T>::pack(v.x, v.y), Mma<T>::pack(v.z, v.w));
                    if (p.lse && d == 0) p.lse[(long long)n.b * p.sh.hq + h] = lse;
                } else {
                    __stcg(reinterpret_cast<float4*>(p.part + (at + g) * D + d), v);
                    if (d == 0) __stcg(p.part_lse + at + g, lse);
                }
            }
            if (alone || !kJoin) {
                consumers_sync();           // res is written again
                continue;
            }
            consumers_sync();
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
            if constexpr (kJoin)
                for (int g = warp; g < group; g += kConsumers)
                    join_parts<T, D, 12>(p, n.b, n.hk * group + g, n.n_splits, n.empty, lane);
        }
    }
    __syncthreads();
    if (tid == 0 && flags[0]) atomicOr(p.sh.err, CODEC_LM_ERR_TIMEOUT);
    // this kernel's end is its predecessors' too
    if (p.after_shared) pdl_wait();
}

template <typename T, int D>
cudaError_t launch(const LmShape& sh, const LmStepArgs& a, cudaStream_t s)
{
    const LmKeys& ks = a.keys;
    Params p{};
    p.sh = sh;
    p.B = a.B;
    p.q = a.q;
    p.qs = a.qs;
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
    p.o = a.o;
    p.os = a.os;
    p.lse = a.lse;
    bool after_shared = false;
    // A short shared part is read by every request, from L2 for all but the first:
    // no second kernel, and nothing to join with.  Device time as a part of its own
    // and so: 3 requests, 1 head, 32 positions 10.4 and 7.4 us; 32, 8, 256 11.7 and
    // 9.4; 32, 1, 1,024 14.6 and 11.0; but 16, 8, 512 11.9 and 13.5; 8, 1, 4,096 13.8
    // and 18.8.  By the largest batch, so that the actual one changes no bits.
    const long long most_short = p.shared_len <= 256 ? 65536 : p.shared_len <= 1024 ? 32768 : 0;
    if (a.ws.heads == sh.hk || a.ws.heads * p.shared_len <= most_short) {
        p.lead = a.shared_table;
        p.lead_len = p.shared_len;
        p.shared_len = 0;
    }
    if (p.shared_len > 0) {
        LmSharedArgs c{a.q, a.qs, a.B, ks, a.shared_table, p.shared_len, 0, a.ws.pre, a.ws.pre_lse};
        // splits by the object's shape and the shared length alone
        const int n = lm_shared_splits(a.ws.shared_ctas, p.shared_len);
        c.split_len = ((p.shared_len + n - 1) / n + 127) & ~127;
        p.n_pre = (p.shared_len + c.split_len - 1) / c.split_len;
        // beside the shared part only while that one's CTAs all fit the GPU at once:
        // then none of them can wait for an SM that this kernel's CTAs hold
        after_shared = lm_shared_ctas(sh, c) <= 152;
        const cudaError_t e = launch_lm_shared(sh, c, s);
        if (e != cudaSuccess) return e;
    }
    const int box = std::min(kKeys, 1 << ks.bs_shift);
    CUtensorMap mk, mv;
    const long long rows = (long long)ks.n_blocks << ks.bs_shift;
    if (!lm_make_map(&mk, sh.type, ks.k, D, sh.hk, rows, (long long)sh.hk * D, 1, box) ||
        !lm_make_map(&mv, sh.type, ks.v, D, sh.hk, rows, (long long)sh.hk * D, 1, box))
        return cudaErrorInvalidValue;
    // two CTAs per SM where two of at least two stages fit
    constexpr size_t kSm = 228 * 1024, kOne = 227 * 1024;
    int per_sm = 2;
    p.stages = kMaxStages;
    while (p.stages > 2 && per_sm * (smem_bytes<D>(p.stages, sh.group, a.B) + 1024) > kSm) p.stages--;
    if (per_sm * (smem_bytes<D>(p.stages, sh.group, a.B) + 1024) > kSm) {
        per_sm = 1;
        p.stages = kMaxStages;
        while (p.stages > 2 && smem_bytes<D>(p.stages, sh.group, a.B) > kOne) p.stages--;
    }
    // a unit per request and head at least, and no more CTAs than the SMs hold at once
    const long long most = (long long)a.B * p.max_splits * sh.hk;
    const unsigned ctas = (unsigned)std::min<long long>(152 * per_sm, most);
    p.after_shared = after_shared;
    // joined in this kernel where a CTA has one unit at most and needs no other kernel's results
    const bool join = most <= ctas && p.n_pre == 0, two = !join && (p.n_pre > 0 || p.max_splits > 1);
    // Units from the counter where requests are split or the shared part holds SMs (300
    // of 500 to 600 positions 113 us, by blockIdx 121; 64 behind a shared 1,024 16.2 and
    // 19.3), else by blockIdx, which is there at once (64 of up to 250: 9.3, 10.6 counted).
    p.taken = two ? a.ws.taken : nullptr;
    const cudaError_t e = launch_pdl(join ? lm_step_kernel<T, D, true> : lm_step_kernel<T, D, false>, dim3(ctas), dim3(kThreads), smem_bytes<D>(p.stages, sh.group, a.B), s, mk,
                                     mv, p);
    if (e != cudaSuccess || !two) return e;
    return launch_pdl(lm_join_kernel<T, D>, dim3((unsigned)(((long long)a.B * sh.hq + kJoinThreads / 32 - 1) / (kJoinThreads / 32))),
                      dim3(kJoinThreads), 0, s, p);
}

}  // namespace

cudaError_t configure_lm_step()
{
    const void* kernels[] = {
        (const void*)lm_step_kernel<__nv_bfloat16, 128, false>, (const void*)lm_step_kernel<__nv_bfloat16, 64, false>,
        (const void*)lm_step_kernel<__half, 128, false>,        (const void*)lm_step_kernel<__half, 64, false>,
        (const void*)lm_step_kernel<__nv_bfloat16, 128, true>,  (const void*)lm_step_kernel<__nv_bfloat16, 64, true>,
        (const void*)lm_step_kernel<__half, 128, true>,         (const void*)lm_step_kernel<__half, 64, true>};
    for (const void* k : kernels) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_lm_step(const LmShape& sh, const LmStepArgs& a, cudaStream_t s)
{
    if (sh.type == CODEC_LM_BF16)
        return sh.D == 128 ? launch<__nv_bfloat16, 128>(sh, a, s) : launch<__nv_bfloat16, 64>(sh, a, s);
    return sh.D == 128 ? launch<__half, 128>(sh, a, s) : launch<__half, 64>(sh, a, s);
}

}  // namespace codec
