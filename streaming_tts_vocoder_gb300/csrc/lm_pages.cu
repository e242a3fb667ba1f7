// Blocks that several rows hold: rows that go on from others, held blocks moved
// together, blocks copied.
//
// fork and compact are integer work with an order: what is counted for a block
// has to be complete before blocks are given out or back, and those are listed by
// ascending id.  One cluster of CTAs does each call in one launch, with the cluster's
// barrier between the phases; sums are the only atomics, so no order shows in a
// result.
//
// Both are chains of dependent steps (lengths, tables, counts, lists), so latency is
// what they cost: 9 us for 16 rows, 11 for 512 rows of 200 to 2,000 positions.  The
// copies behind them are the memory's: 2 GB moved for 256 requests in 2 layers take 307 us
// with their compaction, 6.4 TB/s (94 % of a plain copy's 6.8).
#include <algorithm>
#include <climits>

#include "lm.h"

namespace codec {

namespace {

constexpr int kPageThreads = 1024;
// With 1, 2, 4, 8 CTAs a fork of 64 x 8 rows and its copies take 75.8, 59.3, 50.7, 45.7 us,
// compaction of 256 requests and its copies 368, 346, 334, 331; 16 rows 10 us with any.
constexpr int kPageCtas = 8;

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// *p of the cluster's CTA r (shared memory).
__device__ __forceinline__ int theirs(const int* p, int r)
{
    uint32_t at, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(r));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return (int)v;
}

__device__ __forceinline__ int warp_incl(int v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
    }
    return v;
}

// Inclusive running sum over the CTA's threads; total: the CTA's.  sm: 33 ints.
__device__ __forceinline__ int cta_incl(int v, int* sm, int& total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int at = warp_incl(v);
    __syncthreads();            // sm may still be read
    if (lane == 31) sm[w] = at;
    __syncthreads();
    if (w == 0) {
        const int x = sm[lane], incl = warp_incl(x);
        sm[lane] = incl - x;
        if (lane == 31) sm[32] = incl;
    }
    __syncthreads();
    total = sm[32];
    return at + sm[w];
}

// Entries of the tables that are in use, shared among the cluster's warps: use(row,
// entry, load(row, entry)) for the count(row) first ones of each.  A warp loads
// those of four rows before it uses one (each load alone costs its whole latency).
template <typename Count, typename Load, typename Use>
__device__ __forceinline__ void entries(int B, Count count, Load load, Use use)
{
    constexpr int kRows = 4;
    const int w = blockIdx.x * (kPageThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kPageThreads / 32);
    for (int b0 = w; b0 < B; b0 += kRows * warps) {
        int n[kRows], most = 0;
#pragma unroll
        for (int i = 0; i < kRows; i++) {
            n[i] = b0 + i * warps < B ? count(b0 + i * warps) : 0;
            most = max(most, n[i]);
        }
        for (int j = lane; j < most; j += 32) {
            int id[kRows];
#pragma unroll
            for (int i = 0; i < kRows; i++) id[i] = j < n[i] ? load(b0 + i * warps, j) : 0;
#pragma unroll
            for (int i = 0; i < kRows; i++)
                if (j < n[i]) use(b0 + i * warps, j, id[i]);
        }
    }
}

__device__ __forceinline__ int blocks_of(int n, int shift) { return (int)(((long long)n + (1 << shift) - 1) >> shift); }

// ---- fork -------------------------------------------------------------------

// Shared memory: of each row its parent (-1: none), children, first child,
// length, and its copy's place among them; then the running sums'.
size_t fork_smem(int B) { return (size_t)B * 5 * 4 + 64 * 4; }

__global__ void __launch_bounds__(kPageThreads) lm_fork_kernel(const LmForkArgs a)
{
    extern __shared__ int sm[];
    int* parent = sm;
    int* children = parent + a.B;
    int* first = children + a.B;
    int* len = first + a.B;
    int* copy = len + a.B;          // -1: it makes none
    int* scan = copy + a.B;
    __shared__ int freed;
    const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x, all = ctas * kPageThreads;
    const int most = a.table_blocks << a.bs_shift;
    pdl_wait();
    pdl_launch();
    const long long head = a.free_in[0], tail = a.free_in[1];
    const bool ring_ok = head >= 0 && tail >= head && tail - head <= a.n_blocks;
    const int n_free = ring_ok ? (int)(tail - head) : 0;
    const int head_at = ring_ok ? (int)(head % a.n_blocks) : 0, tail_at = ring_ok ? (int)(tail % a.n_blocks) : 0;
    auto ring = [&](int at, int i) {
        const long long x = (long long)at + i;
        return (int)(x >= a.n_blocks ? x - a.n_blocks : x);
    };

    // owners after: those before, then the changes
    for (int i = rank * kPageThreads + tid; i < a.n_blocks; i += all) a.owners_out[i] = __ldg(a.owners + i);

    // every CTA plans the rows for itself
    for (int b = tid; b < a.B; b += kPageThreads) {
        children[b] = 0;
        first[b] = INT_MAX;
        const int n = __ldg(a.len + b);
        len[b] = n >= 0 && n <= most ? n : -1;
    }
    __syncthreads();
    for (int b = tid; b < a.B; b += kPageThreads) {
        int p = __ldg(a.parents + b);
        if (p < 0 || p >= a.B || len[p] < 0) p = -1;
        parent[b] = p;
        if (p >= 0) atomicMin(&first[p], b);
    }
    __syncthreads();
    auto unfilled = [&](int r) {    // its last block is its own and not full
        const int n = len[r];
        return n > 0 && (n & ((1 << a.bs_shift) - 1)) != 0 && blocks_of(n, a.bs_shift) > a.shared_blocks;
    };
    int before = 0;
    for (int base = 0; base < a.B; base += kPageThreads) {
        const int b = base + tid;
        int need = 0;
        if (b < a.B) {
            const int p = parent[b];
            need = p >= 0 && first[p] != b && unfilled(p);
        }
        int total;
        const int upto = before + cta_incl(need, scan, total);
        before += total;
        if (b < a.B) {
            const int p = parent[b];
            const bool ok = p >= 0 && (!need || upto <= n_free);
            copy[b] = need && ok ? upto - 1 : -1;
            if (ok) atomicAdd(&children[p], 1);
            if (rank == 0) {
                const int want = __ldg(a.parents + b);
                a.status[b] = want != -1 && p < 0 ? 2 : p >= 0 && !ok ? 1 : 0;
                a.kv_len[b] = ok ? len[p] : 0;
                if (want >= 0 && want < a.B && p < 0) atomicOr(a.err, CODEC_LM_ERR_LENGTH);
            }
            if (!ok) parent[b] = -1;
        }
    }
    const int taken = min(before, n_free);
    if (rank == 0 && tid == 0) {
        a.copies[0] = taken;
        if (!ring_ok) atomicOr(a.err, CODEC_LM_ERR_FREE);
    }
    __syncthreads();

    // tables of the rows that go on, and their copies
    entries(a.B, [&](int b) { return parent[b] < 0 ? 0 : blocks_of(len[parent[b]], a.bs_shift); },
            [&](int b, int j) { return __ldg(a.tables + (long long)parent[b] * a.table_blocks + j); },
            [&](int b, int j, int id) {
                const int p = parent[b];
                if (copy[b] >= 0 && j == blocks_of(len[p], a.bs_shift) - 1) {
                    const int fresh = a.free_list[ring(head_at, copy[b])];
                    a.copy_src[copy[b]] = id;
                    a.copy_dst[copy[b]] = fresh;
                    id = fresh;
                }
                a.tables_out[(long long)b * a.table_blocks + j] = id;
            });
    cluster_barrier();              // owners_out holds the numbers before

    // a row's blocks have as many holders more as it has children beyond one
    entries(a.B, [&](int r) { return len[r] <= 0 || children[r] == 1 ? 0 : blocks_of(len[r], a.bs_shift); },
            [&](int r, int j) { return __ldg(a.tables + (long long)r * a.table_blocks + j); },
            [&](int r, int j, int id) {
                if (j < a.shared_blocks) return;
                const bool last = unfilled(r) && j == blocks_of(len[r], a.bs_shift) - 1;
                const int more = (last ? min(children[r], 1) : children[r]) - 1;
                if (more == 0) return;
                if (id < 0 || id >= a.n_blocks) {
                    atomicOr(a.err, CODEC_LM_ERR_BLOCK);
                    return;
                }
                atomicAdd(a.owners_out + id, more);
            });
    cluster_barrier();

    // blocks without a holder, in ascending order: the CTAs have consecutive parts
    const int span = (a.n_blocks + ctas - 1) / ctas;
    const int lo = (int)min((long long)a.n_blocks, (long long)rank * span), hi = (int)min((long long)a.n_blocks, (long long)lo + span);
    int mine = 0;
    for (int i = lo + tid; i < hi; i += kPageThreads) mine += __ldcg(a.owners_out + i) < 0;
    int total;
    cta_incl(mine, scan, total);
    if (tid == 0) freed = total;
    cluster_barrier();
    int ahead = 0, freed_all = 0;
    for (int r = 0; r < ctas; r++) {
        const int n = theirs(&freed, r);
        if (r < rank) ahead += n;
        freed_all += n;
    }
    const int given = ring_ok ? min(freed_all, a.n_blocks - n_free) : 0;
    for (int base = lo; base < hi; base += kPageThreads) {
        const int i = base + tid;
        const int n = i < hi ? __ldcg(a.owners_out + i) : 0;
        const int at = ahead + cta_incl(n < 0, scan, total) - 1;
        ahead += total;
        if (n < 0) {
            if (at < given) a.free_list[ring(tail_at, at)] = i;
            a.owners_out[i] = 0;
            if (n < -1) atomicOr(a.err, CODEC_LM_ERR_OWNERS);
        }
    }
    if (rank == 0 && tid == 0) {
        a.free_out[0] = head + taken;
        a.free_out[1] = tail + given;
    }
    cluster_barrier();              // nobody's shared memory is read any more
}

// ---- compact ----------------------------------------------------------------

__global__ void __launch_bounds__(kPageThreads)
    lm_compact_kernel(const LmCompactArgs a)
{
    __shared__ int scan[64];
    __shared__ int counts[3];
    const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x, all = ctas * kPageThreads;
    const long long most = (long long)a.table_blocks << a.bs_shift;
    pdl_wait();
    pdl_launch();
    for (int i = rank * kPageThreads + tid; i < a.n_blocks; i += all) a.map[i] = 0;
    cluster_barrier();
    auto held = [&](int b) {
        int n = __ldg(a.len + b);
        lm_clamp_len(n, most);
        return blocks_of(n, a.bs_shift);
    };
    // map: 1 for the blocks in use
    auto mark = [&](int id) {
        if (id < 0 || id >= a.n_blocks)
            atomicOr(a.err, CODEC_LM_ERR_BLOCK);
        else
            a.map[id] = 1;
    };
    entries(a.B, held, [&](int b, int j) { return __ldg(a.tables + (long long)b * a.table_blocks + j); },
            [&](int b, int j, int id) {
                if (j >= a.shared_blocks) mark(id);
            });
    for (int j = rank * kPageThreads + tid; j < a.shared_blocks; j += all) mark(__ldg(a.shared_table + j));
    if (rank == 0)
        for (int b = tid; b < a.B; b += kPageThreads) {
            int n = __ldg(a.len + b);
            if (!lm_clamp_len(n, most)) atomicOr(a.err, CODEC_LM_ERR_LENGTH);
        }
    cluster_barrier();

    const int span = (a.n_blocks + ctas - 1) / ctas;
    const int lo = (int)min((long long)a.n_blocks, (long long)rank * span), hi = (int)min((long long)a.n_blocks, (long long)lo + span);
    int mine = 0, total;
    for (int i = lo + tid; i < hi; i += kPageThreads) mine += __ldcg(a.map + i);
    cta_incl(mine, scan, total);
    if (tid == 0) counts[0] = total;
    cluster_barrier();
    int used = 0;
    for (int r = 0; r < ctas; r++) used += theirs(&counts[0], r);

    // of this CTA's ids: those in use that lie behind, those free that lie before
    int away = 0, room = 0;
    for (int i = lo + tid; i < hi; i += kPageThreads) {
        const int u = __ldcg(a.map + i);
        away += u && i >= used;
        room += !u && i < used;
    }
    int total_room;
    cta_incl(away, scan, total);
    cta_incl(room, scan, total_room);
    if (tid == 0) {
        counts[1] = total;
        counts[2] = total_room;
    }
    cluster_barrier();
    int before = 0, before_room = 0, moves = 0;
    for (int r = 0; r < ctas; r++) {
        const int n = theirs(&counts[1], r);
        if (r < rank) {
            before += n;
            before_room += theirs(&counts[2], r);
        }
        moves += n;
    }
    for (int base = lo; base < hi; base += kPageThreads) {
        const int i = base + tid;
        const int u = i < hi ? __ldcg(a.map + i) : 0;
        const bool out = u && i >= used, in = i < hi && !u && i < used;
        const int k = before + cta_incl(out, scan, total) - 1;
        before += total;
        const int m = before_room + cta_incl(in, scan, total) - 1;
        before_room += total;
        if (out) a.copy_src[k] = i;
        if (in) a.copy_dst[m] = i;
    }
    for (int i = rank * kPageThreads + tid; i < a.n_blocks - used; i += all) a.free_list[i] = used + i;
    if (rank == 0 && tid == 0) {
        a.copies[0] = moves;
        a.free_out[0] = 0;
        a.free_out[1] = a.n_blocks - used;
    }
    cluster_barrier();
    // where blocks go: owners (marks below the number in use are not written any
    // more), and map for those that move
    if (a.owners) {
        for (int i = rank * kPageThreads + tid; i < a.n_blocks; i += all) {
            if (i >= used)
                a.owners_out[i] = 0;
            else if (__ldcg(a.map + i))
                a.owners_out[i] = __ldg(a.owners + i);
        }
    }
    for (int k = rank * kPageThreads + tid; k < moves; k += all) {
        const int from = __ldcg(a.copy_src + k), to = __ldcg(a.copy_dst + k);
        a.map[from] = to;
        if (a.owners) a.owners_out[to] = __ldg(a.owners + from);
    }
    cluster_barrier();
    auto moved = [&](int id) { return id >= used && id < a.n_blocks ? __ldcg(a.map + id) : id; };
    entries(a.B, held,
            [&](int b, int j) {
                return moved(__ldg(j < a.shared_blocks ? a.shared_table + j : a.tables + (long long)b * a.table_blocks + j));
            },
            [&](int b, int j, int id) { a.tables_out[(long long)b * a.table_blocks + j] = id; });
    for (int j = rank * kPageThreads + tid; j < a.shared_blocks; j += all)
        a.shared_out[j] = moved(__ldg(a.shared_table + j));
}

// ---- copies -----------------------------------------------------------------

constexpr int kCopyThreads = 256;
constexpr int kCopyPiece = 16 * kCopyThreads * 4;   // bytes that a CTA moves at once: four loads in flight a thread

__global__ void __launch_bounds__(kCopyThreads) lm_copy_kernel(const __grid_constant__ LmCopyArgs a)
{
    pdl_wait();
    pdl_launch();
    const int n = a.copies ? min(max(__ldg(a.copies), 0), a.n) : a.n;
    const int pieces = (int)((a.block_bytes + kCopyPiece - 1) / kCopyPiece);
    const long long all = (long long)n * a.n_caches * pieces;
    for (long long u = blockIdx.x; u < all; u += gridDim.x) {
        const int piece = (int)(u % pieces);
        const long long x = u / pieces;
        const int i = (int)(x / a.n_caches), c = (int)(x - (long long)i * a.n_caches);
        const int from = __ldg(a.src + i), to = __ldg(a.dst + i);
        if (from < 0 || from >= a.n_blocks || to < 0 || to >= a.n_blocks) {
            if (threadIdx.x == 0) atomicOr(a.err, CODEC_LM_ERR_BLOCK);
            continue;
        }
        const long long first = (long long)piece * kCopyPiece;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.caches[c]) + from * a.block_bytes + first);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.caches[c]) + to * a.block_bytes + first);
        const int vectors = (int)(min(a.block_bytes - first, (long long)kCopyPiece) >> 4);
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (threadIdx.x + j * kCopyThreads < vectors) v[j] = src[threadIdx.x + j * kCopyThreads];
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (threadIdx.x + j * kCopyThreads < vectors) dst[threadIdx.x + j * kCopyThreads] = v[j];
    }
}

}  // namespace

cudaError_t configure_lm_pages()
{
    return cudaFuncSetAttribute(lm_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)fork_smem(kLmMaxRequests));
}

// One cluster of `ctas` CTAs.
template <typename A>
static cudaError_t launch_cluster(void (*kernel)(const A), int ctas, size_t smem, cudaStream_t s, const A& a)
{
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPageThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_lm_fork(const LmForkArgs& a, cudaStream_t s)
{
    return launch_cluster(lm_fork_kernel, kPageCtas, fork_smem(a.B), s, a);
}

cudaError_t launch_lm_compact(const LmCompactArgs& a, cudaStream_t s)
{
    return launch_cluster(lm_compact_kernel, kPageCtas, 0, s, a);
}

cudaError_t launch_lm_copy(const LmCopyArgs& a, cudaStream_t s)
{
    // A CTA for a piece as long as there are 32 for an SM: 4, 8, 16, 32, 64 take 340, 329, 314,
    // 307, 304 us for the largest of these copies, and 9,728 CTAs without work take longer
    // than what 64 give.
    const long long pieces = (a.block_bytes + kCopyPiece - 1) / kCopyPiece, most = (long long)a.n * a.n_caches * pieces;
    return launch_pdl(lm_copy_kernel, dim3((unsigned)std::min<long long>(most, 152 * 32)), dim3(kCopyThreads), 0, s, a);
}

}  // namespace codec
