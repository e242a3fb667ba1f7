// Block tables and slot maps of the codec LM's cache, from request lengths.
//
// One launch.  The blocks that request b takes start behind those of all
// requests before it, so everything follows from three running sums over the
// requests (rows, blocks taken, blocks given back).  Every CTA forms them for
// itself in shared memory (at most 4096 requests; a second launch would cost
// more), then the CTAs share the rows and the table entries among them.  No
// atomics, and no order that could change a result.
//
// In place without a barrier between CTAs: a row's slot takes a block that
// this call assigns from the ring (not from the table entry that another CTA
// writes); entries that are given back and entries that are written belong to
// different requests; and the ring positions read, head .. head + taken, lie
// before the ones written, tail .. tail + given back, which are at most n_blocks
// ahead of head (any beyond are dropped: they were given back twice).
#include <climits>

#include "lm.h"

namespace codec {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanRows = 2048;     // rows that make another CTA worth its running sums

struct Scan {
    long long warp[kPlanThreads / 32];
    long long carry;
};

// Exclusive running sum over the block of one value per thread, on top of
// *carry, which then grows by the block's total.
__device__ __forceinline__ long long block_sum(Scan& s, long long v)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s.warp[w] = incl;
    __syncthreads();
    long long before = s.carry, total = 0;
    for (int i = 0; i < kPlanThreads / 32; i++) {
        if (i < w) before += s.warp[i];
        total += s.warp[i];
    }
    __syncthreads();
    if (threadIdx.x == 0) s.carry += total;
    __syncthreads();
    return before + incl - v;
}

__device__ __forceinline__ int owned(int n, int shift, int shared)
{
    return max(0, (int)(((long long)n + (1 << shift) - 1) >> shift) - shared);
}

__device__ __forceinline__ int ring_at(long long i, int n) { return (int)(i % n); }

// Largest b in [0, B) with a[b] <= x (a[0] <= x, a nondecreasing).
__device__ __forceinline__ int last_le(const int* a, int B, long long x)
{
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) lm_plan_kernel(const LmPlanArgs a)
{
    extern __shared__ int sm[];
    int* row0 = sm;                 // first row of each request (clamped to max_rows)
    int* take0 = row0 + a.B;        // blocks taken by those before it
    int* give0 = take0 + a.B;       // blocks given back by those before it
    unsigned char* st = reinterpret_cast<unsigned char*>(give0 + a.B);
    __shared__ Scan s;
    __shared__ long long rows_all, take_all, give_all;
    const int tid = threadIdx.x;
    const bool first_cta = blockIdx.x == 0;
    const long long most = (long long)a.table_blocks << a.bs_shift;

    const long long head = a.free_in[0], tail = a.free_in[1];
    const bool ring_ok = head >= 0 && tail >= head && tail - head <= a.n_blocks;
    const long long n_free = ring_ok ? tail - head : 0;
    const long long room = ring_ok ? a.n_blocks - n_free : 0;   // ids that can be put back

    // rows
    if (tid == 0) s.carry = 0;
    __syncthreads();
    for (int base = 0; base < a.B; base += kPlanThreads) {
        const int b = base + tid;
        int rows = 0;
        bool good = true;
        if (b < a.B) {
            const int n0 = __ldg(a.before + b), n1 = __ldg(a.after + b);
            good = n0 >= 0 && n1 >= 0 && n0 <= most && n1 <= most;
            rows = good ? max(0, n1 - n0) : 0;
        }
        const long long at = block_sum(s, rows);
        if (b < a.B) {
            row0[b] = (int)min(at, (long long)a.max_rows);
            st[b] = !good ? 2 : at + rows > a.max_rows ? 3 : 0;
        }
    }
    if (tid == 0) {
        rows_all = min(s.carry, (long long)a.max_rows);
        s.carry = 0;
    }
    __syncthreads();
    // blocks taken: a request is served while the sum up to it fits
    for (int base = 0; base < a.B; base += kPlanThreads) {
        const int b = base + tid;
        int need = 0;
        if (b < a.B && st[b] == 0)
            need = max(0, owned(__ldg(a.after + b), a.bs_shift, a.shared_blocks) -
                              owned(__ldg(a.before + b), a.bs_shift, a.shared_blocks));
        const long long at = block_sum(s, need);
        if (b < a.B) {
            if (need > 0 && at + need > n_free) st[b] = 1;
            take0[b] = (int)min(at, n_free);
        }
    }
    // the sums of those served: the first one that is not ends the count
    if (tid == 0) {
        take_all = min(s.carry, n_free);
        s.carry = 0;
    }
    __syncthreads();
    for (int b = tid; b < a.B; b += kPlanThreads)
        if (st[b] == 1) atomicMin(&take_all, (long long)take0[b]);
    __syncthreads();
    // blocks given back
    for (int base = 0; base < a.B; base += kPlanThreads) {
        const int b = base + tid;
        int back = 0;
        if (b < a.B && st[b] == 0)
            back = max(0, owned(__ldg(a.before + b), a.bs_shift, a.shared_blocks) -
                              owned(__ldg(a.after + b), a.bs_shift, a.shared_blocks));
        const long long at = block_sum(s, back);
        if (b < a.B) give0[b] = (int)min(at, (long long)INT_MAX);
    }
    if (tid == 0) give_all = min(s.carry, room);
    __syncthreads();

    if (first_cta) {
        for (int b = tid; b < a.B; b += kPlanThreads) {
            a.row_start[b] = row0[b];
            a.status[b] = st[b];
            a.kv_len[b] = st[b] == 0 ? __ldg(a.after + b) : 0;
        }
        if (tid == 0) {
            a.row_start[a.B] = (int)rows_all;
            a.free_out[0] = head + take_all;
            a.free_out[1] = tail + give_all;
            if (!ring_ok) atomicOr(a.err, CODEC_LM_ERR_FREE);
        }
    }

    const long long t0 = (long long)blockIdx.x * kPlanThreads + tid, step = (long long)gridDim.x * kPlanThreads;
    // table entries of the blocks taken
    for (long long e = t0; e < take_all; e += step) {
        const int b = last_le(take0, a.B, e);
        const int j = a.shared_blocks + owned(__ldg(a.before + b), a.bs_shift, a.shared_blocks) + (int)(e - take0[b]);
        a.tables[(long long)b * a.table_blocks + j] = a.free_list[ring_at(head + e, a.n_blocks)];
    }
    // blocks given back
    for (long long e = t0; e < give_all; e += step) {
        const int b = last_le(give0, a.B, e);
        const int j = a.shared_blocks + owned(__ldg(a.after + b), a.bs_shift, a.shared_blocks) + (int)(e - give0[b]);
        a.free_list[ring_at(tail + e, a.n_blocks)] = a.tables[(long long)b * a.table_blocks + j];
    }
    // the shared blocks of requests that start
    if (a.shared_blocks > 0) {
        const long long shared_len = (long long)a.shared_blocks << a.bs_shift;
        for (long long e = t0; e < (long long)a.B * a.shared_blocks; e += step) {
            const int b = (int)(e / a.shared_blocks), j = (int)(e - (long long)b * a.shared_blocks);
            const int n0 = __ldg(a.before + b);
            if (st[b] == 0 && n0 <= shared_len && __ldg(a.after + b) > n0)
                a.tables[(long long)b * a.table_blocks + j] = __ldg(a.shared_table + j);
        }
    }
    // rows
    for (long long t = t0; t < a.max_rows; t += step) {
        int slot = -1, pos = 0;
        if (t < rows_all) {
            const int b = last_le(row0, a.B, t);
            const int n0 = __ldg(a.before + b);
            pos = n0 + (int)(t - row0[b]);
            if (st[b] == 0) {
                const int j = pos >> a.bs_shift;
                const int own = a.shared_blocks + owned(n0, a.bs_shift, a.shared_blocks);
                int id;
                if (j >= own)
                    id = a.free_list[ring_at(head + take0[b] + (j - own), a.n_blocks)];
                else if (j < a.shared_blocks && n0 <= ((long long)a.shared_blocks << a.bs_shift))
                    id = __ldg(a.shared_table + j);
                else
                    id = a.tables[(long long)b * a.table_blocks + j];
                if (id >= 0 && id < a.n_blocks)
                    slot = (id << a.bs_shift) + (pos & ((1 << a.bs_shift) - 1));
                else
                    atomicOr(a.err, CODEC_LM_ERR_BLOCK);
            }
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
}

}  // namespace

size_t lm_plan_smem(int B) { return (size_t)B * 13; }

cudaError_t configure_lm_plan()
{
    // the attribute is the function's, not an object's: always the largest
    return cudaFuncSetAttribute(lm_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)lm_plan_smem(kLmMaxRequests));
}

cudaError_t launch_lm_plan(const LmPlanArgs& a, cudaStream_t s)
{
    const int ctas = min(152, (a.max_rows + kPlanRows - 1) / kPlanRows);
    lm_plan_kernel<<<ctas, kPlanThreads, lm_plan_smem(a.B), s>>>(a);
    return cudaGetLastError();
}

}  // namespace codec
