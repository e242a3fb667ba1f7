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
//
// Bound by latency: 64 requests of one token each take 7.0 us, 1,000 that start
// with 475,000 rows 7.7 us (3.9 MB: 0.6 us).  A launch is 2.3 of it, the rest the
// chain of dependent steps: counters and lengths from memory, the sums, the
// look-up of a row's request, its block's id, the store.
#include <climits>

#include "lm.h"

namespace codec {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 4096;     // rows that make another CTA worth its running sums

struct Sums {
    long long rows, take, give;
    __device__ __forceinline__ Sums operator+(const Sums& o) const { return {rows + o.rows, take + o.take, give + o.give}; }
};

__device__ __forceinline__ Sums warp_sums(Sums v)       // inclusive
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums up = {__shfl_up_sync(0xffffffffu, v.rows, o), __shfl_up_sync(0xffffffffu, v.take, o),
                         __shfl_up_sync(0xffffffffu, v.give, o)};
        if (lane >= o) v = v + up;
    }
    return v;
}

__device__ __forceinline__ int owned(int n, int shift, int shared)
{
    return max(0, (int)(((long long)n + (1 << shift) - 1) >> shift) - shared);
}

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

// vec: slots and positions lie on 16 bytes.
__global__ void __launch_bounds__(kPlanThreads) lm_plan_kernel(const LmPlanArgs a, int vec)
{
    extern __shared__ int sm[];
    int* row0 = sm;                 // first row of each request (clamped to max_rows)
    int* take0 = row0 + a.B;        // blocks taken by those before it
    int* give0 = take0 + a.B;       // blocks given back by those before it
    unsigned char* st = reinterpret_cast<unsigned char*>(give0 + a.B);
    __shared__ Sums warp_total[kPlanThreads / 32];
    __shared__ Sums carry;
    __shared__ long long take_all, give_all;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const bool first_cta = blockIdx.x == 0;
    const int most = a.table_blocks << a.bs_shift;
    pdl_wait();
    pdl_launch();

    const long long head = a.free_in[0], tail = a.free_in[1];
    const bool ring_ok = head >= 0 && tail >= head && tail - head <= a.n_blocks;
    const long long n_free = ring_ok ? tail - head : 0;
    const long long room = ring_ok ? a.n_blocks - n_free : 0;   // ids that can be put back
    const int head_at = ring_ok ? (int)(head % a.n_blocks) : 0, tail_at = ring_ok ? (int)(tail % a.n_blocks) : 0;
    auto ring = [&](int at, long long i) {                      // i < n_blocks
        const long long x = at + i;
        return (int)(x >= a.n_blocks ? x - a.n_blocks : x);
    };

    // All three sums at once.  Requests that grow are served up to the first
    // whose rows or blocks do not fit (later ones that need some fit no better),
    // so the sums need not leave anybody out.
    if (tid == 0) {
        carry = {0, 0, 0};
        take_all = give_all = LLONG_MAX;
    }
    __syncthreads();
    for (int base = 0; base < a.B; base += kPlanThreads) {
        const int b = base + tid;
        Sums own{0, 0, 0};
        bool good = true;
        if (b < a.B) {
            const int n0 = __ldg(a.before + b), n1 = __ldg(a.after + b);
            good = n0 >= 0 && n1 >= 0 && n0 <= most && n1 <= most;
            if (good) {
                const int more = owned(n1, a.bs_shift, a.shared_blocks) - owned(n0, a.bs_shift, a.shared_blocks);
                own = {max(0, n1 - n0), max(0, more), max(0, -more)};
            }
        }
        Sums at = warp_sums(own);
        if (lane == 31) warp_total[w] = at;
        __syncthreads();
        if (w == 0) {
            const Sums v = warp_sums(warp_total[lane]);
            warp_total[lane] = carry + v;                       // everything up to that warp
        }
        __syncthreads();
        const Sums before = w > 0 ? warp_total[w - 1] : carry;
        at = before + at;                                       // up to and with this request
        if (b < a.B) {
            int status = 0;
            if (!good) status = 2;
            else if (at.rows > a.max_rows) status = 3;          // and so for every request behind it
            else if (own.take > 0 && at.take > n_free) status = 1;
            st[b] = status;
            row0[b] = (int)min(at.rows - own.rows, (long long)a.max_rows);
            const long long t = at.take - own.take;
            take0[b] = (int)min(t, n_free);
            give0[b] = (int)min(at.give - own.give, (long long)INT_MAX);
            if (status != 0 && own.take > 0) atomicMin(&take_all, t);
            if (status == 3) atomicMin(&give_all, at.give - own.give);
        }
        __syncthreads();
        if (tid == 0) carry = warp_total[kPlanThreads / 32 - 1];
        __syncthreads();
    }
    const int rows_all = (int)min(carry.rows, (long long)a.max_rows);
    const int taken = (int)min(min(take_all, carry.take), n_free);
    const int given = (int)min(min(give_all, carry.give), room);

    if (first_cta) {
        for (int b = tid; b < a.B; b += kPlanThreads) {
            a.row_start[b] = row0[b];
            a.status[b] = st[b];
            a.kv_len[b] = st[b] == 0 ? __ldg(a.after + b) : 0;
        }
        if (tid == 0) {
            a.row_start[a.B] = rows_all;
            a.free_out[0] = head + taken;
            a.free_out[1] = tail + given;
            if (!ring_ok) atomicOr(a.err, CODEC_LM_ERR_FREE);
        }
    }

    const int t0 = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
    // table entries of the blocks taken
    for (int e = t0; e < taken; e += step) {
        const int b = last_le(take0, a.B, e);
        const int j = a.shared_blocks + owned(__ldg(a.before + b), a.bs_shift, a.shared_blocks) + (e - take0[b]);
        a.tables[(long long)b * a.table_blocks + j] = a.free_list[ring(head_at, e)];
    }
    // blocks given back
    for (int e = t0; e < given; e += step) {
        const int b = last_le(give0, a.B, e);
        const int j = a.shared_blocks + owned(__ldg(a.after + b), a.bs_shift, a.shared_blocks) + (e - give0[b]);
        a.free_list[ring(tail_at, e)] = a.tables[(long long)b * a.table_blocks + j];
    }
    // the shared blocks of requests that start
    if (a.shared_blocks > 0) {
        const long long shared_len = (long long)a.shared_blocks << a.bs_shift;
        for (int b = blockIdx.x * (kPlanThreads / 32) + w; b < a.B; b += gridDim.x * (kPlanThreads / 32)) {
            const int n0 = __ldg(a.before + b);
            if (st[b] != 0 || n0 > shared_len || __ldg(a.after + b) <= n0) continue;
            for (int j = lane; j < a.shared_blocks; j += 32)
                a.tables[(long long)b * a.table_blocks + j] = __ldg(a.shared_table + j);
        }
    }
    // rows, four in a row per thread
    for (long long t4 = 4LL * t0; t4 < a.max_rows; t4 += 4LL * step) {
        int slot[4], pos[4];
        int b = t4 < rows_all ? last_le(row0, a.B, t4) : a.B;
        int n0 = 0, r0 = 0, end = 0, own = 0, status = 0;
        auto request = [&]() {
            n0 = __ldg(a.before + b);
            r0 = row0[b];
            end = b + 1 < a.B ? row0[b + 1] : rows_all;
            own = a.shared_blocks + owned(n0, a.bs_shift, a.shared_blocks);
            status = st[b];
        };
        if (b < a.B) request();
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int t = (int)t4 + i;
            slot[i] = -1;
            pos[i] = 0;
            if (t >= rows_all) continue;
            if (t >= end) {
                b = last_le(row0, a.B, t);
                request();
            }
            pos[i] = n0 + (t - r0);
            if (status != 0) continue;
            const int j = pos[i] >> a.bs_shift;
            int id;
            if (j >= own)
                id = a.free_list[ring(head_at, take0[b] + (j - own))];
            else if (j < a.shared_blocks && n0 <= (a.shared_blocks << a.bs_shift))
                id = __ldg(a.shared_table + j);
            else
                id = a.tables[(long long)b * a.table_blocks + j];
            if (id >= 0 && id < a.n_blocks)
                slot[i] = (id << a.bs_shift) + (pos[i] & ((1 << a.bs_shift) - 1));
            else
                atomicOr(a.err, CODEC_LM_ERR_BLOCK);
        }
        if (vec && t4 + 4 <= a.max_rows) {
            *reinterpret_cast<int4*>(a.slots + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4*>(a.positions + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (t4 + i < a.max_rows) {
                    a.slots[t4 + i] = slot[i];
                    a.positions[t4 + i] = pos[i];
                }
        }
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
    const int vec = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
    return launch_pdl(lm_plan_kernel, dim3(ctas), dim3(kPlanThreads), lm_plan_smem(a.B), s, a, vec);
}

}  // namespace codec
