// Beam search's selection: log-softmax of each beam's logits, and of each
// group's candidates the best.
//
// Two launches.  The first reads the logits once: a part of a row gives its
// log(sum(exp(x))) and its best `beams` tokens; inside a row the order of
// candidates is that of the logits themselves.  A warp holds 4 KB of a row in
// registers: maxima (packed), sums of 2^(x log2 e - C) with a whole number C, and
// then a search of the lanes' maxima, largest first, for values that belong into
// the list of the best; a lane's values are read once more for it, 64 by the
// whole warp.  The second launch joins the parts and picks among a group's rows by
// sums + x - log(sum), in fp64: lists are sorted, so a thread per list and a
// reduction over their heads for each candidate.
//
// What decides between rows is the logarithm, and sums of exponentials in fp32
// are off by up to kNear.  Where two neighbours of the result (or the last and
// the first left out) come from different rows and lie closer, the logarithms
// of those rows are worked out again to about 1e-9, and the choice is made once more.
#include <climits>

#include "lm.h"

namespace codec {

namespace {

constexpr int kThreads = 256;
// Two rows' errors: of 2^-22 by ex2, 16 additions and a product rounded by 2^-24 of
// at most 20 each.
constexpr float kNear = 6e-6f;
constexpr int kLists = 256;                 // of a group: beams x parts of a row

constexpr int kRowWarps = 4;
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kVectors = 8;                 // of 16 bytes a lane: a chunk of a row is 4 KB

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A row that offers tokens.
__device__ __forceinline__ bool offers(const LmBeamArgs& a, int row)
{
    return __ldg(a.ended + row) == 0 && fabsf(__ldg(a.sums + row)) < INFINITY;
}

// Candidate (value, index): the first before the second.
template <typename V>
__device__ __forceinline__ bool ahead(V x, int i, V y, int j) { return x > y || (x == y && i < j); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The values of 16 bytes.
template <typename T> struct Vector;
template <> struct Vector<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float top(uint4 v)
    {
        return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ void get(uint4 v, float* x)
    {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
};
template <> struct Vector<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
    static __device__ __forceinline__ float top(uint4 v)
    {
        const float2 f = __bfloat1622float2(__hmax2_nan(__hmax2_nan(two(v.x), two(v.y)), __hmax2_nan(two(v.z), two(v.w))));
        return max_nan(f.x, f.y);
    }
    static __device__ __forceinline__ void get(uint4 v, float* x)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Vector<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ __half2 two(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
    static __device__ __forceinline__ float top(uint4 v)
    {
        const float2 f = __half22float2(__hmax2_nan(__hmax2_nan(two(v.x), two(v.y)), __hmax2_nan(two(v.z), two(v.w))));
        return max_nan(f.x, f.y);
    }
    static __device__ __forceinline__ void get(uint4 v, float* x)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = __half22float2(two(w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <typename T> __device__ __forceinline__ T minus_infinity();
template <> __device__ __forceinline__ float minus_infinity() { return -INFINITY; }
template <> __device__ __forceinline__ __half minus_infinity() { return __ushort_as_half(0xfc00); }
template <> __device__ __forceinline__ __nv_bfloat16 minus_infinity() { return __ushort_as_bfloat16(0xff80); }

// A float as a whole number of the same order (not NaN).
__device__ __forceinline__ int ordered(float x)
{
    const int i = __float_as_int(x);
    return i >= 0 ? i : i ^ 0x7fffffff;
}

// Row blockIdx.x, part blockIdx.y of it: the chunks of which a warp takes every
// kRowWarps-th.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) lm_beam_rows_kernel(const LmBeamArgs a)
{
    using V = Vector<T>;
    constexpr int kChunk = kVectors * 32 * V::N;
    constexpr float kLog2e = 1.4426950408889634f;
    __shared__ float list_x[kRowThreads];
    __shared__ int list_i[kRowThreads];
    __shared__ double part_l[kRowWarps];
    __shared__ float part_top[kRowWarps];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.beams;
    pdl_wait();
    pdl_launch();
    if (!offers(a, row)) return;
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    // vectors lie on 16 bytes: the first starts `lead` values before the row
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int end = lead + a.vocab, chunks = (end + kChunk - 1) / kChunk;
    const int each = (chunks + gridDim.y - 1) / gridDim.y;
    const int last = min(chunks, ((int)blockIdx.y + 1) * each);
    const T* base = x - lead;

    float best_x = -INFINITY;                   // lane i < K: the i-th best
    int best_i = INT_MAX;
    float least = -INFINITY;                    // the K-th
    int least_i = INT_MAX;
    float top = -INFINITY, hi = 0.f, lo = 0.f;  // of the warp; this lane's sum
    int C = INT_MIN;
    bool bad = false;
    for (int c = blockIdx.y * each + warp; c < last; c += kRowWarps) {
        const int v0 = c * kChunk + lane * V::N;
        uint4 raw[kVectors];
        if (c * kChunk >= lead && (c + 1) * kChunk <= end) {
#pragma unroll
            for (int i = 0; i < kVectors; i++)
                raw[i] = __ldg(reinterpret_cast<const uint4*>(base + v0 + i * 32 * V::N));
        } else {
#pragma unroll
            for (int i = 0; i < kVectors; i++) {
                alignas(16) T e[V::N];
#pragma unroll
                for (int j = 0; j < V::N; j++) {
                    const int v = v0 + i * 32 * V::N + j;
                    e[j] = v >= lead && v < end ? base[v] : minus_infinity<T>();
                }
                raw[i] = *reinterpret_cast<const uint4*>(e);
            }
        }
        float mine = V::top(raw[0]);
#pragma unroll
        for (int i = 1; i < kVectors; i++) mine = max_nan(mine, V::top(raw[i]));
        bad |= !(mine < INFINITY);
        if (__any_sync(0xffffffffu, bad)) break;
        const int key = ordered(mine), most = __reduce_max_sync(0xffffffffu, key);
        const float chunk_top = __int_as_float(most >= 0 ? most : most ^ 0x7fffffff);
        if (chunk_top == -INFINITY) continue;
        if (chunk_top > top) {
            top = chunk_top;
            const int now = (int)ceilf(top * kLog2e);
            const float f = C == INT_MIN ? 0.f : C - now < -126 ? 0.f : __int_as_float((127 + C - now) << 23);
            hi *= f;
            lo *= f;
            C = now;
        }
        const float minus_c = -(float)C;
        float sum[4] = {};
#pragma unroll
        for (int i = 0; i < kVectors; i++) {
            float y[V::N];
            V::get(raw[i], y);
#pragma unroll
            for (int j = 0; j < V::N; j++) sum[j & 3] += exp2_fast(fmaf(y[j], kLog2e, minus_c));
        }
        // added with the rounding error kept
        const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]), t = __fadd_rn(hi, s), b = __fsub_rn(t, hi);
        lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(s, b));
        hi = t;
        // lanes with values that belong into the list, the largest first (equal ones
        // only where a value may come before those of the list)
        int pending = key;
        for (int lanes = 0; lanes < 32; lanes++) {
            const int k = __reduce_max_sync(0xffffffffu, pending);
            const float y = __int_as_float(k >= 0 ? k : k ^ 0x7fffffff);
            if (y == -INFINITY || y < least || (y == least && c * kChunk - lead > least_i)) break;
            const int from = __ffs(__ballot_sync(0xffffffffu, pending == k)) - 1;
            if (lane == from) pending = INT_MIN;
            // its values: V::N / 4 for each lane
            constexpr int kE = V::N / 4;
            const int at = c * kChunk + ((lane >> 2) * 32 + from) * V::N + (lane & 3) * kE;
#pragma unroll
            for (int j = 0; j < kE; j++) {
                const int v = at + j;
                const float z = v >= lead && v < end ? to_float(base[v]) : -INFINITY;
                unsigned in = __ballot_sync(0xffffffffu, z > -INFINITY && ahead(z, v - lead, least, least_i));
                while (in) {
                    const int who = __ffs(in) - 1;
                    in &= in - 1;
                    const float nx = __shfl_sync(0xffffffffu, z, who);
                    const int ni = __shfl_sync(0xffffffffu, v - lead, who);
                    const unsigned before = __ballot_sync(0xffffffffu, ahead(best_x, best_i, nx, ni));
                    const float ux = __shfl_up_sync(0xffffffffu, best_x, 1);
                    const int ui = __shfl_up_sync(0xffffffffu, best_i, 1);
                    const int place = __popc(before);
                    if (lane > place) {
                        best_x = ux;
                        best_i = ui;
                    } else if (lane == place) {
                        best_x = nx;
                        best_i = ni;
                    }
                }
                least = __shfl_sync(0xffffffffu, best_x, K - 1);
                least_i = __shfl_sync(0xffffffffu, best_i, K - 1);
            }
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    list_x[tid] = lane < K ? best_x : -INFINITY;
    list_i[tid] = lane < K ? best_i : INT_MAX;
    double l = (double)hi + (double)lo;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
        // kLog2e is 1.33e-8 of itself too small
        part_l[warp] = top == -INFINITY ? -INFINITY : ((double)C + log2(l)) * 0.6931471805599453 + 1.3349623e-8 * (double)top;
        part_top[warp] = bad ? NAN : top;
    }
    __syncthreads();
    const long long at = (long long)row * gridDim.y + blockIdx.y;
    // the warps' lists: a value's place is the number of those before it
    const float mx = list_x[tid];
    const int mi = list_i[tid];
    if (lane < K && mx > -INFINITY) {
        int place = 0;
        for (int w = 0; w < kRowWarps; w++)
            for (int j = 0; j < K; j++) place += ahead(list_x[w * 32 + j], list_i[w * 32 + j], mx, mi);
        if (place < K) a.ws.best[at * K + place] = make_uint2(__float_as_uint(mx), (unsigned)mi);
    }
    // places that nothing takes
    const int there = __syncthreads_count(lane < K && mx > -INFINITY);
    if (tid >= there && tid < K) a.ws.best[at * K + tid] = make_uint2(__float_as_uint(-INFINITY), (unsigned)INT_MAX);
    if (tid == 0) {
        float m = part_top[0];
        for (int w = 1; w < kRowWarps; w++) m = max_nan(m, part_top[w]);
        double sum = 0., most = part_l[0];
        for (int w = 1; w < kRowWarps; w++) most = fmax(most, part_l[w]);
        if (most > -INFINITY)
            for (int w = 0; w < kRowWarps; w++) sum += exp(part_l[w] - most);
        a.ws.part[at] = LmBeamPart{most > -INFINITY ? most + log(sum) : most, m, 0};
    }
}

// log(sum(exp(x))) of a row to about 1e-9, by the whole CTA.  exp(d) = 2^k 2^(j / 64)
// (1 + p): the power of two of the table in two floats, p a short series of what
// is left (at most ln 2 / 128), terms added with their rounding errors kept.
template <typename T>
__device__ double exact_log_sum(const T* x, int n, float top, const float2* table, double* sm)
{
    constexpr float kInv = 92.332482616893656f;             // 64 / ln 2
    constexpr float kHi = 0x1.62cp-7f;                      // ln 2 / 64: 11 bits, and the rest
    const float lo = (float)(0.010830424696249145 - (double)kHi);
    const int tid = threadIdx.x;
    float s = 0.f, c = 0.f;
    for (int v = tid; v < n; v += kThreads) {
        const float y = to_float(x[v]);
        const float d = __fsub_rn(y, top);
        if (!(d > -80.f)) continue;                         // nothing beside the maximum's 1
        const float u = __fsub_rn(d, y), w = __fsub_rn(d, u);
        const float e = __fadd_rn(__fsub_rn(y, w), __fsub_rn(-top, u));     // what d was rounded by
        const float m = rintf(d * kInv);
        const float r = fmaf(-m, lo, fmaf(-m, kHi, d)) + e;
        const float p = r * fmaf(r, fmaf(r, fmaf(r, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f);
        const int im = (int)m;
        const float scale = __int_as_float(((im >> 6) + 127) << 23);
        const float2 t = table[im & 63];
        const float h = t.x * scale, l = fmaf(t.x, p, t.y) * scale;
        const float now = __fadd_rn(s, h), b = __fsub_rn(now, s);
        c += __fadd_rn(__fsub_rn(s, __fsub_rn(now, b)), __fsub_rn(h, b)) + l;
        s = now;
    }
    double sum = (double)s + (double)c;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if ((tid & 31) == 0) sm[tid >> 5] = sum;
    __syncthreads();
    sum = 0.;
    for (int w = 0; w < kThreads / 32; w++) sum += sm[w];
    return (double)top + log(sum);
}

// One group.  Dynamic shared memory: the lists, [K x parts][K].
template <typename T>
__global__ void __launch_bounds__(kThreads) lm_beam_pick_kernel(const LmBeamArgs a, int parts)
{
    extern __shared__ uint2 list[];
    __shared__ double base[kLmMaxBeams];        // sums - log(sum(exp)), or the sum of an ended beam
    __shared__ float top[kLmMaxBeams];
    __shared__ int kind[kLmMaxBeams];           // 0: offers nothing, 1: tokens, 2: itself
    __shared__ double ws[2][kThreads / 32], sums[kThreads / 32], got[kLmMaxBeams + 1];
    __shared__ int wi[2][kThreads / 32], got_i[kLmMaxBeams + 1];
    __shared__ float2 table[64];
    __shared__ unsigned again;
    const int K = a.beams, row0 = blockIdx.x * K, lists = K * parts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch();
    for (int e = tid; e < lists * K; e += kThreads) list[e] = __ldcg(a.ws.best + (long long)row0 * parts * K + e);
    for (int r = warp; r < K; r += kThreads / 32) {
        const int row = row0 + r;
        const float sum = __ldg(a.sums + row);
        const bool there = fabsf(sum) < INFINITY, end = __ldg(a.ended + row) != 0;
        double l = 0.;
        float m = -INFINITY;
        if (there && !end) {
            double most = -INFINITY;
            for (int i = lane; i < parts; i += 32) {
                const LmBeamPart* p = a.ws.part + (long long)row * parts + i;
                m = max_nan(m, __ldcg(&p->top));
                most = fmax(most, __ldcg(&p->lse));
            }
            for (int o = 16; o > 0; o >>= 1) {
                m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                most = fmax(most, __shfl_xor_sync(0xffffffffu, most, o));
            }
            if (fabsf(m) < INFINITY) {
                for (int i = lane; i < parts; i += 32) l += exp(__ldcg(&a.ws.part[(long long)row * parts + i].lse) - most);
                for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                l = most + log(l);
            }
        }
        if (lane == 0) {
            top[r] = m;
            kind[r] = !there ? 0 : end ? 2 : fabsf(m) < INFINITY ? 1 : 0;
            base[r] = end ? (double)sum : (double)sum - l;
        }
    }
    if (tid == 0) again = 0;
    __syncthreads();
    // this thread's list: its row, and its head's score and index (row of the group, token)
    const int r = min(tid / parts, K - 1);
    int at = 0;
    double s = -INFINITY;
    int i = INT_MAX;
    auto head = [&]() {
        s = -INFINITY;
        i = INT_MAX;
        if (tid >= lists || at == K) return;
        if (kind[r] == 1) {
            const uint2 c = list[tid * K + at];
            const float x = __uint_as_float(c.x);
            if (x > -INFINITY) {
                s = base[r] + (double)x;
                i = r * a.vocab + (int)c.y;
            }
        } else if (kind[r] == 2 && tid == r * parts && at == 0) {
            s = base[r];
            i = r * a.vocab + max(a.end_token, 0);
        }
    };
    for (int round = 0; round < 2; round++) {
        at = 0;
        head();
        // one more than are wanted, to see how near it is
        for (int k = 0; k <= K; k++) {
            double best = s;
            int best_i = i;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const double y = __shfl_xor_sync(0xffffffffu, best, o);
                const int j = __shfl_xor_sync(0xffffffffu, best_i, o);
                if (ahead(y, j, best, best_i)) {
                    best = y;
                    best_i = j;
                }
            }
            if (lane == 0) {
                ws[k & 1][warp] = best;
                wi[k & 1][warp] = best_i;
            }
            __syncthreads();                    // two sets: the next round writes the other
            best = ws[k & 1][0];
            best_i = wi[k & 1][0];
#pragma unroll
            for (int w = 1; w < kThreads / 32; w++)
                if (ahead(ws[k & 1][w], wi[k & 1][w], best, best_i)) {
                    best = ws[k & 1][w];
                    best_i = wi[k & 1][w];
                }
            if (tid == 0) {
                got[k] = best;
                got_i[k] = best_i;
            }
            if (i == best_i && i != INT_MAX) {
                at++;
                head();
            }
        }
        __syncthreads();
        if (round == 1) break;
        if (tid < K && got_i[tid + 1] != INT_MAX) {
            const int p = got_i[tid] / a.vocab, q = got_i[tid + 1] / a.vocab;
            if (p != q && got[tid] - got[tid + 1] < kNear) atomicOr(&again, 1u << p | 1u << q);
        }
        __syncthreads();
        if (again == 0) break;
        // and all that lie as near to the last one
        for (int e = tid; e < lists * K; e += kThreads) {
            const int row = e / K / parts;
            if (kind[row] == 1 && fabs(base[row] + (double)__uint_as_float(list[e].x) - got[K - 1]) < kNear)
                atomicOr(&again, 1u << row);
        }
        if (tid < 64) {
            const double t = exp2(tid / 64.);
            table[tid] = make_float2((float)t, (float)(t - (double)(float)t));
        }
        __syncthreads();
        for (int q = 0; q < K; q++)
            if (again >> q & 1 && kind[q] == 1) {
                const double l = exact_log_sum(static_cast<const T*>(a.logits) + (row0 + q) * a.stride, a.vocab, top[q],
                                               table, sums);
                if (tid == 0) base[q] = (double)__ldg(a.sums + row0 + q) - l;
            }
        __syncthreads();
    }
    if (tid < K) {
        const int c = got_i[tid], row = row0 + tid;
        const bool there = c != INT_MAX;
        const int p = there ? c / a.vocab : 0, token = there ? c - p * a.vocab : -1;
        const bool itself = there && kind[p] == 2;
        a.sums_out[row] = there ? itself ? __ldg(a.sums + row0 + p) : (float)got[tid] : -INFINITY;
        a.parents[row] = there ? row0 + p : -1;
        a.tokens[row] = itself ? a.end_token : token;
        a.ended_out[row] = !there || itself || token == a.end_token;
    }
}

template <typename T>
cudaError_t launch(const LmBeamArgs& a, cudaStream_t s)
{
    // parts of a row: about eight CTAs per SM, a chunk for each warp at least, and lists
    // for the second kernel's threads
    const int rows = a.groups * a.beams;
    const long long chunks = (a.vocab * (long long)sizeof(T) + 4095) / 4096;
    const int parts = (int)std::max<long long>(1, std::min<long long>({152 * 8 / rows, chunks / kRowWarps, kLists / a.beams}));
    const cudaError_t e = launch_pdl(lm_beam_rows_kernel<T>, dim3(rows, parts), dim3(kRowThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(lm_beam_pick_kernel<T>, dim3(a.groups), dim3(kThreads), sizeof(uint2) * a.beams * parts * a.beams, s, a,
                      parts);
}

template <typename T>
cudaError_t configure()
{
    return cudaFuncSetAttribute(lm_beam_pick_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(uint2) * kLists * kLmMaxBeams);
}

}  // namespace

cudaError_t configure_lm_beams()
{
    for (const cudaError_t e : {configure<float>(), configure<__half>(), configure<__nv_bfloat16>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

cudaError_t launch_lm_beams(const LmBeamArgs& a, cudaStream_t s)
{
    return a.type == CODEC_LM_FP32   ? launch<float>(a, s)
           : a.type == CODEC_LM_BF16 ? launch<__nv_bfloat16>(a, s)
                                     : launch<__half>(a, s);
}

}  // namespace codec
