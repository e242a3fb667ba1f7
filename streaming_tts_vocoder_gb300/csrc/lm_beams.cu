// Beam search's selection: log-softmax of each beam's logits, and of each
// group's candidates the best.
//
// Two launches.  The first reads the logits once: a part of a row gives its
// maximum m, the sum of exp(x - m) and its best `beams` tokens; inside a row the
// order of candidates is that of the logits themselves.  The second joins the
// parts and picks among a group's rows by sums + x - log(sum), in fp64.
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
constexpr float kNear = 3e-6f;

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

template <typename T>
__global__ void __launch_bounds__(kThreads) lm_beam_rows_kernel(const LmBeamArgs a)
{
    __shared__ float wx[kThreads / 32];
    __shared__ int wi[kThreads / 32];
    __shared__ double ws[kThreads / 32];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch();
    if (!offers(a, row)) return;
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    float last = INFINITY, top = 0.f;
    int last_i = -1;
    bool bad = false;
    for (int k = 0; k < a.beams; k++) {
        float best = -INFINITY;
        int at = INT_MAX;
        for (int v = tid; v < a.vocab; v += kThreads) {
            const float y = to_float(x[v]);
            bad |= !(y < INFINITY);
            if (ahead(last, last_i, y, v) && ahead(y, v, best, at)) {
                best = y;
                at = v;
            }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, best, o);
            const int j = __shfl_xor_sync(0xffffffffu, at, o);
            if (ahead(y, j, best, at)) {
                best = y;
                at = j;
            }
        }
        const bool any = __syncthreads_or(bad);
        if (lane == 0) {
            wx[warp] = best;
            wi[warp] = at;
        }
        __syncthreads();
        best = wx[0];
        at = wi[0];
        for (int w = 1; w < kThreads / 32; w++)
            if (ahead(wx[w], wi[w], best, at)) {
                best = wx[w];
                at = wi[w];
            }
        if (k == 0) {
            top = any ? NAN : best;
            if (!(fabsf(top) < INFINITY)) {
                if (tid == 0) a.ws.part[row] = LmBeamPart{0., top, 0};
                return;
            }
        }
        if (tid == 0) a.ws.best[(long long)row * a.beams + k] = make_uint2(__float_as_uint(best), (unsigned)at);
        last = best;
        last_i = at;
    }
    double sum = 0.;
    for (int v = tid; v < a.vocab; v += kThreads) sum += expf(to_float(x[v]) - top);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) ws[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kThreads / 32; w++) sum += ws[w];
        a.ws.part[row] = LmBeamPart{sum, top, 0};
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

template <typename T>
__global__ void __launch_bounds__(kThreads) lm_beam_pick_kernel(const LmBeamArgs a, int parts)
{
    __shared__ double base[kLmMaxBeams];        // sums - log(sum(exp)), or the sum of an ended beam
    __shared__ float top[kLmMaxBeams];
    __shared__ int kind[kLmMaxBeams];           // 0: offers nothing, 1: tokens, 2: itself
    __shared__ double ws[kThreads / 32], got[kLmMaxBeams + 1];
    __shared__ int wi[kThreads / 32], got_i[kLmMaxBeams + 1];
    __shared__ float2 table[64];
    __shared__ unsigned again;
    const int K = a.beams, row0 = blockIdx.x * K;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch();
    for (int r = warp; r < K; r += kThreads / 32) {
        const int row = row0 + r;
        const float sum = __ldg(a.sums + row);
        const bool there = fabsf(sum) < INFINITY, end = __ldg(a.ended + row) != 0;
        double l = 0.;
        float m = -INFINITY;
        if (there && !end) {
            bool nan = false;
            for (int i = lane; i < parts; i += 32) {
                const float y = a.ws.part[(long long)row * parts + i].top;
                nan |= y != y;
                m = fmaxf(m, y);
            }
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (__any_sync(0xffffffffu, nan)) m = NAN;
            if (fabsf(m) < INFINITY) {
                for (int i = lane; i < parts; i += 32) {
                    const LmBeamPart p = a.ws.part[(long long)row * parts + i];
                    if (p.top > -INFINITY) l += p.top == m ? p.sum : p.sum * exp((double)p.top - (double)m);
                }
                for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            }
        }
        if (lane == 0) {
            top[r] = m;
            kind[r] = !there ? 0 : end ? 2 : fabsf(m) < INFINITY ? 1 : 0;
            base[r] = end ? (double)sum : (double)sum - ((double)m + log(l));
        }
    }
    if (tid == 0) again = 0;
    __syncthreads();
    const int lists = K * parts, n = lists * K;
    // candidate e: its score and index (row of the group, token); false: there is none
    auto candidate = [&](int e, double& s, int& i) {
        if (e < n) {
            const int r = e / K / parts;
            if (kind[r] != 1) return false;
            const uint2 c = __ldcg(a.ws.best + (long long)row0 * parts * K + e);
            const float x = __uint_as_float(c.x);
            s = base[r] + (double)x;
            i = r * a.vocab + (int)c.y;
            return x > -INFINITY;
        }
        const int r = e - n;
        s = base[r];
        i = r * a.vocab + max(a.end_token, 0);
        return kind[r] == 2;
    };
    for (int round = 0; round < 2; round++) {
        double last = INFINITY;
        int last_i = -1;
        // one more than are wanted, to see how near it is
        for (int k = 0; k <= K; k++) {
            double best = -INFINITY;
            int at = INT_MAX;
            for (int e = tid; e < n + K; e += kThreads) {
                double s;
                int i;
                if (!candidate(e, s, i)) continue;
                if (ahead(last, last_i, s, i) && ahead(s, i, best, at)) {
                    best = s;
                    at = i;
                }
            }
            for (int o = 16; o > 0; o >>= 1) {
                const double y = __shfl_xor_sync(0xffffffffu, best, o);
                const int j = __shfl_xor_sync(0xffffffffu, at, o);
                if (ahead(y, j, best, at)) {
                    best = y;
                    at = j;
                }
            }
            __syncthreads();
            if (lane == 0) {
                ws[warp] = best;
                wi[warp] = at;
            }
            __syncthreads();
            best = ws[0];
            at = wi[0];
            for (int w = 1; w < kThreads / 32; w++)
                if (ahead(ws[w], wi[w], best, at)) {
                    best = ws[w];
                    at = wi[w];
                }
            if (tid == 0) {
                got[k] = best;
                got_i[k] = at;
            }
            last = best;
            last_i = at;
        }
        __syncthreads();
        if (round == 1) break;
        if (tid < K && got_i[tid + 1] != INT_MAX) {
            const int r = got_i[tid] / a.vocab, o = got_i[tid + 1] / a.vocab;
            if (r != o && got[tid] - got[tid + 1] < kNear) atomicOr(&again, 1u << r | 1u << o);
        }
        __syncthreads();
        if (again == 0) break;
        // and all that lie as near to the last one
        for (int e = tid; e < n; e += kThreads) {
            double s;
            int i;
            if (candidate(e, s, i) && fabs(s - got[K - 1]) < kNear) atomicOr(&again, 1u << i / a.vocab);
        }
        if (tid < 64) {
            const double t = exp2(tid / 64.);
            table[tid] = make_float2((float)t, (float)(t - (double)(float)t));
        }
        __syncthreads();
        for (int r = 0; r < K; r++)
            if (again >> r & 1 && kind[r] == 1) {
                const double l = exact_log_sum(static_cast<const T*>(a.logits) + (row0 + r) * a.stride, a.vocab,
                                               top[r], table, ws);
                if (tid == 0) base[r] = (double)__ldg(a.sums + row0 + r) - l;
            }
        __syncthreads();
    }
    if (tid < K) {
        const int i = got_i[tid], row = row0 + tid;
        const bool there = i != INT_MAX;
        const int r = there ? i / a.vocab : 0, token = there ? i - r * a.vocab : -1;
        const bool itself = there && kind[r] == 2;
        a.sums_out[row] = there ? itself ? __ldg(a.sums + row0 + r) : (float)got[tid] : -INFINITY;
        a.parents[row] = there ? row0 + r : -1;
        a.tokens[row] = itself ? a.end_token : token;
        a.ended_out[row] = !there || itself || token == a.end_token;
    }
}

template <typename T>
cudaError_t launch(const LmBeamArgs& a, cudaStream_t s)
{
    const cudaError_t e = launch_pdl(lm_beam_rows_kernel<T>, dim3(a.groups * a.beams), dim3(kThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(lm_beam_pick_kernel<T>, dim3(a.groups), dim3(kThreads), 0, s, a, 1);
}

}  // namespace

cudaError_t launch_lm_beams(const LmBeamArgs& a, cudaStream_t s)
{
    return a.type == CODEC_LM_FP32   ? launch<float>(a, s)
           : a.type == CODEC_LM_BF16 ? launch<__nv_bfloat16>(a, s)
                                     : launch<__half>(a, s);
}

}  // namespace codec
