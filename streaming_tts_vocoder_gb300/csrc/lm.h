// Internal launchers of the codec LM's attention operators (lm_*.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "codec.h"
#include "common.cuh"

namespace codec {

// Rows of requests and where their keys and values are.  Packed: K/V rows of
// request b are row_start[b] ..; paged: position p is in block
// tables[b][p / bs] of the cache.
struct LmKeys {
    const void* k;
    const void* v;
    long long k_stride, v_stride;   // packed: elements between rows
    const int* tables;              // paged: [B][table_blocks]; null: packed
    const int* kv_len;              // paged: [B]
    int table_blocks;
    int bs_shift;                   // log2(block_size)
    int n_blocks;
};

struct LmShape {
    int type;                       // CODEC_LM_BF16 / CODEC_LM_FP16
    int hq, hk, group, D;
    float scale;
    unsigned* err;
    unsigned unarrived;             // != 0: one warp per CTA waits so many polls for a barrier that nothing arrives on
};
// Polls of a wait before it gives up: 1.5 us each where nothing arrives; the longest
// table, 2^18 tiles of 128 keys, takes 0.4 s.  A constant: as a kernel argument it
// made prompts of 6,904 and 9,000 tokens 688 us instead of 654.
constexpr unsigned kLmPolls = 1u << 20;

struct LmPlanArgs {
    const int* before;
    const int* after;
    int B;
    int* tables;
    const int* shared_table;
    int shared_blocks;
    int table_blocks, bs_shift, n_blocks;
    int* free_list;
    const long long* free_in;
    long long* free_out;
    int *row_start, *kv_len, *status, *slots, *positions;
    int max_rows;
    unsigned* err;
};
size_t lm_plan_smem(int B);
constexpr int kLmMaxRequests = 4096;
cudaError_t configure_lm_plan();
cudaError_t launch_lm_plan(const LmPlanArgs& a, cudaStream_t s);

struct LmRotateArgs {
    const void *q, *k, *v;
    long long qs, ks, vs;           // row strides, elements
    int rows;
    const float *q_gain, *k_gain;
    const int *positions, *slots;
    long long n_slots;
    void *q_out, *k_dst, *v_dst;
    const float2* turn;             // [max_positions][D / 2] cos, sin
    int max_positions;
    float eps;
    int pairs;
};
cudaError_t launch_lm_rotate(const LmShape& sh, const LmRotateArgs& a, int in_type, cudaStream_t s);
cudaError_t launch_lm_turn_table(float2* turn, int max_positions, int D, double theta, cudaStream_t s);

// Workspace of prompt attention.
constexpr int kLmSlots = 256;       // pieces of items that are cut, with their K/V heads
struct LmPromptSpace {
    void* list;                     // [items + kLmSlots] x 32 bytes
    int* counts;                    // [3]
    void* joins;                    // [kLmSlots] x 16 bytes
    float *piece, *piece_lse;       // [kLmSlots][256][D], [kLmSlots][256]
};

struct LmPromptArgs {
    const void* q;
    long long qs;
    int rows;
    const int* row_start;
    int B;
    LmKeys keys;
    void* o;
    long long os;
    float* lse;
    LmPromptSpace ws;
};
// Pairs of query tiles that `rows` rows of at most B requests can make.
__host__ __device__ inline long long lm_list_items(int rows, int B, int group)
{
    return rows / (2 * (128 / group)) + (rows < B ? rows : B);
}
cudaError_t configure_lm_prompt();
cudaError_t launch_lm_prompt(const LmShape& sh, const LmPromptArgs& a, cudaStream_t s);

// Single tokens over a part of the context that all requests share: partial
// results of splits of split_len positions, [split][B][hq][D] and [split][B][hq].
struct LmSharedArgs {
    const void* q;
    long long qs;
    int B;
    LmKeys keys;                    // tables unused
    const int* shared_table;
    int shared_len, split_len;
    float* part;
    float* part_lse;
};
long long lm_shared_ctas(const LmShape& sh, const LmSharedArgs& a);
cudaError_t launch_lm_shared(const LmShape& sh, const LmSharedArgs& a, cudaStream_t s);

// Workspace of single-token attention.
// Splits of a shared part of `len` positions whose every split takes `ctas`: 256
// positions at least while all of them make at most 64 CTAs (the rest of the SMs
// stream the requests' own parts meanwhile), 128 while they make at most 32.
// 64 CTAs of one tile each: 1,024 positions, 8 heads 23.5 us, 32 of two 18.8.
inline int lm_shared_splits(long long ctas, long long len)
{
    const long long wide = std::min<long long>({32, 64 / ctas, len / 256}), narrow = std::min<long long>({8, 32 / ctas, len / 128});
    return (int)std::max<long long>({1, wide, narrow});
}
struct LmStepSpace {
    int chunk;                      // positions per split of a request's own part
    int max_splits;                 // splits of a full table
    int shared_ctas;                // of each split of the shared part, with max_requests
    long long heads;                // max_requests x kv_heads
    float *part, *part_lse;         // [max_requests][max_splits][hq][D], [..][hq]
    float *pre, *pre_lse;           // [pre_max][max_requests][hq][D], [..][hq]
    int* done;                      // [max_requests][hk], zero between calls
    int* taken;                     // the same (behind done)
};

struct LmStepArgs {
    const void* q;
    long long qs;
    int B;
    LmKeys keys;
    const int* shared_table;
    int shared_blocks;
    void* o;
    long long os;
    float* lse;
    LmStepSpace ws;
};
cudaError_t configure_lm_step();
cudaError_t launch_lm_step(const LmShape& sh, const LmStepArgs& a, cudaStream_t s);

// Tensor map of [rows][heads][D] 16-bit values, rows `stride` elements apart,
// boxes of 64 elements x box_heads x box_rows.
bool lm_make_map(CUtensorMap* map, int type, const void* base, int D, int heads, long long rows, long long stride,
                 int box_heads, int box_rows);

// Rows of request b, from a row_start that is device data: inside [0, rows]
// and never negative in number.  False: it was not, and was bent to fit.
__device__ __forceinline__ bool lm_rows(const int* row_start, int b, int rows, int& first, int& n)
{
    const int a = __ldg(row_start + b), e = __ldg(row_start + b + 1);
    first = min(max(a, 0), rows);
    const int end = min(max(e, first), rows);
    n = end - first;
    return first == a && end == e;
}

__device__ __forceinline__ bool lm_clamp_len(int& n, long long most)
{
    const int want = n;
    n = (int)min(max((long long)n, 0LL), most);
    return n == want;
}

}  // namespace codec
