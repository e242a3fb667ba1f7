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
    const float* row_c = nullptr;   // fp16 queries, each (row, head) with a factor c of its own
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
    float *part, *part_lse;         // [max_requests][max_splits][hq][D], [..][hq]; in 4 bits max_splits_q4 + 1
    float *pre, *pre_lse;           // [pre_max][max_requests][hq][D], [..][hq]
    int* done;                      // [max_requests][hk], zero between calls
    int* taken;                     // the same (behind done)
    int chunk_q4, max_splits_q4;    // chunk and max_splits over the cache in 4 bits
    unsigned char* zeros;           // two tiles of 16 positions in 4 bits that stand for zero
    // A shared part in 4 bits, as halves: at most shared_q4 positions [shared_q4][hk][D],
    // the queries [max_requests][hq][D] and their factors, and the numbers 0, 1, ..;
    // nothing of it where no shared part of the object comes to that (lm_halves_q4)
    int shared_q4;
    void *k16, *v16, *q16;
    float* row_c;
    int* count;
};
constexpr int kLmZeroBytes = 2 * 16 * 128 * 5 / 8;
constexpr int kLmSharedQ4 = 32768;
// Sets of eight columns that a unit over 4 bits has.
inline int lm_sets_q4(int group) { return group > 8 ? 2 : 1; }
// Whether a shared part of len positions becomes halves: of an object for heads = max_requests
// x kv_heads, by tiles of 16 keys and a unit's columns (both sides measured at the launch).
inline bool lm_halves_q4(int type, int max_requests, long long heads, int group, long long len)
{
    return type == CODEC_LM_BF16 && max_requests > 1 && heads * group / (8 * lm_sets_q4(group)) * (len / 16) > 16384;
}

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

// Single tokens over the cache in 4 bits (keys.k, keys.v: its bytes).
cudaError_t configure_lm_step_q4();
cudaError_t launch_lm_step_q4(const LmShape& sh, const LmStepArgs& a, cudaStream_t s);

struct LmStoreQ4Args {
    const void *k, *v;
    long long ks, vs;               // row strides, elements
    int rows;
    const int* slots;
    long long n_slots;
    int bs_shift;
    void *k_cache, *v_cache;
};
cudaError_t launch_lm_store_q4(const LmShape& sh, const LmStoreQ4Args& a, int in_type, cudaStream_t s);

struct LmLoadQ4Args {
    const void *k_cache, *v_cache;
    const int *src, *dst;
    int n, bs_shift, n_blocks, dst_blocks;
    void *k_dst, *v_dst;
};
cudaError_t launch_lm_load_q4(const LmShape& sh, const LmLoadQ4Args& a, cudaStream_t s);

// Blocks 0 .. n - 1 of table in halves to k16, v16 [n][block][hk][D] (zeros for an id
// out of range), and queries [B][hq][D], bf16, in halves to q16, each
// head times a power of two, with scale log2(e) / that in row_c.
struct LmHalvesArgs {
    const void *k_cache, *v_cache;
    const int* table;
    int n, bs_shift, n_blocks;
    const void* q;
    long long qs;
    int B;
    void *k16, *v16, *q16;
    float* row_c;
};
cudaError_t launch_lm_halves_q4(const LmShape& sh, const LmHalvesArgs& a, cudaStream_t s);
cudaError_t launch_lm_count(int* count, int n, cudaStream_t s);     // 0, 1, .. n - 1

struct LmForkArgs {
    const int *parents, *len;
    int B;
    const int* tables;
    int* tables_out;
    int shared_blocks, table_blocks, bs_shift, n_blocks;
    const int* owners;
    int* owners_out;
    int* free_list;
    const long long* free_in;
    long long* free_out;
    int *kv_len, *status, *copy_src, *copy_dst, *copies;
    unsigned* err;
};
struct LmCompactArgs {
    const int* len;
    int B;
    const int* tables;
    int* tables_out;
    const int* shared_table;
    int* shared_out;
    int shared_blocks, table_blocks, bs_shift, n_blocks;
    const int* owners;
    int* owners_out;
    int* free_list;
    long long* free_out;
    int *copy_src, *copy_dst, *copies;
    int* map;                       // workspace [n_blocks]
    unsigned* err;
};
constexpr int kLmMaxCaches = 256;
struct LmCopyArgs {
    const int *src, *dst, *copies;
    int n, n_caches, n_blocks;
    long long block_bytes;
    unsigned* err;
    void* caches[kLmMaxCaches];
};
cudaError_t configure_lm_pages();
cudaError_t launch_lm_fork(const LmForkArgs& a, cudaStream_t s);
cudaError_t launch_lm_compact(const LmCompactArgs& a, cudaStream_t s);
cudaError_t launch_lm_copy(const LmCopyArgs& a, cudaStream_t s);

// Beam search: the best candidates of a part of a row, its maximum and sum.
constexpr int kLmMaxBeams = 32;
struct LmBeamPart {
    double sum;                     // of 2^(x log2 e - c)
    float top;
    int c;
};
struct LmBeamSpace {
    int parts;                      // that the workspace holds
    LmBeamPart* part;               // [parts]
    uint2* best;                    // [parts][beams]: logit's bits (fp32), token, best first
};
inline int lm_beam_parts(int max_requests) { return max_requests + 152 * 8; }

struct LmBeamArgs {
    const void* logits;
    long long stride;
    int type;
    int groups, beams, vocab;
    const float* sums;
    const int* ended;
    int end_token;
    float* sums_out;
    int *parents, *tokens, *ended_out;
    LmBeamSpace ws;
};
cudaError_t configure_lm_beams();
cudaError_t launch_lm_beams(const LmBeamArgs& a, cudaStream_t s);

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
