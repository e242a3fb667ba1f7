// The codec LM's attention operators: object, argument checks, launches.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <new>

#include "lm.h"

using namespace codec;

struct codec_lm_s {
    codec_lm_config cfg{};
    int device = 0;
    int bs_shift = 0;
    LmShape shape{};
    float2* turn = nullptr;
    unsigned* err = nullptr;
    LmStepSpace step{};
    LmPromptSpace prompt{};
    LmBeamSpace beam{};
    int* block_map = nullptr;
};

namespace {

// Calls run on the object's device, whichever is current.  It is set even where it
// is current already: that binds its context to a host thread that has made no CUDA
// call yet, and the driver encodes no tensor map without one.
struct OnDevice {
    int was = -1;
    bool ok = false;
    explicit OnDevice(int device)
    {
        if (cudaGetDevice(&was) != cudaSuccess) return;
        ok = cudaSetDevice(device) == cudaSuccess;
        if (was == device) was = -1;
    }
    ~OnDevice()
    {
        if (was >= 0) cudaSetDevice(was);
    }
};

void lm_free(codec_lm_s* lm)
{
    cudaFree(lm->turn);
    cudaFree(lm->err);
    cudaFree(lm->step.part);
    cudaFree(lm->step.part_lse);
    cudaFree(lm->step.pre);
    cudaFree(lm->step.pre_lse);
    cudaFree(lm->step.done);
    cudaFree(lm->step.zeros);
    cudaFree(lm->step.k16);
    cudaFree(lm->step.v16);
    cudaFree(lm->step.q16);
    cudaFree(lm->step.row_c);
    cudaFree(lm->step.count);
    cudaFree(lm->prompt.list);
    cudaFree(lm->prompt.counts);
    cudaFree(lm->prompt.joins);
    cudaFree(lm->prompt.piece);
    cudaFree(lm->prompt.piece_lse);
    cudaFree(lm->beam.part);
    cudaFree(lm->beam.best);
    cudaFree(lm->block_map);
    delete lm;
}

// Each output an array of its own.
bool apart(std::initializer_list<const void*> outputs, std::initializer_list<const void*> inputs)
{
    for (const void* const* o = outputs.begin(); o != outputs.end(); o++) {
        if (!*o) continue;
        if (std::find(o + 1, outputs.end(), *o) != outputs.end()) return false;
        if (std::find(inputs.begin(), inputs.end(), *o) != inputs.end()) return false;
    }
    return true;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Rows of `n` elements of `size` bytes, stride elements apart, that 16-byte accesses can walk.
bool row_ok(const void* p, int64_t stride, int64_t n, int size)
{
    return aligned16(p) && stride >= n && stride <= (1LL << 32) && stride * size % 16 == 0;
}

codec_status done(cudaError_t e) { return e == cudaSuccess ? CODEC_OK : CODEC_ERR_CUDA; }

LmKeys paged(const codec_lm_s* lm, const void* k, const void* v, const int32_t* tables, const int32_t* kv_len)
{
    return LmKeys{k, v, 0, 0, tables, kv_len, lm->cfg.table_blocks, lm->bs_shift, lm->cfg.n_blocks};
}

}  // namespace

codec_status codec_lm_create(const codec_lm_config* cfg, codec_lm_t** out)
{
    if (!cfg || !out) return CODEC_ERR_NULL;
    *out = nullptr;
    codec_lm_config c = *cfg;
    if ((c.type != CODEC_LM_BF16 && c.type != CODEC_LM_FP16) || (c.head_dim != 64 && c.head_dim != 128) ||
        c.kv_heads < 1 || c.q_heads < c.kv_heads || c.q_heads > 256 || c.q_heads % c.kv_heads ||
        c.q_heads / c.kv_heads > 16 ||
        (c.block_size != 16 && c.block_size != 32 && c.block_size != 64 && c.block_size != 128) || c.n_blocks < 1 ||
        (int64_t)c.n_blocks * c.block_size >= (1LL << 31) - 128 || c.table_blocks < 1 ||
        (int64_t)c.table_blocks * c.block_size > (1LL << 25) || c.max_requests < 1 || c.max_requests > kLmMaxRequests ||
        c.max_rows < 1 || c.max_rows > (1 << 24) || c.max_positions < 0 || c.max_positions > (1 << 30) ||
        (c.rope_pairs != 0 && c.rope_pairs != 1) || !(c.rope_theta > 1.f) || !std::isfinite(c.rope_theta) ||
        !(c.rms_eps >= 0.f) || !std::isfinite(c.rms_eps) || !(c.scale >= 0.f) || !std::isfinite(c.scale))
        return CODEC_ERR_CONFIG;
    if (c.max_positions == 0) c.max_positions = c.table_blocks * c.block_size;
    if (c.scale == 0.f) c.scale = 1.f / std::sqrt((float)c.head_dim);
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess || major < 10)
        return CODEC_ERR_NO_DEVICE;
    codec_lm_s* lm = new (std::nothrow) codec_lm_s();
    if (!lm) return CODEC_ERR_OOM;
    lm->cfg = c;
    lm->device = dev;
    while ((1 << lm->bs_shift) < c.block_size) lm->bs_shift++;
    // Single tokens: splits of 64 positions, of up to 256 as long as the largest
    // batch over full tables still makes one for every CTA that fits the GPU (304),
    // of up to 512 as long as it makes eight, and of as many as leave a full table
    // 64.  A split costs about 2 us whatever it holds, an idle SM more: 16 requests
    // of 3,000 to 4,000 positions take 47 us in splits of 256 and 52 in 128, 64 of up
    // to 500 behind a shared part 17.5 in 256 and 19 in 512.  Tables of up to 512
    // positions are not split where the requests' heads alone occupy most SMs, and
    // then nothing is joined: 64 requests of 200 to 250 positions 12.7 us, in
    // splits of 64 22.4.
    LmStepSpace& sp = lm->step;
    const int64_t positions = (int64_t)c.table_blocks * c.block_size;
    const int64_t heads = (int64_t)c.max_requests * c.kv_heads;
    sp.chunk = 64;
    if (heads >= 152 && positions <= 512) sp.chunk = 512;
    while ((sp.chunk < 512 && heads * ((positions + 2 * sp.chunk - 1) / (2 * sp.chunk)) >=
                                  (sp.chunk < 256 ? 1 : 8) * 304) ||
           positions > 64LL * sp.chunk ||
           // and the partial results of full tables stay within 2 GB
           (sp.chunk < positions && heads * (c.q_heads / c.kv_heads) * ((positions + sp.chunk - 1) / sp.chunk) *
                                            c.head_dim > (1LL << 29)))
        sp.chunk *= 2;
    sp.max_splits = (int)((positions + sp.chunk - 1) / sp.chunk);
    // In 4 bits a split is one warp's, and 1,824 of them run at once: about as long as
    // makes one for each from full tables, of 32 positions at least and 256 at most (512
    // from 4,096 a warp on), at most 64 of a table, and none where the heads alone
    // occupy three warps an SM and a table makes two.  Requests x positions (16 / 8
    // heads of 128), us with splits of 32, 64, 128, 256, 512: 1 x 700 9.5, 9.5, 11.0, 14.5,
    // 22.0; 1 x 9,000 39.7, 22.5, 18.6, 18.1, 23.5; 16 x 3,000 to 3,750 56.6, 39.0, 29.3,
    // 23.9, 27.2; 64 of 1 to 1,500 (16 / 16 of 64) 24.3, 17.9, 18.5, 17.2, 23.5; 256 of 500
    // to 4,000 (32 / 8) 457, 306, 216, 172, 155; 64 x 250 21.1, 19.7, 15.1, whole 13.5.
    // 256 and 512 by positions a warp: 2,000 (64 of 500 to 7,000, 32 / 8) 62.6, 60.7; 2,260
    // (128 of up to 4,000) 73.5, 76.8; 3,950 (128 of up to 7,000) 102, 92; 4,490 (64 of up to
    // 8,000, 16 / 16 of 64) 87.8, 79.8; 8,430 (64 of up to 30,000) 157 both; 8,980 (256 of up
    // to 8,000) 199, 177.
    const int64_t each = heads * positions / 1824;
    sp.chunk_q4 = 32;
    while ((sp.chunk_q4 < each && sp.chunk_q4 < (each >= 4096 ? 512 : 256)) || positions > 64LL * sp.chunk_q4 ||
           // and the partial results of full tables stay within 2 GB
           (sp.chunk_q4 < positions && heads * (c.q_heads / c.kv_heads) * ((positions + sp.chunk_q4 - 1) / sp.chunk_q4) *
                                               c.head_dim > (1LL << 29)))
        sp.chunk_q4 *= 2;
    if (heads >= 3 * 152 && positions <= 2 * sp.chunk_q4) sp.chunk_q4 *= 2;
    sp.max_splits_q4 = (int)((positions + sp.chunk_q4 - 1) / sp.chunk_q4);
    const size_t most_splits = std::max(sp.max_splits, sp.max_splits_q4 + 1);
    // The shared part's splits: by the largest batch, so that the actual one changes no bits.
    const int tokens = 2 * (128 / (c.q_heads / c.kv_heads));
    const int64_t pairs = (c.max_requests + tokens - 1) / tokens;
    sp.shared_ctas = (int)(pairs * c.kv_heads);
    sp.heads = heads;
    const int pre_max = lm_shared_splits(sp.shared_ctas, positions);
    const bool halves = lm_halves_q4(c.type, c.max_requests, heads, c.q_heads / c.kv_heads, positions);
    sp.shared_q4 = halves ? (int)std::min<int64_t>(positions, kLmSharedQ4) : 0;
    LmBeamSpace& bm = lm->beam;
    bm.parts = lm_beam_parts(c.max_requests);
    LmPromptSpace& pr = lm->prompt;
    const size_t items = (size_t)lm_list_items(c.max_rows, c.max_requests, c.q_heads / c.kv_heads) + kLmSlots;
    const size_t row = (size_t)c.max_requests * c.q_heads;
    if (cudaMalloc(&lm->turn, sizeof(float2) * (size_t)c.max_positions * (c.head_dim / 2)) != cudaSuccess ||
        cudaMalloc(&lm->err, sizeof(unsigned)) != cudaSuccess ||
        cudaMalloc(&sp.part, sizeof(float) * row * most_splits * c.head_dim) != cudaSuccess ||
        cudaMalloc(&sp.part_lse, sizeof(float) * row * most_splits) != cudaSuccess ||
        cudaMalloc(&sp.pre, sizeof(float) * row * pre_max * c.head_dim) != cudaSuccess ||
        cudaMalloc(&sp.pre_lse, sizeof(float) * row * pre_max) != cudaSuccess ||
        cudaMalloc(&pr.list, 32 * items) != cudaSuccess || cudaMalloc(&pr.counts, 3 * sizeof(int)) != cudaSuccess ||
        cudaMalloc(&pr.joins, 16 * kLmSlots) != cudaSuccess ||
        cudaMalloc(&pr.piece, sizeof(float) * kLmSlots * 256 * c.head_dim) != cudaSuccess ||
        cudaMalloc(&pr.piece_lse, sizeof(float) * kLmSlots * 256) != cudaSuccess ||
        cudaMalloc(&bm.part, sizeof(LmBeamPart) * bm.parts) != cudaSuccess ||
        cudaMalloc(&bm.best, sizeof(uint2) * kLmMaxBeams * (size_t)bm.parts) != cudaSuccess ||
        cudaMalloc(&lm->block_map, sizeof(int) * (size_t)c.n_blocks) != cudaSuccess ||
        cudaMalloc(&sp.zeros, kLmZeroBytes) != cudaSuccess ||
        cudaMalloc(&sp.k16, 2 * (size_t)sp.shared_q4 * c.kv_heads * c.head_dim) != cudaSuccess ||
        cudaMalloc(&sp.v16, 2 * (size_t)sp.shared_q4 * c.kv_heads * c.head_dim) != cudaSuccess ||
        cudaMalloc(&sp.q16, halves ? 2 * row * c.head_dim : 0) != cudaSuccess ||
        cudaMalloc(&sp.row_c, halves ? sizeof(float) * row : 0) != cudaSuccess ||
        cudaMalloc(&sp.count, sizeof(int) * (sp.shared_q4 / c.block_size)) != cudaSuccess ||
        cudaMalloc(&sp.done, sizeof(int) * ((size_t)c.max_requests * c.kv_heads + 1)) != cudaSuccess) {
        cudaGetLastError();
        lm_free(lm);
        return CODEC_ERR_OOM;
    }
    sp.taken = sp.done + (size_t)c.max_requests * c.kv_heads;
    lm->shape = LmShape{c.type, c.q_heads, c.kv_heads, c.q_heads / c.kv_heads, c.head_dim, c.scale, lm->err, 0};
    if (configure_lm_plan() != cudaSuccess || configure_lm_prompt() != cudaSuccess ||
        configure_lm_step() != cudaSuccess || configure_lm_step_q4() != cudaSuccess ||
        configure_lm_pages() != cudaSuccess || configure_lm_beams() != cudaSuccess ||
        cudaMemset(sp.done, 0, sizeof(int) * ((size_t)c.max_requests * c.kv_heads + 1)) != cudaSuccess ||
        cudaMemset(sp.zeros, 0, kLmZeroBytes) != cudaSuccess ||
        (sp.shared_q4 > 0 && launch_lm_count(sp.count, sp.shared_q4 / c.block_size, nullptr) != cudaSuccess) ||
        cudaMemset(lm->err, 0, sizeof(unsigned)) != cudaSuccess ||
        launch_lm_turn_table(lm->turn, c.max_positions, c.head_dim, c.rope_theta, nullptr) != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
        lm_free(lm);
        return CODEC_ERR_CUDA;
    }
    *out = lm;
    return CODEC_OK;
}

void codec_lm_destroy(codec_lm_t* lm)
{
    if (!lm) return;
    OnDevice on(lm->device);
    cudaDeviceSynchronize();
    lm_free(lm);
}

codec_status codec_lm_errors(codec_lm_t* lm, uint32_t* bits, int32_t clear, void* stream)
{
    if (!lm || !bits) return CODEC_ERR_NULL;
    OnDevice on(lm->device);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!on.ok || cudaMemcpyAsync(bits, lm->err, sizeof(uint32_t), cudaMemcpyDeviceToHost, cs) != cudaSuccess ||
        (clear && (cudaMemsetAsync(lm->err, 0, sizeof(uint32_t), cs) != cudaSuccess ||
                   // a call that gave up may have left its counts of finished units
                   cudaMemsetAsync(lm->step.done, 0, sizeof(int) * ((size_t)lm->cfg.max_requests * lm->cfg.kv_heads + 1),
                                   cs) != cudaSuccess)) ||
        cudaStreamSynchronize(cs) != cudaSuccess)
        return CODEC_ERR_CUDA;
    return CODEC_OK;
}

codec_status codec_lm_set_unarrived_wait(codec_lm_t* lm, uint32_t polls)
{
    if (!lm) return CODEC_ERR_NULL;
    lm->shape.unarrived = std::min(polls, kLmPolls);
    return CODEC_OK;
}

codec_status codec_lm_plan(codec_lm_t* lm, const int32_t* len_before, const int32_t* len_after, int32_t B,
                           int32_t* tables, const int32_t* shared_table, int32_t shared_blocks, int32_t* free_list,
                           const int64_t* free_in, int64_t* free_out, int32_t* row_start, int32_t* kv_len,
                           int32_t* status, int32_t* slots, int32_t* positions, int32_t max_rows, void* stream)
{
    if (!lm || !len_before || !len_after || !tables || (shared_blocks > 0 && !shared_table) || !free_list ||
        !free_in || !free_out || !row_start || !kv_len || !status || !slots || !positions)
        return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    if (B < 1 || max_rows < 1 || shared_blocks < 0 || shared_blocks > c.table_blocks || free_in == free_out ||
        kv_len == len_before || kv_len == len_after)
        return CODEC_ERR_ARG;
    if (B > c.max_requests || max_rows > c.max_rows) return CODEC_ERR_CAPACITY;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmPlanArgs a{len_before, len_after, B, tables, shared_table, shared_blocks, c.table_blocks, lm->bs_shift,
                 c.n_blocks, free_list, reinterpret_cast<const long long*>(free_in),
                 reinterpret_cast<long long*>(free_out), row_start, kv_len, status, slots, positions, max_rows,
                 lm->err};
    return done(launch_lm_plan(a, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_rotate(codec_lm_t* lm, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, int32_t in_type, int32_t rows, const float* q_gain,
                             const float* k_gain, const int32_t* positions, const int32_t* slots, void* q_out,
                             void* k_dst, void* v_dst, void* stream)
{
    if (!lm || !q || !k || !positions || !q_out || !k_dst || (slots && (!v || !v_dst))) return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    const int64_t nq = (int64_t)c.q_heads * c.head_dim, nk = (int64_t)c.kv_heads * c.head_dim;
    const int size = in_type == CODEC_LM_FP32 ? 4 : 2;
    if (rows < 0 || (in_type != c.type && in_type != CODEC_LM_FP32) || !q_gain != !k_gain || !v != !v_dst ||
        !row_ok(q, q_stride, nq, size) || !row_ok(k, k_stride, nk, size) ||
        (v && (!row_ok(v, v_stride, nk, size) || !aligned16(v_dst))) || !aligned16(q_out) || !aligned16(k_dst) ||
        (q_gain && (!aligned16(q_gain) || !aligned16(k_gain))) ||
        (q == q_out && (in_type != c.type || q_stride != nq)) ||
        (k == k_dst && (slots || in_type != c.type || k_stride != nk)) ||
        (v && v == v_dst && (slots || in_type != c.type || v_stride != nk)))
        return CODEC_ERR_ARG;
    if (rows > c.max_rows) return CODEC_ERR_CAPACITY;
    if (rows == 0) return CODEC_OK;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmRotateArgs a{q, k, v, q_stride, k_stride, v_stride, rows, q_gain, k_gain, positions, slots,
                   (int64_t)c.n_blocks * c.block_size, q_out, k_dst, v_dst, lm->turn, c.max_positions, c.rms_eps,
                   c.rope_pairs};
    return done(launch_lm_rotate(lm->shape, a, in_type, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_prompt(codec_lm_t* lm, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, int32_t rows, const int32_t* row_start, int32_t B,
                             void* o, int64_t o_stride, float* lse, void* stream)
{
    if (!lm || !q || !k || !v || !row_start || !o) return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    const int64_t nq = (int64_t)c.q_heads * c.head_dim, nk = (int64_t)c.kv_heads * c.head_dim;
    if (B < 1 || rows < 0 || !row_ok(q, q_stride, nq, 2) || !row_ok(k, k_stride, nk, 2) ||
        !row_ok(v, v_stride, nk, 2) || !row_ok(o, o_stride, nq, 2) || o == q || o == k || o == v)
        return CODEC_ERR_ARG;
    if (B > c.max_requests || rows > c.max_rows) return CODEC_ERR_CAPACITY;
    if (rows == 0) return CODEC_OK;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmPromptArgs a{q, q_stride, rows, row_start, B, LmKeys{k, v, k_stride, v_stride}, o, o_stride, lse,
                   lm->prompt};
    return done(launch_lm_prompt(lm->shape, a, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_prompt_paged(codec_lm_t* lm, const void* q, int64_t q_stride, int32_t rows,
                                   const int32_t* row_start, int32_t B, const void* k_cache, const void* v_cache,
                                   const int32_t* tables, const int32_t* kv_len, void* o, int64_t o_stride,
                                   float* lse, void* stream)
{
    if (!lm || !q || !row_start || !k_cache || !v_cache || !tables || !kv_len || !o) return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    const int64_t nq = (int64_t)c.q_heads * c.head_dim;
    if (B < 1 || rows < 0 || !row_ok(q, q_stride, nq, 2) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !row_ok(o, o_stride, nq, 2) || o == q || o == k_cache || o == v_cache)
        return CODEC_ERR_ARG;
    if (B > c.max_requests || rows > c.max_rows) return CODEC_ERR_CAPACITY;
    if (rows == 0) return CODEC_OK;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmPromptArgs a{q, q_stride, rows, row_start, B, paged(lm, k_cache, v_cache, tables, kv_len), o, o_stride, lse,
                   lm->prompt};
    return done(launch_lm_prompt(lm->shape, a, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_step(codec_lm_t* lm, const void* q, int64_t q_stride, int32_t B, const void* k_cache,
                           const void* v_cache, const int32_t* tables, const int32_t* kv_len,
                           const int32_t* shared_table, int32_t shared_blocks, void* o, int64_t o_stride, float* lse,
                           void* stream)
{
    if (!lm || !q || !k_cache || !v_cache || !tables || !kv_len || (shared_blocks > 0 && !shared_table) || !o)
        return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    const int64_t nq = (int64_t)c.q_heads * c.head_dim;
    if (B < 1 || shared_blocks < 0 || shared_blocks > c.table_blocks || !row_ok(q, q_stride, nq, 2) ||
        !aligned16(k_cache) || !aligned16(v_cache) || !row_ok(o, o_stride, nq, 2) || o == q || o == k_cache ||
        o == v_cache)
        return CODEC_ERR_ARG;
    if (B > c.max_requests) return CODEC_ERR_CAPACITY;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmStepArgs a{q, q_stride, B, paged(lm, k_cache, v_cache, tables, kv_len), shared_table, shared_blocks, o,
                 o_stride, lse, lm->step};
    return done(launch_lm_step(lm->shape, a, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_store_q4(codec_lm_t* lm, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               int32_t in_type, int32_t rows, const int32_t* slots, void* k_cache, void* v_cache,
                               void* stream)
{
    if (!lm || !k || !v || !slots || !k_cache || !v_cache) return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    const int64_t nk = (int64_t)c.kv_heads * c.head_dim;
    const int size = in_type == CODEC_LM_FP32 ? 4 : 2;
    if (rows < 0 || (in_type != c.type && in_type != CODEC_LM_FP32) || !row_ok(k, k_stride, nk, size) ||
        !row_ok(v, v_stride, nk, size) || !aligned16(k_cache) || !aligned16(v_cache) || k_cache == v_cache ||
        k == k_cache || k == v_cache || v == k_cache || v == v_cache)
        return CODEC_ERR_ARG;
    if (rows > c.max_rows) return CODEC_ERR_CAPACITY;
    if (rows == 0) return CODEC_OK;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmStoreQ4Args a{k, v, k_stride, v_stride, rows, slots, (int64_t)c.n_blocks * c.block_size, lm->bs_shift, k_cache,
                    v_cache};
    return done(launch_lm_store_q4(lm->shape, a, in_type, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_load_q4(codec_lm_t* lm, const void* k_cache, const void* v_cache, const int32_t* src,
                              const int32_t* dst, int32_t n, void* k_dst, void* v_dst, int32_t dst_blocks,
                              void* stream)
{
    if (!lm || !k_cache || !v_cache || !src || !dst || !k_dst || !v_dst) return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    if (n < 0 || dst_blocks < 1 || (int64_t)dst_blocks * c.block_size >= (1LL << 31) - 128 || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned16(k_dst) || !aligned16(v_dst) || k_dst == v_dst || k_dst == k_cache ||
        k_dst == v_cache || v_dst == k_cache || v_dst == v_cache)
        return CODEC_ERR_ARG;
    if (n == 0) return CODEC_OK;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmLoadQ4Args a{k_cache, v_cache, src, dst, n, lm->bs_shift, c.n_blocks, dst_blocks, k_dst, v_dst};
    return done(launch_lm_load_q4(lm->shape, a, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_step_q4(codec_lm_t* lm, const void* q, int64_t q_stride, int32_t B, const void* k_cache,
                              const void* v_cache, const int32_t* tables, const int32_t* kv_len,
                              const int32_t* shared_table, int32_t shared_blocks, void* o, int64_t o_stride,
                              float* lse, void* stream)
{
    if (!lm || !q || !k_cache || !v_cache || !tables || !kv_len || (shared_blocks > 0 && !shared_table) || !o)
        return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    const int64_t nq = (int64_t)c.q_heads * c.head_dim;
    if (B < 1 || shared_blocks < 0 || shared_blocks > c.table_blocks || !row_ok(q, q_stride, nq, 2) ||
        !aligned16(k_cache) || !aligned16(v_cache) || !row_ok(o, o_stride, nq, 2) || o == q || o == k_cache ||
        o == v_cache)
        return CODEC_ERR_ARG;
    if (B > c.max_requests) return CODEC_ERR_CAPACITY;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmStepArgs a{q, q_stride, B, paged(lm, k_cache, v_cache, tables, kv_len), shared_table, shared_blocks, o,
                 o_stride, lse, lm->step};
    return done(launch_lm_step_q4(lm->shape, a, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_beams(codec_lm_t* lm, const void* logits, int64_t stride, int32_t in_type, int32_t groups,
                            int32_t beams, int32_t vocab, const float* sums, const int32_t* ended, int32_t end_token,
                            float* sums_out, int32_t* parents, int32_t* tokens, int32_t* ended_out, void* stream)
{
    if (!lm || !logits || !sums || !ended || !sums_out || !parents || !tokens || !ended_out) return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    const bool typed = in_type == CODEC_LM_BF16 || in_type == CODEC_LM_FP16 || in_type == CODEC_LM_FP32;
    const uintptr_t size = in_type == CODEC_LM_FP32 ? 4 : 2;
    if (!typed || groups < 1 || beams < 1 || beams > kLmMaxBeams || vocab < 2 || vocab > (1 << 24) || stride < vocab ||
        stride > (1LL << 32) || reinterpret_cast<uintptr_t>(logits) % size || end_token < -1 || end_token >= vocab ||
        !apart({sums_out, parents, tokens, ended_out}, {logits, sums, ended}))
        return CODEC_ERR_ARG;
    if ((int64_t)groups * beams > c.max_requests) return CODEC_ERR_CAPACITY;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmBeamArgs a{logits, stride, in_type, groups, beams, vocab, sums, ended, end_token, sums_out, parents, tokens,
                 ended_out, lm->beam};
    return done(launch_lm_beams(a, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_fork(codec_lm_t* lm, const int32_t* parents, const int32_t* len, int32_t B,
                           const int32_t* tables, int32_t* tables_out, int32_t shared_blocks, const int32_t* owners,
                           int32_t* owners_out, int32_t* free_list, const int64_t* free_in, int64_t* free_out,
                           int32_t* kv_len, int32_t* status, int32_t* copy_src, int32_t* copy_dst, int32_t* copies,
                           void* stream)
{
    if (!lm || !parents || !len || !tables || !tables_out || !owners || !owners_out || !free_list || !free_in ||
        !free_out || !kv_len || !status || !copy_src || !copy_dst || !copies)
        return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    if (B < 1 || shared_blocks < 0 || shared_blocks > c.table_blocks ||
        !apart({tables_out, owners_out, free_list, free_out, kv_len, status, copy_src, copy_dst, copies},
               {parents, len, tables, owners, free_in}))
        return CODEC_ERR_ARG;
    if (B > c.max_requests) return CODEC_ERR_CAPACITY;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmForkArgs a{parents, len, B, tables, tables_out, shared_blocks, c.table_blocks, lm->bs_shift, c.n_blocks, owners,
                 owners_out, free_list, reinterpret_cast<const long long*>(free_in),
                 reinterpret_cast<long long*>(free_out), kv_len, status, copy_src, copy_dst, copies, lm->err};
    return done(launch_lm_fork(a, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_compact(codec_lm_t* lm, const int32_t* len, int32_t B, const int32_t* tables,
                              int32_t* tables_out, const int32_t* shared_table, int32_t* shared_out,
                              int32_t shared_blocks, const int32_t* owners, int32_t* owners_out, int32_t* free_list,
                              int64_t* free_out, int32_t* copy_src, int32_t* copy_dst, int32_t* copies, void* stream)
{
    if (!lm || !len || !tables || !tables_out || (shared_blocks > 0 && (!shared_table || !shared_out)) || !free_list ||
        !free_out || (lm->cfg.n_blocks > 1 && (!copy_src || !copy_dst)) || !copies || !owners != !owners_out)
        return CODEC_ERR_NULL;
    const codec_lm_config& c = lm->cfg;
    if (B < 1 || shared_blocks < 0 || shared_blocks > c.table_blocks ||
        !apart({tables_out, shared_out, owners_out, free_list, free_out, copy_src, copy_dst, copies},
               {len, tables, shared_table, owners}))
        return CODEC_ERR_ARG;
    if (B > c.max_requests) return CODEC_ERR_CAPACITY;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    LmCompactArgs a{len, B, tables, tables_out, shared_table, shared_out, shared_blocks, c.table_blocks, lm->bs_shift,
                    c.n_blocks, owners, owners_out, free_list, reinterpret_cast<long long*>(free_out), copy_src,
                    copy_dst, copies, lm->block_map, lm->err};
    return done(launch_lm_compact(a, static_cast<cudaStream_t>(stream)));
}

codec_status codec_lm_copy(codec_lm_t* lm, void* const* caches, int32_t n_caches, int64_t block_bytes,
                           const int32_t* src, const int32_t* dst, int32_t n, const int32_t* copies, void* stream)
{
    if (!lm || !caches || (n > 0 && (!src || !dst))) return CODEC_ERR_NULL;
    if (n < 0 || n_caches < 1 || n_caches > kLmMaxCaches || block_bytes < 16 || block_bytes % 16 ||
        block_bytes > (1LL << 28))
        return CODEC_ERR_ARG;
    LmCopyArgs a{};
    for (int i = 0; i < n_caches; i++) {
        if (!caches[i]) return CODEC_ERR_NULL;
        if (!aligned16(caches[i])) return CODEC_ERR_ARG;
        a.caches[i] = caches[i];
    }
    if (n == 0) return CODEC_OK;
    OnDevice on(lm->device);
    if (!on.ok) return CODEC_ERR_CUDA;
    a.src = src;
    a.dst = dst;
    a.copies = copies;
    a.n = n;
    a.n_caches = n_caches;
    a.n_blocks = lm->cfg.n_blocks;
    a.block_bytes = block_bytes;
    a.err = lm->err;
    return done(launch_lm_copy(a, static_cast<cudaStream_t>(stream)));
}
