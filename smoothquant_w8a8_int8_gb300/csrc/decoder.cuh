// Host interfaces of the decoder's operators: the RMS norm with its quantiser, the
// paged cache's append and the attention over it.
#pragma once
#include "common.cuh"

namespace sq {

// RMS norm of H (+ residual, nullable) with the quantiser on it; R, Y nullable.
sq_status launch_rmsnorm_quant(const float *H, const float *residual, const float *gamma,
                               float eps, const float *s, int64_t rows, int64_t K,
                               float static_scale, float *R, float *Y, int8_t *q, float *scale,
                               __nv_bfloat16 *op, int32_t *l1, cudaStream_t st);
// The rotation's table, and the append to the paged cache with the rotation.
sq_status launch_rope_table(const float *inv_freq, int64_t positions, int64_t rot, float *table,
                            cudaStream_t st);
sq_status launch_kv_append(const float *QKV, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                           const float *rope, int64_t rope_positions, int64_t rot,
                           int interleaved, const int32_t *q_start, const int32_t *kv_len,
                           int64_t B, const int32_t *block_table, int64_t max_pages,
                           void *k_cache, void *v_cache, int cache_type, int64_t num_pages,
                           int64_t page_size, float *Q, int64_t ldq, cudaStream_t st);
// The error word of the attention over the paged cache, and its workspace.
sq_status paged_take_error(cudaStream_t st);
sq_status paged_workspace_bytes(int64_t T, int64_t Hq, int64_t D, int64_t prefix_len,
                                size_t *bytes);
// Attention over the paged cache (the arguments of sq_paged_attention, checked).
struct PagedCall {
    const float *Q;
    int64_t ldq, T, Hq, Hkv, D;
    const void *k_cache, *v_cache;
    int cache_type;
    int64_t num_pages, page_size;
    const int32_t *block_table;
    int64_t max_pages;
    const int32_t *q_start, *kv_len;
    int64_t B, max_q;
    const int32_t *prefix_pages;
    int64_t prefix_len;
    float scale;
    float *O;
    void *workspace;
};
sq_status launch_paged_attention(const PagedCall &c, cudaStream_t st);

}  // namespace sq
