// C-ABI boundary: argument checks, then one launch per call on the caller's
// stream.  Declarations and the contract of every entry point are in sq.h.
#include "decoder.cuh"
#include "gated.cuh"

#include <cmath>
#include <mutex>

namespace sq {

sq_status device_info(DeviceInfo *out) {
    static std::mutex mu;
    static DeviceInfo cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SQ_ERR_CUDA;
    if (dev < 0 || dev >= 64) return SQ_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(mu);
    DeviceInfo &c = cache[dev];
    if (c.device != dev) {
        cudaDeviceProp p;
        if (cudaGetDeviceProperties(&p, dev) != cudaSuccess) return SQ_ERR_CUDA;
        c.sms = p.multiProcessorCount;
        c.major = p.major;
        c.minor = p.minor;
        c.smem_optin = p.sharedMemPerBlockOptin;
        c.device = dev;
    }
    *out = c;
    return SQ_OK;
}

}  // namespace sq

using namespace sq;

namespace {

inline cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }

// The kernels are built for sm_103a only.
sq_status require_sm103() {
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    if (di.major != 10 || di.minor != 3) return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

constexpr int64_t kMaxK = 133144;  // K * 127^2 < 2^31
constexpr int64_t kMaxGated = (int64_t)1 << 24;  // outputs of a gated block: rows fit a grid

sq_status check_linear_args(const void *X, const float *sx, const void *W, const float *sw,
                            const float *bias, const float *residual, int64_t M, int64_t N,
                            int64_t K, int mode, const void *Y) {
    if (M < 0 || N < 0 || K <= 0) return SQ_ERR_INVALID_ARG;
    if (mode < SQ_EPI_NONE || mode > SQ_EPI_RAW_I32) return SQ_ERR_INVALID_ARG;
    if (K % 16 != 0) return SQ_ERR_ALIGNMENT;
    if (K > kMaxK) return SQ_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return SQ_OK;  // empty: pointers may be NULL, nothing is launched
    if (!X || !W || !Y) return SQ_ERR_INVALID_ARG;
    if (mode != SQ_EPI_RAW_I32 && (!sx || !sw)) return SQ_ERR_INVALID_ARG;
    if ((mode == SQ_EPI_BIAS || mode == SQ_EPI_BIAS_GELU || mode == SQ_EPI_BIAS_RESIDUAL) &&
        !bias)
        return SQ_ERR_INVALID_ARG;
    if (mode == SQ_EPI_BIAS_RESIDUAL && !residual) return SQ_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(W) || !aligned16(Y)) return SQ_ERR_ALIGNMENT;
    if (mode != SQ_EPI_RAW_I32 && (!aligned4(sx) || !aligned4(sw))) return SQ_ERR_ALIGNMENT;
    if (bias && !aligned4(bias)) return SQ_ERR_ALIGNMENT;
    if (mode == SQ_EPI_BIAS_RESIDUAL && !aligned16(residual)) return SQ_ERR_ALIGNMENT;
    return SQ_OK;
}

sq_status check_quant_args(const float *A, const float *s, int64_t rows, int64_t K,
                           const int8_t *q, const float *scale, const void *op) {
    if (rows < 0 || K <= 0) return SQ_ERR_INVALID_ARG;
    if (K % 16 != 0) return SQ_ERR_ALIGNMENT;
    if (K > (int64_t)1 << 30) return SQ_ERR_UNSUPPORTED;
    if (rows == 0) return SQ_OK;  // empty: pointers may be NULL, nothing is launched
    if (!A || !s || !scale) return SQ_ERR_INVALID_ARG;
    if (!q && !op) return SQ_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(s) || (q && !aligned16(q)) || (op && !aligned16(op)))
        return SQ_ERR_ALIGNMENT;
    if (!aligned4(scale)) return SQ_ERR_ALIGNMENT;
    return SQ_OK;
}

// Sizes of the paged cache and of the rows that go with it.
sq_status check_paged_shape(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int cache_type,
                            int64_t num_pages, int64_t page_size, int64_t B, int64_t max_pages,
                            int64_t ldq) {
    if (T < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || num_pages < 0 || B < 0 || max_pages < 0)
        return SQ_ERR_INVALID_ARG;
    if (cache_type != SQ_CACHE_BF16 && cache_type != SQ_CACHE_F16) return SQ_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SQ_ERR_UNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 &&
        page_size != 256)
        return SQ_ERR_UNSUPPORTED;
    if (Hq % Hkv != 0) return SQ_ERR_INVALID_ARG;
    if (Hq > 4096 || Hq / Hkv > 128) return SQ_ERR_UNSUPPORTED;
    if (ldq < Hq * D) return SQ_ERR_INVALID_ARG;
    if (ldq % 4 != 0) return SQ_ERR_ALIGNMENT;
    // token, sequence, key and cache-row numbers are 32-bit; element offsets are not
    const int64_t lim = (int64_t)1 << 30;
    if (T > (int64_t)1 << 24 || B > lim || max_pages > lim / page_size || num_pages > lim / (Hkv * page_size))
        return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

}  // namespace

namespace sq {

sq_status validate_linear(const void *Xop, const float *x_scale, const int32_t *x_row_l1,
                          const void *Wop, const float *w_scale, const int32_t *w_row_l1,
                          const float *bias, const float *residual, int64_t M, int64_t N,
                          int64_t K, int mode, const void *Y) {
    sq_status rc = check_linear_args(Xop, x_scale, Wop, w_scale, bias, residual, M, N, K, mode, Y);
    if (rc != SQ_OK) return rc;
    if (M == 0 || N == 0) return SQ_OK;
    if ((x_row_l1 && !aligned4(x_row_l1)) || (w_row_l1 && !aligned4(w_row_l1)))
        return SQ_ERR_ALIGNMENT;
    return SQ_OK;
}

sq_status require_gb300() { return require_sm103(); }

}  // namespace sq

namespace {

// The appends' arguments apart from the shape; *empty: a valid call without work.
sq_status check_append(const float *QKV, int64_t T, int64_t D, const float *rope,
                       int64_t rope_positions, int64_t rot, const int32_t *q_start,
                       const int32_t *kv_len, int64_t B, const int32_t *block_table,
                       const void *k_cache, const void *v_cache, int64_t num_pages,
                       const float *Q, bool *empty) {
    if (rot < 0 || rot > D || rope_positions < 0) return SQ_ERR_INVALID_ARG;
    if (rot % 8 != 0) return SQ_ERR_ALIGNMENT;
    *empty = T == 0 || B == 0;
    if (*empty) return SQ_OK;
    if (num_pages == 0 || !QKV || !q_start || !kv_len || !block_table || !k_cache || !v_cache || !Q ||
        (rot > 0 && !rope))
        return SQ_ERR_INVALID_ARG;
    if (!aligned16(QKV) || !aligned16(Q) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (rot > 0 && !aligned16(rope)) || !aligned4(q_start) || !aligned4(kv_len) ||
        !aligned4(block_table))
        return SQ_ERR_ALIGNMENT;
    return SQ_OK;
}

// The scales of an int8 cache (read 16 bytes at a time).
sq_status check_cache_scales(const float *k_scale, const float *v_scale) {
    if (!k_scale || !v_scale) return SQ_ERR_INVALID_ARG;
    return aligned16(k_scale) && aligned16(v_scale) ? SQ_OK : SQ_ERR_ALIGNMENT;
}

// The attentions' other checks, and the call.
sq_status attention_impl(const PagedCall &c, size_t workspace_bytes, void *stream) {
    if (!(fabsf(c.scale) <= 0x1p127f)) return SQ_ERR_INVALID_ARG;  // (times log2 e it is finite)
    if (c.max_q < 0 || c.prefix_len < 0) return SQ_ERR_INVALID_ARG;
    if (c.prefix_len > (int64_t)1 << 30) return SQ_ERR_UNSUPPORTED;
    if (c.T == 0 || c.B == 0) return SQ_OK;
    if (c.num_pages == 0 || !c.Q || !c.q_start || !c.kv_len || !c.block_table || !c.k_cache ||
        !c.v_cache || !c.O || !c.workspace || (c.prefix_len > 0 && !c.prefix_pages))
        return SQ_ERR_INVALID_ARG;
    if (!aligned16(c.Q) || !aligned16(c.O) || !aligned16(c.k_cache) || !aligned16(c.v_cache) ||
        !aligned16(c.workspace) || !aligned4(c.q_start) || !aligned4(c.kv_len) ||
        !aligned4(c.block_table) || (c.prefix_len > 0 && !aligned4(c.prefix_pages)))
        return SQ_ERR_ALIGNMENT;
    sq_status rc = c.cache_type == kCacheI8 ? check_cache_scales(c.k_scale, c.v_scale) : SQ_OK;
    if (rc != SQ_OK) return rc;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    size_t need = 0;
    if ((rc = paged_workspace_bytes(c.T, c.Hq, c.D, c.prefix_len, &need)) != SQ_OK) return rc;
    if (workspace_bytes < need) return SQ_ERR_INVALID_ARG;
    return launch_paged_attention(c, as_stream(stream));
}

sq_status linear_impl(const void *Xop, const float *x_scale, const int32_t *x_row_l1,
                      const void *Wop, const float *w_scale, const int32_t *w_row_l1,
                      const float *bias, const float *residual, int64_t M, int64_t N, int64_t K,
                      int mode, void *Y, void *workspace, size_t workspace_bytes, void *stream) {
    sq_status rc = validate_linear(Xop, x_scale, x_row_l1, Wop, w_scale, w_row_l1, bias, residual,
                                   M, N, K, mode, Y);
    if (rc != SQ_OK) return rc;
    if (M == 0 || N == 0) return SQ_OK;
    if (workspace && !aligned16(workspace)) return SQ_ERR_ALIGNMENT;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_gemm_tc(static_cast<const __nv_bfloat16 *>(Xop), x_scale, x_row_l1,
                          static_cast<const __nv_bfloat16 *>(Wop), w_scale, w_row_l1, bias,
                          residual, M, N, K, mode, Y, nullptr, workspace, workspace_bytes,
                          as_stream(stream));
}

sq_status requant_impl(const void *Xop, const float *x_scale, const int32_t *x_row_l1,
                       const void *Wop, const float *w_scale, const int32_t *w_row_l1,
                       const float *bias, const float *residual, int64_t M, int64_t N, int64_t K,
                       int mode, const float *s_next, float scale, int8_t *Yq, void *Yop,
                       float *x_scale_next, void *workspace, size_t workspace_bytes,
                       void *stream) {
    if (mode == SQ_EPI_RAW_I32) return SQ_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !(scale <= 3.4028234663852886e38f)) return SQ_ERR_INVALID_ARG;
    const void *out = Yop ? Yop : static_cast<const void *>(Yq);
    sq_status rc = check_linear_args(Xop, x_scale, Wop, w_scale, bias, residual, M, N, K, mode,
                                     out);
    if (rc != SQ_OK) return rc;
    if (M == 0 || N == 0) return SQ_OK;
    if (!s_next || (!Yq && !Yop)) return SQ_ERR_INVALID_ARG;
    if (!aligned4(s_next) || (x_scale_next && !aligned4(x_scale_next)) ||
        (Yop && (reinterpret_cast<uintptr_t>(Yop) & 1u)))
        return SQ_ERR_ALIGNMENT;
    if ((x_row_l1 && !aligned4(x_row_l1)) || (w_row_l1 && !aligned4(w_row_l1)))
        return SQ_ERR_ALIGNMENT;
    if (workspace && !aligned16(workspace)) return SQ_ERR_ALIGNMENT;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    RequantOut rq;
    rq.s_next = s_next;
    rq.scale = scale;
    rq.rscale = 1.0f / scale;  // IEEE division: the correctly rounded reciprocal
    rq.Yq = Yq;
    rq.Yop = static_cast<__nv_bfloat16 *>(Yop);
    rq.x_scale = x_scale_next;
    return launch_gemm_tc(static_cast<const __nv_bfloat16 *>(Xop), x_scale, x_row_l1,
                          static_cast<const __nv_bfloat16 *>(Wop), w_scale, w_row_l1, bias,
                          residual, M, N, K, mode, nullptr, &rq, workspace, workspace_bytes,
                          as_stream(stream));
}

}  // namespace

extern "C" {

const char *sq_status_string(int status) {
    switch (status) {
    case SQ_OK: return "SQ_OK";
    case SQ_ERR_INVALID_ARG: return "SQ_ERR_INVALID_ARG: invalid argument";
    case SQ_ERR_ALIGNMENT: return "SQ_ERR_ALIGNMENT: K not a multiple of 16 or misaligned pointer";
    case SQ_ERR_UNSUPPORTED: return "SQ_ERR_UNSUPPORTED: size limit exceeded or device not sm_103";
    case SQ_ERR_CUDA: return "SQ_ERR_CUDA: CUDA call or kernel launch failed";
    case SQ_ERR_TIMEOUT: return "SQ_ERR_TIMEOUT: a kernel's bounded pipeline wait ran out";
    default: return "unknown sq_status";
    }
}

int sq_version(void) { return (1 << 16) | 0; }

size_t sq_operand_bytes(int64_t rows, int64_t K) {
    if (rows < 0 || K < 0) return 0;
    return (size_t)rows * (size_t)K * sizeof(__nv_bfloat16);
}

size_t sq_packed_weight_bytes(int64_t N, int64_t K) { return sq_operand_bytes(N, K); }

sq_status sq_channel_absmax(const float *A, int64_t rows, int64_t cols, float *amax,
                            void *stream) {
    if (rows < 0 || cols <= 0) return SQ_ERR_INVALID_ARG;
    if (rows == 0) return SQ_OK;
    if (!A || !amax) return SQ_ERR_INVALID_ARG;
    if (!aligned4(A) || !aligned4(amax)) return SQ_ERR_ALIGNMENT;
    sq_status rc = require_sm103();
    if (rc != SQ_OK) return rc;
    return launch_channel_absmax(A, rows, cols, amax, as_stream(stream));
}

sq_status sq_smooth_factor(const float *x_amax, const float *w_amax, int64_t K, float alpha,
                           float *s, void *stream) {
    if (!x_amax || !w_amax || !s || K <= 0) return SQ_ERR_INVALID_ARG;
    if (!(alpha >= 0.0f && alpha <= 1.0f)) return SQ_ERR_INVALID_ARG;
    if (!aligned4(x_amax) || !aligned4(w_amax) || !aligned4(s)) return SQ_ERR_ALIGNMENT;
    sq_status rc = require_sm103();
    if (rc != SQ_OK) return rc;
    return launch_smooth_factor(x_amax, w_amax, K, alpha, s, as_stream(stream));
}

sq_status sq_pack_weight(const float *W, const float *s, int64_t N, int64_t K, int8_t *Wq,
                         float *w_scale, void *Wop, int32_t *w_row_l1, void *stream) {
    sq_status rc = check_quant_args(W, s, N, K, Wq, w_scale, Wop);
    if (rc != SQ_OK) return rc;
    if (N == 0) return SQ_OK;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    if (w_row_l1 && !aligned4(w_row_l1)) return SQ_ERR_ALIGNMENT;
    return launch_quantize_rows(1, W, s, N, K, Wq, w_scale, static_cast<__nv_bfloat16 *>(Wop),
                                w_row_l1, 0.0f, as_stream(stream));
}

sq_status sq_quantize_act(const float *X, const float *s, int64_t M, int64_t K, int8_t *Xq,
                          float *x_scale, void *Xop, int32_t *x_row_l1, void *stream) {
    sq_status rc = check_quant_args(X, s, M, K, Xq, x_scale, Xop);
    if (rc != SQ_OK) return rc;
    if (M == 0) return SQ_OK;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    if (x_row_l1 && !aligned4(x_row_l1)) return SQ_ERR_ALIGNMENT;
    return launch_quantize_rows(0, X, s, M, K, Xq, x_scale, static_cast<__nv_bfloat16 *>(Xop),
                                x_row_l1, 0.0f, as_stream(stream));
}

sq_status sq_act_absmax(const float *X, const float *s, int64_t M, int64_t K, float *amax,
                        void *stream) {
    if (M < 0 || K <= 0) return SQ_ERR_INVALID_ARG;
    if (K % 16 != 0) return SQ_ERR_ALIGNMENT;
    if (M == 0) return SQ_OK;
    if (!X || !s || !amax) return SQ_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(s) || !aligned4(amax)) return SQ_ERR_ALIGNMENT;
    sq_status rc = require_sm103();
    if (rc != SQ_OK) return rc;
    return launch_act_absmax(X, s, M, K, amax, as_stream(stream));
}

sq_status sq_division_table(const float *s, int64_t K, float *table, void *stream) {
    if (K < 0) return SQ_ERR_INVALID_ARG;
    if (K == 0) return SQ_OK;
    if (!s || !table) return SQ_ERR_INVALID_ARG;
    if (!aligned4(s) || !aligned16(table)) return SQ_ERR_ALIGNMENT;
    sq_status rc = require_sm103();
    if (rc != SQ_OK) return rc;
    return launch_division_table(s, K, table, as_stream(stream));
}

sq_status sq_linear_i8_rowmax(const void *Xop, const float *x_scale, const int32_t *x_row_l1,
                              const void *Wop, const float *w_scale, const int32_t *w_row_l1,
                              const float *bias, const float *residual, int64_t M, int64_t N,
                              int64_t K, int mode, void *Y, const float *next_table,
                              float *row_amax, void *stream) {
    if (mode == SQ_EPI_RAW_I32) return SQ_ERR_INVALID_ARG;
    sq_status rc = validate_linear(Xop, x_scale, x_row_l1, Wop, w_scale, w_row_l1, bias, residual,
                                   M, N, K, mode, Y);
    if (rc != SQ_OK) return rc;
    if (M == 0 || N == 0) return SQ_OK;
    if (!next_table || !row_amax) return SQ_ERR_INVALID_ARG;
    if (!aligned16(next_table) || !aligned4(row_amax)) return SQ_ERR_ALIGNMENT;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_gemm_tc(static_cast<const __nv_bfloat16 *>(Xop), x_scale, x_row_l1,
                          static_cast<const __nv_bfloat16 *>(Wop), w_scale, w_row_l1, bias,
                          residual, M, N, K, mode, Y, nullptr, nullptr, 0, as_stream(stream),
                          next_table, row_amax);
}

sq_status sq_quantize_act_rowmax(const float *X, const float *s, const float *row_amax,
                                 int64_t M, int64_t K, int8_t *Xq, float *x_scale, void *Xop,
                                 int32_t *x_row_l1, void *stream) {
    sq_status rc = check_quant_args(X, s, M, K, Xq, x_scale, Xop);
    if (rc != SQ_OK) return rc;
    if (M == 0) return SQ_OK;
    if (!row_amax) return SQ_ERR_INVALID_ARG;
    if (!aligned4(row_amax) || (x_row_l1 && !aligned4(x_row_l1))) return SQ_ERR_ALIGNMENT;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_quantize_act_given_max(X, s, row_amax, M, K, Xq, x_scale,
                                         static_cast<__nv_bfloat16 *>(Xop), x_row_l1,
                                         as_stream(stream));
}

sq_status sq_quantize_act_table(const float *X, const float *s, const float *s_table,
                                const float *row_amax, int64_t M, int64_t K, int8_t *Xq,
                                float *x_scale, void *Xop, int32_t *x_row_l1, void *stream) {
    sq_status rc = check_quant_args(X, s, M, K, Xq, x_scale, Xop);
    if (rc != SQ_OK) return rc;
    if (M == 0) return SQ_OK;
    if (!s_table) return SQ_ERR_INVALID_ARG;
    if (!aligned16(s_table) || (row_amax && !aligned4(row_amax)) ||
        (x_row_l1 && !aligned4(x_row_l1)))
        return SQ_ERR_ALIGNMENT;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_quantize_act_table(X, s, s_table, row_amax, M, K, Xq, x_scale,
                                     static_cast<__nv_bfloat16 *>(Xop), x_row_l1,
                                     as_stream(stream));
}

sq_status sq_attention(const float *QKV, int64_t B, int64_t S, int64_t H, int64_t D,
                       float scale, float *O, void *stream) {
    if (B < 0 || S < 0 || H < 0 || D <= 0) return SQ_ERR_INVALID_ARG;
    if (!(scale == scale) || !(fabsf(scale) <= 3.4028234663852886e38f)) return SQ_ERR_INVALID_ARG;
    if (D != 64 || S % 64 != 0 || S > 448) return SQ_ERR_UNSUPPORTED;
    if (B == 0 || S == 0 || H == 0) return SQ_OK;
    if (B * S >= ((int64_t)1 << 31) || H > 65536) return SQ_ERR_UNSUPPORTED;
    if (!QKV || !O) return SQ_ERR_INVALID_ARG;
    if (!aligned16(QKV) || !aligned16(O)) return SQ_ERR_ALIGNMENT;
    sq_status rc = require_sm103();
    if (rc != SQ_OK) return rc;
    return launch_attention(QKV, B, S, H, scale, O, as_stream(stream));
}

sq_status sq_static_scale(const float *amax, float *scale, void *stream) {
    if (!amax || !scale) return SQ_ERR_INVALID_ARG;
    if (!aligned4(amax) || !aligned4(scale)) return SQ_ERR_ALIGNMENT;
    sq_status rc = require_sm103();
    if (rc != SQ_OK) return rc;
    return launch_static_scale(amax, scale, as_stream(stream));
}

sq_status sq_quantize_act_static(const float *X, const float *s, int64_t M, int64_t K,
                                 float scale, int8_t *Xq, float *x_scale, void *Xop,
                                 int32_t *x_row_l1, void *stream) {
    if (!(scale > 0.0f) || !(scale <= 3.4028234663852886e38f)) return SQ_ERR_INVALID_ARG;
    sq_status rc = check_quant_args(X, s, M, K, Xq, x_scale, Xop);
    if (rc != SQ_OK) return rc;
    if (M == 0) return SQ_OK;
    if (x_row_l1 && !aligned4(x_row_l1)) return SQ_ERR_ALIGNMENT;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_quantize_rows(2, X, s, M, K, Xq, x_scale, static_cast<__nv_bfloat16 *>(Xop),
                                x_row_l1, scale, as_stream(stream));
}

sq_status sq_layernorm_quant(const float *H, const float *gamma, const float *beta, float eps,
                             const float *s, int64_t M, int64_t K, float static_scale, float *Y,
                             int8_t *Xq, float *x_scale, void *Xop, int32_t *x_row_l1,
                             void *stream) {
    if (!(eps >= 0.0f) || !(eps <= 3.4028234663852886e38f)) return SQ_ERR_INVALID_ARG;
    if (!(static_scale >= 0.0f) || !(static_scale <= 3.4028234663852886e38f))
        return SQ_ERR_INVALID_ARG;
    sq_status rc = check_quant_args(H, s, M, K, Xq, x_scale, Xop);
    if (rc != SQ_OK) return rc;
    if (M == 0) return SQ_OK;
    if (!gamma || !beta) return SQ_ERR_INVALID_ARG;
    if (!aligned16(gamma) || !aligned16(beta) || (Y && !aligned16(Y)) ||
        (x_row_l1 && !aligned4(x_row_l1)))
        return SQ_ERR_ALIGNMENT;
    if (K > 8192) return SQ_ERR_UNSUPPORTED;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_layernorm_quant(H, gamma, beta, eps, s, M, K, static_scale, Y, Xq, x_scale,
                                  static_cast<__nv_bfloat16 *>(Xop), x_row_l1, as_stream(stream));
}

sq_status sq_rmsnorm_quant(const float *H, const float *residual, const float *gamma, float eps,
                           const float *s, int64_t M, int64_t K, float static_scale, float *R,
                           float *Y, int8_t *Xq, float *x_scale, void *Xop, int32_t *x_row_l1,
                           void *stream) {
    if (!(eps >= 0.0f) || !(eps <= 3.4028234663852886e38f)) return SQ_ERR_INVALID_ARG;
    if (!(static_scale >= 0.0f) || !(static_scale <= 3.4028234663852886e38f))
        return SQ_ERR_INVALID_ARG;
    sq_status rc = check_quant_args(H, s, M, K, Xq, x_scale, Xop);
    if (rc != SQ_OK) return rc;
    if (M == 0) return SQ_OK;
    if (!gamma) return SQ_ERR_INVALID_ARG;
    if (!aligned16(gamma) || (residual && !aligned16(residual)) || (R && !aligned16(R)) ||
        (Y && !aligned16(Y)) || (x_row_l1 && !aligned4(x_row_l1)))
        return SQ_ERR_ALIGNMENT;
    if (K > 16384) return SQ_ERR_UNSUPPORTED;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_rmsnorm_quant(H, residual, gamma, eps, s, M, K, static_scale, R, Y, Xq, x_scale,
                                static_cast<__nv_bfloat16 *>(Xop), x_row_l1, as_stream(stream));
}

sq_status sq_rope_table(const float *inv_freq, int64_t positions, int64_t rot, float *table,
                        void *stream) {
    if (positions < 0 || rot < 0) return SQ_ERR_INVALID_ARG;
    if (rot % 8 != 0) return SQ_ERR_ALIGNMENT;
    if (positions > (int64_t)1 << 31 || rot > 1024) return SQ_ERR_UNSUPPORTED;
    if (positions == 0 || rot == 0) return SQ_OK;
    if (!inv_freq || !table) return SQ_ERR_INVALID_ARG;
    if (!aligned4(inv_freq) || !aligned16(table)) return SQ_ERR_ALIGNMENT;
    sq_status rc = require_sm103();
    if (rc != SQ_OK) return rc;
    return launch_rope_table(inv_freq, positions, rot, table, as_stream(stream));
}

sq_status sq_kv_append(const float *QKV, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                       const float *rope, int64_t rope_positions, int64_t rot, int interleaved,
                       const int32_t *q_start, const int32_t *kv_len, int64_t B,
                       const int32_t *block_table, int64_t max_pages, void *k_cache,
                       void *v_cache, int cache_type, int64_t num_pages, int64_t page_size,
                       float *Q, int64_t ldq, void *stream) {
    sq_status rc = check_paged_shape(T, Hq, Hkv, D, cache_type, num_pages, page_size, B,
                                     max_pages, ldq);
    if (rc != SQ_OK) return rc;
    bool empty = false;
    rc = check_append(QKV, T, D, rope, rope_positions, rot, q_start, kv_len, B, block_table, k_cache,
                      v_cache, num_pages, Q, &empty);
    if (rc != SQ_OK || empty) return rc;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_kv_append(QKV, T, Hq, Hkv, D, rope, rope_positions, rot, interleaved ? 1 : 0,
                            q_start, kv_len, B, block_table, max_pages, k_cache, v_cache,
                            cache_type, num_pages, page_size, Q, ldq, as_stream(stream));
}

sq_status sq_kv_append_i8(const float *QKV, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                          const float *rope, int64_t rope_positions, int64_t rot, int interleaved,
                          const int32_t *q_start, const int32_t *kv_len, int64_t B,
                          const int32_t *block_table, int64_t max_pages, int8_t *k_cache,
                          int8_t *v_cache, float *k_scale, float *v_scale, int64_t num_pages,
                          int64_t page_size, float *Q, int64_t ldq, void *stream) {
    sq_status rc = check_paged_shape(T, Hq, Hkv, D, SQ_CACHE_BF16, num_pages, page_size, B,
                                     max_pages, ldq);
    if (rc != SQ_OK) return rc;
    bool empty = false;
    rc = check_append(QKV, T, D, rope, rope_positions, rot, q_start, kv_len, B, block_table, k_cache,
                      v_cache, num_pages, Q, &empty);
    if (rc != SQ_OK || empty) return rc;
    if ((rc = check_cache_scales(k_scale, v_scale)) != SQ_OK) return rc;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_kv_append_i8(QKV, T, Hq, Hkv, D, rope, rope_positions, rot, interleaved ? 1 : 0,
                               q_start, kv_len, B, block_table, max_pages, k_cache, v_cache,
                               k_scale, v_scale, num_pages, page_size, Q, ldq, as_stream(stream));
}

sq_status sq_paged_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                             int64_t prefix_len, size_t *bytes) {
    if (!bytes) return SQ_ERR_INVALID_ARG;
    *bytes = 0;
    if (prefix_len < 0) return SQ_ERR_INVALID_ARG;
    sq_status rc = check_paged_shape(T, Hq, Hkv, D, SQ_CACHE_BF16, 1, 16, 0, 0, Hq * D);
    if (rc != SQ_OK) return rc;
    if (T == 0) return SQ_OK;
    return paged_workspace_bytes(T, Hq, D, prefix_len, bytes);
}

sq_status sq_paged_attention(const float *Q, int64_t ldq, int64_t T, int64_t Hq, int64_t Hkv,
                             int64_t D, const void *k_cache, const void *v_cache, int cache_type,
                             int64_t num_pages, int64_t page_size, const int32_t *block_table,
                             int64_t max_pages, const int32_t *q_start, const int32_t *kv_len,
                             int64_t B, int64_t max_q, const int32_t *prefix_pages,
                             int64_t prefix_len, float scale, float *O, void *workspace,
                             size_t workspace_bytes, void *stream) {
    sq_status rc = check_paged_shape(T, Hq, Hkv, D, cache_type, num_pages, page_size, B,
                                     max_pages, ldq);
    if (rc != SQ_OK) return rc;
    const PagedCall c = {Q,         ldq,         T,         Hq,      Hkv,          D,
                         k_cache,   v_cache,     cache_type, num_pages, page_size,  block_table,
                         max_pages, q_start,     kv_len,    B,       max_q,        prefix_pages,
                         prefix_len, scale,      O,         workspace, nullptr,     nullptr};
    return attention_impl(c, workspace_bytes, stream);
}

sq_status sq_paged_attention_i8(const float *Q, int64_t ldq, int64_t T, int64_t Hq, int64_t Hkv,
                                int64_t D, const int8_t *k_cache, const int8_t *v_cache,
                                const float *k_scale, const float *v_scale, int64_t num_pages,
                                int64_t page_size, const int32_t *block_table, int64_t max_pages,
                                const int32_t *q_start, const int32_t *kv_len, int64_t B,
                                int64_t max_q, const int32_t *prefix_pages, int64_t prefix_len,
                                float scale, float *O, void *workspace, size_t workspace_bytes,
                                void *stream) {
    sq_status rc = check_paged_shape(T, Hq, Hkv, D, SQ_CACHE_BF16, num_pages, page_size, B,
                                     max_pages, ldq);
    if (rc != SQ_OK) return rc;
    const PagedCall c = {Q,         ldq,         T,         Hq,      Hkv,          D,
                         k_cache,   v_cache,     kCacheI8,  num_pages, page_size,  block_table,
                         max_pages, q_start,     kv_len,    B,       max_q,        prefix_pages,
                         prefix_len, scale,      O,         workspace, k_scale,    v_scale};
    return attention_impl(c, workspace_bytes, stream);
}

sq_status sq_linear_i8(const void *Xop, const float *x_scale, const int32_t *x_row_l1,
                       const void *Wop, const float *w_scale, const int32_t *w_row_l1,
                       const float *bias, const float *residual, int64_t M, int64_t N, int64_t K,
                       int mode, void *Y, void *stream) {
    return linear_impl(Xop, x_scale, x_row_l1, Wop, w_scale, w_row_l1, bias, residual, M, N, K,
                       mode, Y, nullptr, 0, stream);
}

sq_status sq_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t *bytes) {
    if (!bytes) return SQ_ERR_INVALID_ARG;
    *bytes = 0;
    if (M < 0 || N < 0 || K <= 0) return SQ_ERR_INVALID_ARG;
    if (K > kMaxK) return SQ_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return SQ_OK;
    return gemm_tc_workspace_bytes(M, N, K, bytes);
}

sq_status sq_linear_i8_ws(const void *Xop, const float *x_scale, const int32_t *x_row_l1,
                          const void *Wop, const float *w_scale, const int32_t *w_row_l1,
                          const float *bias, const float *residual, int64_t M, int64_t N,
                          int64_t K, int mode, void *Y, void *workspace, size_t workspace_bytes,
                          void *stream) {
    return linear_impl(Xop, x_scale, x_row_l1, Wop, w_scale, w_row_l1, bias, residual, M, N, K,
                       mode, Y, workspace, workspace_bytes, stream);
}

sq_status sq_linear_codes_workspace_bytes(int64_t M, int64_t K, size_t *bytes) {
    if (!bytes) return SQ_ERR_INVALID_ARG;
    *bytes = 0;
    if (M < 0 || K <= 0) return SQ_ERR_INVALID_ARG;
    if (K % 16 != 0) return SQ_ERR_ALIGNMENT;
    if (K > kMaxK || M > ((int64_t)1 << 40) / K) return SQ_ERR_UNSUPPORTED;
    *bytes = (size_t)((M * K * 2 + 255) / 256 * 256);
    return SQ_OK;
}

sq_status sq_linear_i8_codes(const int8_t *Xq, const float *x_scale, const int32_t *x_row_l1,
                             const void *Wop, const float *w_scale, const int32_t *w_row_l1,
                             const float *bias, const float *residual, int64_t M, int64_t N,
                             int64_t K, int mode, void *Y, void *workspace, size_t workspace_bytes,
                             void *stream) {
    size_t need = 0;
    sq_status rc = sq_linear_codes_workspace_bytes(M, K, &need);
    if (rc != SQ_OK) return rc;
    if (M > 0 && N > 0) {
        if (!Xq || !workspace) return SQ_ERR_INVALID_ARG;
        if (!aligned16(Xq) || !aligned16(workspace)) return SQ_ERR_ALIGNMENT;
        if (workspace_bytes < need) return SQ_ERR_INVALID_ARG;
    }
    // the operand the codes widen into is the workspace: the checks of sq_linear_i8 on it
    if ((rc = validate_linear(workspace, x_scale, x_row_l1, Wop, w_scale, w_row_l1, bias,
                              residual, M, N, K, mode, Y)) != SQ_OK ||
        M == 0 || N == 0)
        return rc;
    if ((rc = require_gb300()) != SQ_OK) return rc;
    __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(workspace);
    if ((rc = launch_widen_codes(Xq, op, M * K, as_stream(stream))) != SQ_OK) return rc;
    return linear_impl(op, x_scale, x_row_l1, Wop, w_scale, w_row_l1, bias, residual, M, N, K,
                       mode, Y, nullptr, 0, stream);
}

int64_t sq_gated_rows(int64_t F) {
    return F < 0 || F > kMaxGated ? 0 : gated_rows(F);
}

sq_status sq_pack_gated_weight(const float *W_gate, const float *W_up, const float *s, int64_t F,
                               int64_t K, float *w_scale, void *Wop, int32_t *w_row_l1,
                               void *stream) {
    sq_status rc = check_quant_args(W_gate, s, F, K, nullptr, w_scale, Wop);
    if (rc != SQ_OK) return rc;
    if (F > kMaxGated) return SQ_ERR_UNSUPPORTED;
    if (F == 0) return SQ_OK;
    if (!W_up) return SQ_ERR_INVALID_ARG;
    if (!aligned16(W_up) || (w_row_l1 && !aligned4(w_row_l1))) return SQ_ERR_ALIGNMENT;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_pack_gated(W_gate, W_up, s, F, K, w_scale, static_cast<__nv_bfloat16 *>(Wop),
                             w_row_l1, as_stream(stream));
}

sq_status sq_gated_workspace_bytes(int64_t M, int64_t F, int64_t K, size_t *bytes) {
    if (!bytes) return SQ_ERR_INVALID_ARG;
    *bytes = 0;
    if (M < 0 || F < 0 || K <= 0) return SQ_ERR_INVALID_ARG;
    if (F > kMaxGated || K > kMaxK) return SQ_ERR_UNSUPPORTED;
    if (M == 0 || F == 0) return SQ_OK;
    return gemm_tc_workspace_bytes(M, gated_rows(F), K, bytes, true);
}

sq_status sq_linear_i8_gated(const void *Xop, const float *x_scale, const int32_t *x_row_l1,
                             const void *Wop, const float *w_scale, const int32_t *w_row_l1,
                             const float *bias_gate, const float *bias_up, int64_t M, int64_t F,
                             int64_t K, int act, float *Y, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (act < SQ_GATE_SILU || act > SQ_GATE_GELU_TANH) return SQ_ERR_INVALID_ARG;
    sq_status rc = check_linear_args(Xop, x_scale, Wop, w_scale, nullptr, nullptr, M, F, K,
                                     SQ_EPI_NONE, Y);
    if (rc != SQ_OK) return rc;
    if (F > kMaxGated) return SQ_ERR_UNSUPPORTED;
    if (M == 0 || F == 0) return SQ_OK;
    if ((bias_gate && !aligned4(bias_gate)) || (bias_up && !aligned4(bias_up)) ||
        (x_row_l1 && !aligned4(x_row_l1)) || (w_row_l1 && !aligned4(w_row_l1)) ||
        (workspace && !aligned16(workspace)))
        return SQ_ERR_ALIGNMENT;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    constexpr float kLog2e = 1.4426950408889634f;
    GatedOut g = {bias_gate, bias_up, (int)F, act, 1, 0, 0, -kLog2e, 0.0f};
    if (act == SQ_GATE_GELU_TANH) {
        const double two_root = 1.5957691216057308;  // 2 sqrt(2 / pi)
        g.c1 = (float)(-two_root * 1.4426950408889634);
        g.c3 = (float)(-two_root * 1.4426950408889634 * 0.044715);
    }
    return launch_gemm_tc(static_cast<const __nv_bfloat16 *>(Xop), x_scale, x_row_l1,
                          static_cast<const __nv_bfloat16 *>(Wop), w_scale, w_row_l1, nullptr,
                          nullptr, M, gated_rows(F), K, SQ_EPI_NONE, Y, nullptr, workspace,
                          workspace_bytes, as_stream(stream), nullptr, nullptr, &g);
}

sq_status sq_linear_i8_requant(const void *Xop, const float *x_scale, const int32_t *x_row_l1,
                               const void *Wop, const float *w_scale, const int32_t *w_row_l1,
                               const float *bias, const float *residual, int64_t M, int64_t N,
                               int64_t K, int mode, const float *s_next, float scale, int8_t *Yq,
                               void *Yop, float *x_scale_next, void *stream) {
    return requant_impl(Xop, x_scale, x_row_l1, Wop, w_scale, w_row_l1, bias, residual, M, N, K,
                        mode, s_next, scale, Yq, Yop, x_scale_next, nullptr, 0, stream);
}

sq_status sq_linear_i8_requant_ws(const void *Xop, const float *x_scale,
                                  const int32_t *x_row_l1, const void *Wop, const float *w_scale,
                                  const int32_t *w_row_l1, const float *bias,
                                  const float *residual, int64_t M, int64_t N, int64_t K,
                                  int mode, const float *s_next, float scale, int8_t *Yq,
                                  void *Yop, float *x_scale_next, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    return requant_impl(Xop, x_scale, x_row_l1, Wop, w_scale, w_row_l1, bias, residual, M, N, K,
                        mode, s_next, scale, Yq, Yop, x_scale_next, workspace, workspace_bytes,
                        stream);
}

sq_status sq_linear_i8_mma_sync(const int8_t *Xq, const float *x_scale, const int8_t *Wq,
                                const float *w_scale, const float *bias, const float *residual,
                                int64_t M, int64_t N, int64_t K, int mode, void *Y,
                                void *stream) {
    sq_status rc = check_linear_args(Xq, x_scale, Wq, w_scale, bias, residual, M, N, K, mode, Y);
    if (rc != SQ_OK) return rc;
    if (M == 0 || N == 0) return SQ_OK;
    if ((rc = require_sm103()) != SQ_OK) return rc;
    return launch_gemm_mma_sync(Xq, x_scale, Wq, w_scale, bias, residual, M, N, K, mode, Y,
                                as_stream(stream));
}

sq_status sq_check_division(uint32_t b_first, uint32_t b_count, uint32_t a_first,
                            uint32_t a_count, int corrected, unsigned long long *out,
                            void *stream) {
    const uint64_t lim = 1ull << 23;
    if ((uint64_t)b_first + b_count > lim || (uint64_t)a_first + a_count > lim)
        return SQ_ERR_INVALID_ARG;
    if (b_count == 0 || a_count == 0) return SQ_OK;
    if (!out) return SQ_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(out) & 7u) != 0) return SQ_ERR_ALIGNMENT;
    sq_status rc = require_sm103();
    if (rc != SQ_OK) return rc;
    return launch_check_division(b_first, b_count, a_first, a_count, corrected ? 1 : 0, out,
                                 as_stream(stream));
}

sq_status sq_device_status(void *stream) {
    if (cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) return SQ_ERR_CUDA;
    const sq_status rq = quant_take_error(as_stream(stream));
    if (rq == SQ_ERR_CUDA) return rq;
    const sq_status ra = attention_take_error(as_stream(stream));
    if (ra == SQ_ERR_CUDA) return ra;
    const sq_status rp = paged_take_error(as_stream(stream));
    if (rp == SQ_ERR_CUDA) return rp;
    sq_status rc = gemm_tc_take_error(as_stream(stream));
    if (rc == SQ_OK) rc = rp;
    if (rc == SQ_OK) rc = rq;
    if (rc == SQ_OK) rc = ra;
    if (rc == SQ_ERR_TIMEOUT) {
        // a split-K launch that gave up may have left counters in the static
        // scratch: clear them before the next sq_linear_i8_static_ws call
        const sq_status r2 = static_ws_reset_counters(as_stream(stream));
        if (r2 != SQ_OK) return r2;
    }
    return rc;
}

sq_status sq_get_device_status(void *stream) { return sq_device_status(stream); }

}  // extern "C"
