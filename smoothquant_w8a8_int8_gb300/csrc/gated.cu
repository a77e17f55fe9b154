// Packing of a gated block's two weight matrices into one operand (offline).
//
// Row p of the operand is row f of the gate's weights or of the other projection's,
// blocks of kGatedBlock rows in turn; per row, as sq_pack_weight has it,
//   w'_j = RN(w_j s_j),  scale = RN(max |w'_j| / 127) (1 for a row of zeros),
//   code_j = clamp(round_half_even(RN(w'_j / scale)), +-127).
// Once a layer, so it is as simple as it can be: a block per row, which reads it twice.
#include "gated.cuh"

namespace sq {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) pack_gated_kernel(
    const float *__restrict__ W_gate, const float *__restrict__ W_up, const float *__restrict__ s,
    int64_t F, int64_t K, float *__restrict__ w_scale, __nv_bfloat16 *__restrict__ Wop,
    int32_t *__restrict__ l1) {
    __shared__ float warp_max[kThreads / 32];
    __shared__ long long warp_l1[kThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t p = blockIdx.x;
    const int64_t f = p / (2 * kGatedBlock) * kGatedBlock + p % kGatedBlock;
    const float *w = (p & kGatedBlock ? W_up : W_gate) + f * K;
    const bool real = f < F;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float top = 0.0f;
    for (int64_t j = threadIdx.x; real && j < K; j += kThreads)
        top = fmaxf(top, fabsf(__fmul_rn(w[j], s[j])));
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) warp_max[warp] = top;
    __syncthreads();
    for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, warp_max[i]);
    const float scale = top == 0.0f ? 1.0f : __fdiv_rn(top, 127.0f);
    int sum = 0;
    for (int64_t j = threadIdx.x; j < K; j += kThreads) {
        float c = 0.0f;
        if (real) {
            c = rintf(__fdiv_rn(__fmul_rn(w[j], s[j]), scale));
            c = fminf(fmaxf(c, -127.0f), 127.0f);
        }
        Wop[p * K + j] = __float2bfloat16_rn(c);
        sum += abs(__float2int_rn(c));
    }
    // (a thread's part fits 32 bits, K being 2^30 at most; a row's norm may not)
    long long norm = sum;
    for (int o = 16; o > 0; o >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, o);
    if (lane == 0) warp_l1[warp] = norm;
    __syncthreads();
    if (threadIdx.x == 0) {
        w_scale[p] = scale;
        if (l1) {
            norm = 0;
            for (int i = 0; i < kThreads / 32; ++i) norm += warp_l1[i];
            l1[p] = norm > 0x7fffffffLL ? 0x7fffffff : (int32_t)norm;
        }
    }
}

}  // namespace

sq_status launch_pack_gated(const float *W_gate, const float *W_up, const float *s, int64_t F,
                            int64_t K, float *w_scale, __nv_bfloat16 *Wop, int32_t *l1,
                            cudaStream_t st) {
    return launch_pdl(pack_gated_kernel, dim3((unsigned)gated_rows(F)), dim3(kThreads), 0, st, 1,
                      W_gate, W_up, s, F, K, w_scale, Wop, l1);
}

}  // namespace sq
