// The gated feed-forward block's linear: both projections are one operand, whose rows
// alternate in blocks, so that an epilogue warp finds a gate's column and the one it is
// multiplied with in two neighbouring slices of its own accumulators.
#pragma once
#include "common.cuh"

namespace sq {

// Rows of the gate's weights in a row of the packed operand, then as many of the other
// projection's: an epilogue slice's columns.
constexpr int kGatedBlock = 32;

// Rows of the packed operand for F outputs: the last block of each side is filled with
// rows of zeros.
constexpr int64_t gated_rows(int64_t F) {
    return (F + kGatedBlock - 1) / kGatedBlock * (2 * kGatedBlock);
}

struct GatedOut {
    const float *bias_gate, *bias_up;  // [F], nullable
    int F;
    int act;       // sq_gate
    int group;     // row blocks that share a pass over the weights (grouped_item_at)
    int tile_n;    // columns of a whole tile (plan_gated)
    int a_rows;    // rows of a copy of the activations (gemm_tc_kernel)
    float c1, c3;  // the logistic function's argument, times -log2 e (see sigmoid_gate2)
};

// W_gate, W_up fp32 [F][K] -> the packed operand, its rows' scales and L1 norms
// (nullable), each row as sq_pack_weight makes it.
sq_status launch_pack_gated(const float *W_gate, const float *W_up, const float *s, int64_t F,
                            int64_t K, float *w_scale, __nv_bfloat16 *Wop, int32_t *l1,
                            cudaStream_t st);

}  // namespace sq
