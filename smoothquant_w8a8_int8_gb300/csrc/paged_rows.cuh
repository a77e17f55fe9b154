// Shared parts of the attention kernels for few query rows (16-bit and int8 caches):
// the warp-level tensor instruction, its operands' parts, and the order of launches.
#pragma once
#include "paged.cuh"

namespace sq {
namespace {

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The instruction's operand sets for rows of which each thread holds RPT (ROWS
// / 8) pairs of elements: N parts of ROWS = 8 rows in (N + 1) / 2 sets, of 16
// rows in N sets.
template <bool BF, int ROWS>
struct Parts {
    static constexpr int kParts = BF ? 3 : 2;
    static constexpr int kSets = ROWS == 8 ? (kParts + 1) / 2 : kParts;
    static constexpr int kRows = ROWS / 8;
    // registers r and r + 1 of every set (rows 0-7 and 8-15) from this thread's
    // pairs (x[row][0], x[row][1])
    static __device__ __forceinline__ void fill(const float (&x)[kRows][2], int r,
                                                uint32_t (&f)[kSets][4]) {
        uint32_t w[kRows][kParts];
#pragma unroll
        for (int i = 0; i < kRows; ++i) split16<BF, kParts>(x[i][0], x[i][1], w[i]);
        if (ROWS == 8) {
            f[0][r] = w[0][0];
            f[0][r + 1] = w[0][1];
            if (kSets > 1) {
                f[kSets - 1][r] = w[0][kParts - 1];
                f[kSets - 1][r + 1] = 0;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSets; ++j) {
                f[j][r] = w[0][j];
                f[j][r + 1] = w[kRows - 1][j];
            }
        }
    }
};

// The order of launches.  The prefix's launch, of either kernel, lets the next one
// start only when the kernels before it are complete, so that the launch behind it
// (after_prefix) need not wait for them, but for the prefix's state and the workspace
// alone (end_of_prefix, in front of the first access to either); its first copies
// are on their way meanwhile: 4 us less of 70 to 140.  (The kernel for many rows
// gains nothing: 117 us either way.)
__device__ __forceinline__ void begin_rows(const PagedArgs &a) {
    if (!a.prefix_phase) pdl_launch_dependents();
    if (!a.after_prefix) pdl_wait();  // the accesses below follow the previous kernel
    if (a.prefix_phase) pdl_launch_dependents();
}
__device__ __forceinline__ void end_of_prefix(const PagedArgs &a) {
    if (a.after_prefix) pdl_wait();
}

}  // namespace
}  // namespace sq
