// block_internal.h -- declarations shared by the host checks (block_api.cu) and the kernels of
// the operators around the attention (rotary.cu, gated_norm.cu, gated_norm_backward.cu). Not part of the public C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bsa_block.h"
#include "internal.h"

namespace bsa {

// ------------------------------------------------------------ rotary
// One of Q, K, V. Forward: src -> dst. Backward: src is the arriving gradient, dst the gradient
// written, x the forward's input.
struct HeadsView {
    const char *src, *x;
    char *dst;
    int64_t src_b, src_n, src_h, x_b, x_n, x_h, dst_b, dst_n, dst_h;  // elements
    const float *weight;
    float *dweight;
    int heads;  // 0: absent
};

struct RotaryArgs {
    HeadsView t[3];  // Q, K, V
    const int32_t *positions;
    int64_t pos_batch;
    int dt, B, N, norm;
    float eps;
    bsa_rotary_plan plan;
    float *partial;  // backward: weight gradients' partial sums, [CTA][2][d]
};

constexpr int kRotaryMaxCtas = 1024;  // partial sums that the workspace holds
bsa_status launch_rotary(const RotaryArgs &a, cudaStream_t st);
bsa_status launch_rotary_backward(const RotaryArgs &a, cudaStream_t st);

// ------------------------------------------------------------ gated norm
struct RowsView {
    char *p;
    int64_t b, n;  // elements
};

struct NormArgs {
    bsa_gated_norm_desc d;
    RowsView x, y, h, z;  // forward; backward reads h, y
    RowsView dh, dz, dx, dy;
    char *dgate, *dscale, *dshift;
    float *dpost_w, *dpost_b, *dpre_w, *dpre_b;
    float *partial;  // backward: partial column sums
};

// Backward: the rows are cut into contiguous ranges, one per worker (a CTA). kNormMaxThreads bounds the
// workers, and with them the workspace, whatever the device: 512 threads for each SM, all that the kernel's registers
// leave room for.
constexpr int64_t kNormMaxThreads = 152 * 512;
int64_t gated_norm_max_workers(int64_t rows, int C);
// floats of partial sums per worker: 4 sums of the first group that it shares with others, of the last, and for weights
__host__ __device__ inline int64_t gated_norm_worker_floats(int C) { return int64_t(12) * C; }
bsa_status launch_gated_norm(const NormArgs &a, cudaStream_t st);
bsa_status launch_gated_norm_backward(const NormArgs &a, cudaStream_t st);

}  // namespace bsa
