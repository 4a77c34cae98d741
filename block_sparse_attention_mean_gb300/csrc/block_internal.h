// block_internal.h -- declarations shared by the host checks (block_api.cu) and the kernels of
// the operators around the attention (rotary.cu, gated_norm.cu). Not part of the public C ABI.
#pragma once

#include <cuda_bf16.h>
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
    uint32_t *tickets;  // behind them: how many CTAs are done with 32 channels (zeroed by the first kernel)
};

// Backward: the rows are cut into contiguous ranges, one per worker (a CTA). kNormMaxThreads bounds the
// workers, and with them the workspace, whatever the device.
constexpr int64_t kNormMaxThreads = 152 * 512;
int64_t gated_norm_max_workers(int64_t rows, int C);
// floats of partial sums per worker: two unfinished groups of 4 sums, and 4 sums for weights
__host__ __device__ inline int64_t gated_norm_worker_floats(int C) { return int64_t(12) * C; }
constexpr int kNormTickets = 256;
bsa_status launch_gated_norm(const NormArgs &a, cudaStream_t st);
bsa_status launch_gated_norm_backward(const NormArgs &a, cudaStream_t st);

// ------------------------------------------------------------ eight channels of a row
// The unit of the row kernels: 16 bytes of bf16, 32 bytes of fp32, kept raw until used so that
// loads in flight cost few registers.
template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const void *base, int64_t elem)
    {
        r = *reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + elem * 2);
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // round to nearest even: half a bf16 step per element
    __device__ __forceinline__ void pack(const float (&f)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store(void *base, int64_t elem) const
    {
        *reinterpret_cast<uint4 *>(static_cast<char *>(base) + elem * 2) = r;
    }
};

template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *base, int64_t elem)
    {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const char *>(base) + elem * 4);
        a = p[0];
        b = p[1];
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const
    {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    __device__ __forceinline__ void pack(const float (&f)[8])
    {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ void store(void *base, int64_t elem) const
    {
        float4 *p = reinterpret_cast<float4 *>(static_cast<char *>(base) + elem * 4);
        p[0] = a;
        p[1] = b;
    }
};

}  // namespace bsa
