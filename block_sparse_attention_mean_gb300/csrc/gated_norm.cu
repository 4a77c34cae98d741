// gated_norm.cu -- the step between two sub-blocks of a transformer block: norm of the branch,
// gate, residual add, norm of the sum, scale and shift, in one pass; and its backward pass.
//
//   u = post(y),  h = x + alpha * gate * u,  z = pre(h) * (1 + scale) + shift
//
// A row of C channels is read once into registers, so that mean, variance and result come from one
// reading (the variance from the centred values: no cancellation for rows far from zero), and is
// written once. HBM bounds it.
//
// Split: a row is held by LANES lanes of a warp (rows of up to 32 groups of 8 channels) or by whole
// warps of one CTA, VPT groups of 8 channels per thread; groups are dealt out lane by lane so that
// a warp reads contiguous memory.
#include "block_internal.h"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int kMaxWarps = 32;

__host__ __device__ constexpr int pow2_ceil(int v)
{
    int p = 1;
    while (p < v) p *= 2;
    return p;
}

// Threads that hold a row of `groups` groups of 8 channels, vpt of them per thread
__host__ __device__ inline int row_threads(int groups, int vpt)
{
    return groups <= 32 ? pow2_ceil(groups) : (groups + 32 * vpt - 1) / (32 * vpt) * 32;
}

// Sums of K values over the threads of a row. `lanes`: a power of two up to 32. With several warps per
// row the CTA holds one row, and the warps' sums go through shared memory (two buffers in turn, so
// that one barrier per sum is enough); every thread adds them in the same order.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int lanes, int warps, float (*buf)[2][kMaxWarps], int &turn)
{
    for (int o = lanes / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
    if (warps == 1) return;
    float (*b)[kMaxWarps] = buf[turn];
    turn ^= 1;
    if (threadIdx.x % 32 == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) b[k][threadIdx.x / 32] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float s = 0.0f;
        for (int w = 0; w < warps; ++w) s += b[k][w];
        v[k] = s;
    }
}

// eight channels of a modulation (or of a weight: fp32) as fp32
__device__ __forceinline__ void load_mod(const void *p, int dt, int64_t at, float (&f)[8])
{
    if (dt == BSA_BF16) {
        Vec8<__nv_bfloat16> v;
        v.load(p, at);
        v.unpack(f);
    } else {
        Vec8<float> v;
        v.load(p, at);
        v.unpack(f);
    }
}

// Normalises the row held in v (fp32, zeros in the slots past its end): LAYER subtracts the mean, then both
// divide by the root of the mean square. Returns 1 / the scale.
template <int VPT>
__device__ __forceinline__ float normalise(float (&v)[VPT][8], const bool (&on)[VPT], int kind, float eps, int C, int lanes,
                                           int warps, float (*buf)[2][kMaxWarps], int &turn)
{
    const float inv_c = 1.0f / static_cast<float>(C);
    if (kind == BSA_NORM_LAYER) {
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += v[k][j];
        }
        row_sums<1>(s, lanes, warps, buf, turn);
        const float mean = s[0] * inv_c;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = on[k] ? v[k][j] - mean : 0.0f;
        }
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[0] += v[k][j] * v[k][j];
    }
    row_sums<1>(q, lanes, warps, buf, turn);
    const float r = rsqrtf(q[0] * inv_c + eps);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] *= r;
    }
    return r;
}

// v = v * weight + bias (either may be null)
__device__ __forceinline__ void affine(float (&v)[8], const bsa_norm &n, int c)
{
    float f[8];
    if (n.weight) {
        load_mod(n.weight, BSA_FP32, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= f[j];
    }
    if (n.bias) {
        load_mod(n.bias, BSA_FP32, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
}

template <typename TS, typename TB, int VPT>
__global__ void __launch_bounds__(1024 / VPT) gated_norm_kernel(const __grid_constant__ NormArgs a, int tpr)
{
    __shared__ float buf[2][2][kMaxWarps];
    const bsa_gated_norm_desc &d = a.d;
    const int C = d.C, groups = C / 8;
    const int lanes = min(tpr, 32), warps = (tpr + 31) / 32;
    const int64_t rows = static_cast<int64_t>(d.B) * d.N;
    int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = row < rows;
    if (!live) row = rows - 1;  // shuffles and barriers take every thread
    const int b = static_cast<int>(row / d.N), n = static_cast<int>(row % d.N);
    const int f = n / (d.N / d.F);
    const int t = threadIdx.x % tpr;
    int turn = 0;

    bool on[VPT];
    int c[VPT];
    Vec8<TS> xr[VPT];
    Vec8<TB> yr[VPT];
    const bool branch = a.y.p != nullptr;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        on[k] = t + k * tpr < groups;
        c[k] = on[k] ? 8 * (t + k * tpr) : 0;
        if (on[k]) {
            xr[k].load(a.x.p, b * a.x.b + n * a.x.n + c[k]);
            if (branch) yr[k].load(a.y.p, b * a.y.b + n * a.y.n + c[k]);
        }
    }
    float h[VPT][8];
    if (branch) {
        float u[VPT][8];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) u[k][j] = 0.0f;
            if (on[k]) yr[k].unpack(u[k]);
        }
        if (d.post.kind != BSA_NORM_NONE) normalise<VPT>(u, on, d.post.kind, d.post.eps, C, lanes, warps, buf, turn);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] = 0.0f;
            if (!on[k]) continue;
            affine(u[k], d.post, c[k]);
            xr[k].unpack(h[k]);
            if (d.gate.ptr) {
                float g[8];
                load_mod(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c[k], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[k][j] *= g[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] += d.alpha * u[k][j];
            xr[k].pack(h[k]);
            if (live) xr[k].store(a.h.p, b * a.h.b + n * a.h.n + c[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] = 0.0f;
            if (on[k]) xr[k].unpack(h[k]);
        }
    }
    if (d.pre.kind == BSA_NORM_NONE) return;
    // of h before its rounding: the norm sees the exact sum
    normalise<VPT>(h, on, d.pre.kind, d.pre.eps, C, lanes, warps, buf, turn);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        if (!on[k]) continue;
        affine(h[k], d.pre, c[k]);
        float m[8];
        if (d.scale.ptr) {
            load_mod(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c[k], m);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] *= 1.0f + m[j];
        }
        if (d.shift.ptr) {
            load_mod(d.shift.ptr, d.mod_dt, b * d.shift.batch + f * d.shift.frame + c[k], m);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] += m[j];
        }
        yr[k].pack(h[k]);
        if (live) yr[k].store(a.z.p, b * a.z.b + n * a.z.n + c[k]);
    }
}

// ------------------------------------------------------------ backward
//
// The rows, in order of (batch, token), are cut into equal ranges, one per worker (the threads that hold
// a row). A worker walks its range and keeps four sums per channel in registers,
//   A = sum dz,  S = sum dz n,  P = sum dx,  Q = sum dx m      (m = y without a post norm),
// from which every parameter's gradient follows by factors that are constant over the rows that share a
// modulation (a group):
//   dshift = A,  dscale = w S + b A,  dgate = alpha (w2 Q + b2 P),
//   dpre_weight = sum_g (1 + scale_g) S_g,  dpre_bias = sum_g (1 + scale_g) A_g,
//   dpost_weight = alpha sum_g gate_g Q_g,  dpost_bias = alpha sum_g gate_g P_g.
// At the end of a group the worker writes the group's gradients itself if it held the whole group, else the
// four sums into one of its two slots (groups that its range's ends cut); the weights' sums go on in its
// third. A second kernel adds the slots in the order of the workers, so that results do not depend on timing.

struct Groups {
    int64_t rows, per_group, per_worker;
    int workers;
};

struct Wants {
    bool pre_sums, post_sums, weights;
};

__device__ __forceinline__ Wants wants_of(const NormArgs &a)
{
    Wants w;
    w.pre_sums = a.dscale || a.dshift || a.dpre_w || a.dpre_b;
    w.post_sums = a.dgate || a.dpost_w || a.dpost_b;
    w.weights = a.dpre_w || a.dpre_b || a.dpost_w || a.dpost_b;
    return w;
}

__device__ __forceinline__ void store_mod(char *p, int dt, int64_t at, const float (&f)[8])
{
    if (dt == BSA_BF16) {
        Vec8<__nv_bfloat16> v;
        v.pack(f);
        v.store(p, at);
    } else {
        Vec8<float> v;
        v.pack(f);
        v.store(p, at);
    }
}

// the gradients of a group's modulations from its four sums, at channels c .. c + 7
__device__ __forceinline__ void write_group(const NormArgs &a, int64_t g, int c, const float (&A)[8], const float (&S)[8],
                                            const float (&P)[8], const float (&Q)[8])
{
    const bsa_gated_norm_desc &d = a.d;
    const int64_t at = g * d.C + c;
    if (a.dshift) store_mod(a.dshift, d.mod_dt, at, A);
    float o[8], w[8];
    if (a.dscale) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = S[j];
        if (d.pre.weight) {
            load_mod(d.pre.weight, BSA_FP32, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] *= w[j];
        }
        if (d.pre.bias) {
            load_mod(d.pre.bias, BSA_FP32, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] += w[j] * A[j];
        }
        store_mod(a.dscale, d.mod_dt, at, o);
    }
    if (a.dgate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = Q[j];
        if (d.post.weight) {
            load_mod(d.post.weight, BSA_FP32, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] *= w[j];
        }
        if (d.post.bias) {
            load_mod(d.post.bias, BSA_FP32, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] += w[j] * P[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= d.alpha;
        store_mod(a.dgate, d.mod_dt, at, o);
    }
}

// the four sums of a group, weighted for the parameters that all groups share
__device__ __forceinline__ void weigh_group(const NormArgs &a, int64_t g, int c, float (&A)[8], float (&S)[8], float (&P)[8],
                                            float (&Q)[8])
{
    const bsa_gated_norm_desc &d = a.d;
    const int b = static_cast<int>(g / d.F), f = static_cast<int>(g % d.F);
    float m[8];
    if (d.scale.ptr) {
        load_mod(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            A[j] *= 1.0f + m[j];
            S[j] *= 1.0f + m[j];
        }
    }
    if (d.gate.ptr) {
        load_mod(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            P[j] *= m[j];
            Q[j] *= m[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        P[j] *= d.alpha;
        Q[j] *= d.alpha;
    }
}

template <typename TS, typename TB, int VPT>
__global__ void __launch_bounds__(512) gated_norm_backward_kernel(const __grid_constant__ NormArgs a, Groups gr, int tpr)
{
    __shared__ float buf[2][2][kMaxWarps];
    const bsa_gated_norm_desc &d = a.d;
    const int C = d.C, groups = C / 8;
    const float inv_c = 1.0f / static_cast<float>(C);
    const int lanes = min(tpr, 32), warps = (tpr + 31) / 32;
    const int t = threadIdx.x % tpr;
    const int64_t worker = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    const int64_t first = worker * gr.per_worker, end = min(first + gr.per_worker, gr.rows);
    const Wants want = wants_of(a);
    const bool pre = d.pre.kind != BSA_NORM_NONE, branch = a.dy.p != nullptr;
    const bool need_y = a.y.p != nullptr;
    int turn = 0;

    bool on[VPT];
    int c[VPT];
    float A[VPT][8], S[VPT][8], P[VPT][8], Q[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        on[k] = t + k * tpr < groups;
        c[k] = on[k] ? 8 * (t + k * tpr) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) A[k][j] = S[k][j] = P[k][j] = Q[k][j] = 0.0f;
    }
    float *const slots = a.partial + worker * gated_norm_worker_floats(C);
    bool weighed = false;  // the worker's third slot holds sums

    for (int64_t i = 0; i < gr.per_worker; ++i) {
        // a worker past its range (or past all rows) goes on with the last row, writing nothing:
        // shuffles and barriers take every thread
        const bool live = first + i < end;
        const int64_t row = min(first + i, gr.rows - 1);
        const int b = static_cast<int>(row / d.N), n = static_cast<int>(row % d.N);
        const int f = n / static_cast<int>(gr.per_group);
        Vec8<TS> hr[VPT], dhr[VPT];
        Vec8<TB> yr[VPT], dzr[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!on[k]) continue;
            if (pre) {
                hr[k].load(a.h.p, b * a.h.b + n * a.h.n + c[k]);
                dzr[k].load(a.dz.p, b * a.dz.b + n * a.dz.n + c[k]);
            }
            if (a.dh.p) dhr[k].load(a.dh.p, b * a.dh.b + n * a.dh.n + c[k]);
            if (need_y) yr[k].load(a.y.p, b * a.y.b + n * a.y.n + c[k]);
        }
        float g[VPT][8];  // the gradient at h
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[k][j] = 0.0f;
            if (on[k] && a.dh.p) dhr[k].unpack(g[k]);
        }
        if (pre) {
            float v[VPT][8], q[VPT][8];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[k][j] = q[k][j] = 0.0f;
                if (on[k]) hr[k].unpack(v[k]);
            }
            const float r = normalise<VPT>(v, on, d.pre.kind, d.pre.eps, C, lanes, warps, buf, turn);
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (!on[k]) continue;
                dzr[k].unpack(q[k]);
                if (want.pre_sums && live) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        A[k][j] += q[k][j];
                        S[k][j] += q[k][j] * v[k][j];
                    }
                }
                float m[8];
                if (d.scale.ptr) {
                    load_mod(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c[k], m);
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[k][j] *= 1.0f + m[j];
                }
                if (d.pre.weight) {
                    load_mod(d.pre.weight, BSA_FP32, c[k], m);
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[k][j] *= m[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[0] += q[k][j] * v[k][j];
                    s[1] += q[k][j];
                }
            }
            row_sums<2>(s, lanes, warps, buf, turn);
            const float along = s[0] * inv_c, mean = d.pre.kind == BSA_NORM_LAYER ? s[1] * inv_c : 0.0f;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
#pragma unroll
                for (int j = 0; j < 8; ++j) g[k][j] += on[k] ? r * (q[k][j] - mean - v[k][j] * along) : 0.0f;
            }
        }
        if (a.dx.p && live) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (!on[k]) continue;
                dhr[k].pack(g[k]);
                dhr[k].store(a.dx.p, b * a.dx.b + n * a.dx.n + c[k]);
            }
        }
        if (need_y) {
            float v[VPT][8];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
                if (on[k]) yr[k].unpack(v[k]);
            }
            float r = 1.0f;
            if (d.post.kind != BSA_NORM_NONE) r = normalise<VPT>(v, on, d.post.kind, d.post.eps, C, lanes, warps, buf, turn);
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (!on[k]) continue;
                if (want.post_sums && live) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        P[k][j] += g[k][j];
                        Q[k][j] += g[k][j] * v[k][j];
                    }
                }
                float m[8];
                if (d.gate.ptr) {
                    load_mod(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c[k], m);
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[k][j] *= m[j];
                }
                if (d.post.weight) {
                    load_mod(d.post.weight, BSA_FP32, c[k], m);
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[k][j] *= m[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    g[k][j] *= d.alpha;
                    s[0] += g[k][j] * v[k][j];
                    s[1] += g[k][j];
                }
            }
            if (branch) {
                float along = 0.0f, mean = 0.0f;
                if (d.post.kind != BSA_NORM_NONE) {
                    row_sums<2>(s, lanes, warps, buf, turn);
                    along = s[0] * inv_c;
                    mean = d.post.kind == BSA_NORM_LAYER ? s[1] * inv_c : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    if (!on[k] || !live) continue;
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[k][j] = r * (g[k][j] - mean - v[k][j] * along);
                    yr[k].pack(g[k]);
                    yr[k].store(a.dy.p, b * a.dy.b + n * a.dy.n + c[k]);
                }
            }
        }
        // the end of a group, or of the range
        if (!live || (!want.pre_sums && !want.post_sums)) continue;
        const int64_t group = row / gr.per_group;
        if (row + 1 != end && (row + 1) % gr.per_group != 0) continue;
        const bool whole = group * gr.per_group >= first && (group + 1) * gr.per_group <= end;
        float *const slot = slots + (group == first / gr.per_group ? 0 : 4 * C);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!on[k]) continue;
            float(*const sums[4])[8] = {&A[k], &S[k], &P[k], &Q[k]};
            if (whole) {
                write_group(a, group, c[k], A[k], S[k], P[k], Q[k]);
            } else {
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    Vec8<float> o;
                    o.pack(*sums[i4]);
                    o.store(slot, i4 * C + c[k]);
                }
            }
            if (want.weights) {
                weigh_group(a, group, c[k], A[k], S[k], P[k], Q[k]);
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    Vec8<float> o;
                    if (weighed) {
                        float before[8];
                        o.load(slots, (8 + i4) * C + c[k]);
                        o.unpack(before);
#pragma unroll
                        for (int j = 0; j < 8; ++j) (*sums[i4])[j] += before[j];
                    }
                    o.pack(*sums[i4]);
                    o.store(slots, (8 + i4) * C + c[k]);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) A[k][j] = S[k][j] = P[k][j] = Q[k][j] = 0.0f;
        }
        weighed = true;
    }
}

// Adds the workers' slots, 32 channels per CTA, kSumSlices slices of the workers each. blockIdx.y == 0: the
// weights' sums over all workers; blockIdx.y > 0: one group that several workers share.
constexpr int kSumSlices = 32;

__global__ void __launch_bounds__(32 * kSumSlices) gated_norm_sums_kernel(const __grid_constant__ NormArgs a, Groups gr,
                                                                          int64_t n_groups)
{
    __shared__ float part[kSumSlices][32][5];
    grid_dependency_wait();
    const bsa_gated_norm_desc &d = a.d;
    const int C = d.C;
    const int64_t stride = gated_norm_worker_floats(C);
    const Wants want = wants_of(a);
    int64_t w0 = 0, w1 = gr.workers - 1, group = -1;
    if (blockIdx.y == 0) {
        if (!want.weights) return;
    } else {
        // the group itself where there are at most as many groups as workers; else the one that worker y - 1's
        // range begins inside
        const int64_t i = blockIdx.y - 1;
        group = n_groups <= gr.workers ? i : i * gr.per_worker / gr.per_group;
        w0 = group * gr.per_group / gr.per_worker;
        w1 = ((group + 1) * gr.per_group - 1) / gr.per_worker;
        if (w0 == w1) return;                              // written by its worker
        if (n_groups > gr.workers && i != w0 + 1) return;  // one CTA per group
    }
    const int c = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < C) {
        for (int64_t w = w0 + slice; w <= w1; w += kSumSlices) {
            const int slot = group < 0 ? 8 : (w * gr.per_worker / gr.per_group == group ? 0 : 4);
            const float *p = a.partial + w * stride + slot * C + c;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += p[k * C];
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) part[slice][threadIdx.x % 32][k] = v[k];
    __syncthreads();
    if (slice != 0 || c >= C) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[k] = 0.0f;
        for (int i = 0; i < kSumSlices; ++i) v[k] += part[i][threadIdx.x][k];
    }
    if (group < 0) {
        if (a.dpre_b) a.dpre_b[c] = v[0];
        if (a.dpre_w) a.dpre_w[c] = v[1];
        if (a.dpost_b) a.dpost_b[c] = v[2];
        if (a.dpost_w) a.dpost_w[c] = v[3];
        return;
    }
    auto put = [&](char *p, float x) {
        const int64_t at = group * C + c;
        if (d.mod_dt == BSA_BF16)
            reinterpret_cast<__nv_bfloat16 *>(p)[at] = __float2bfloat16_rn(x);
        else
            reinterpret_cast<float *>(p)[at] = x;
    };
    auto by = [&](const float *w, float one, float x) { return (w ? w[c] : one) * x; };
    if (a.dshift) put(a.dshift, v[0]);
    if (a.dscale) put(a.dscale, by(d.pre.weight, 1.0f, v[1]) + by(d.pre.bias, 0.0f, v[0]));
    if (a.dgate) put(a.dgate, d.alpha * (by(d.post.weight, 1.0f, v[3]) + by(d.post.bias, 0.0f, v[2])));
}

template <typename F>
bsa_status by_types(const bsa_gated_norm_desc &d, F &&run)
{
    if (d.stream_dt == BSA_BF16) return run(__nv_bfloat16(), __nv_bfloat16());
    if (d.branch_dt == BSA_BF16) return run(float(), __nv_bfloat16());
    return run(float(), float());
}

template <typename TS, typename TB, int VPT>
bsa_status forward(const NormArgs &a, cudaStream_t st)
{
    const int tpr = row_threads(a.d.C / 8, VPT);
    const int threads = tpr <= 32 ? 128 : tpr;
    const int64_t rows = static_cast<int64_t>(a.d.B) * a.d.N, per_cta = threads / tpr;
    gated_norm_kernel<TS, TB, VPT><<<static_cast<unsigned>((rows + per_cta - 1) / per_cta), threads, 0, st>>>(a, tpr);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

// vectors per thread of the backward kernel, whose CTAs have up to 512 threads
int backward_vpt(int C) { return C > 4096 ? 2 : 1; }

template <typename TS, typename TB, int VPT>
bsa_status backward(const NormArgs &a, int sms, cudaStream_t st)
{
    const int tpr = row_threads(a.d.C / 8, VPT);
    const int threads = tpr <= 32 ? 128 : tpr;
    Groups gr;
    gr.rows = static_cast<int64_t>(a.d.B) * a.d.N;
    gr.per_group = a.d.N / a.d.F;
    int64_t workers = gated_norm_max_workers(gr.rows, a.d.C);
    const int64_t fill = static_cast<int64_t>(sms) * 512 / tpr;  // 512 threads per SM
    if (workers > fill && fill > 0) workers = fill;
    gr.per_worker = (gr.rows + workers - 1) / workers;
    gr.workers = static_cast<int>((gr.rows + gr.per_worker - 1) / gr.per_worker);
    const int per_cta = threads / tpr;
    gated_norm_backward_kernel<TS, TB, VPT>
        <<<(gr.workers + per_cta - 1) / per_cta, threads, 0, st>>>(a, gr, tpr);
    if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
    if (a.partial == nullptr) return BSA_OK;
    const int64_t n_groups = static_cast<int64_t>(a.d.B) * a.d.F;
    const int64_t items = n_groups < gr.workers ? n_groups : gr.workers;
    const dim3 grid((a.d.C + 31) / 32, static_cast<unsigned>(items + 1));
    return pdl_launch(gated_norm_sums_kernel, grid, 32 * kSumSlices, 0, st, a, gr, n_groups) ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace

int64_t gated_norm_max_workers(int64_t rows, int C)
{
    const int64_t w = kNormMaxThreads / row_threads(C / 8, backward_vpt(C));
    return rows < w ? rows : w;
}

bsa_status launch_gated_norm(const NormArgs &a, cudaStream_t st)
{
    return by_types(a.d, [&](auto s, auto b) { return forward<decltype(s), decltype(b), 2>(a, st); });
}

bsa_status launch_gated_norm_backward(const NormArgs &a, cudaStream_t st)
{
    int sms = 0;
    const bsa_status s = current_sm_count(&sms);
    if (s != BSA_OK) return s;
    return by_types(a.d, [&](auto ts, auto tb) {
        return backward_vpt(a.d.C) == 2 ? backward<decltype(ts), decltype(tb), 2>(a, sms, st)
                                        : backward<decltype(ts), decltype(tb), 1>(a, sms, st);
    });
}

}  // namespace bsa
