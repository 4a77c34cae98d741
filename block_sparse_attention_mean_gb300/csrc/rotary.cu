// rotary.cu -- rotary positions with several axes, the per-head RMS norm of Q and K, and the
// change from the projection's layout to the attention's, in one pass; and its backward pass.
//
// Per token n, head and channel pair (a, b) of axis s:
//   u = x * rsqrt(mean x^2 + eps) * w,  t = pos[n][s] * f,
//   y_a = u_a cos t - u_b sin t,  y_b = u_b cos t + u_a sin t.
// Each element is read once and written once and takes about ten operations: HBM bounds it.
//
// Split: d / 16 threads hold one head of one token, 16 channels (8 pairs) each, and walk over
// the heads of that token, so that a thread's eight angles, the one costly part, are computed
// once for many heads.
//
// Angles: frequencies are 64-bit fixed point in turns, so pos * f modulo one turn is the low
// 64 bits of an integer product. Its top 32 bits, as a signed fraction of half turns, go to
// sincospif in fp32: the angle is off by at most 2^-25 half turns whatever the position,
// without fp64 or a slow argument reduction.
#include "block_internal.h"
#include "ptx.cuh"

#include <type_traits>

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // heads in flight per thread, forward

// Where a thread's two groups of 8 channels start, and how many of its 8 pairs turn.
struct Lane {
    int c0, c1, nrot;
};

template <bool HALVES>
__device__ __forceinline__ Lane lane_of(int t, int rot)
{
    Lane l;
    l.nrot = min(8, max(0, rot / 2 - 8 * t));
    const bool halves = HALVES && l.nrot > 0;  // rot / 2 is a multiple of 8: all eight turn, or none
    l.c0 = halves ? 8 * t : 16 * t;
    l.c1 = halves ? rot / 2 + 8 * t : 16 * t + 8;
    return l;
}

__device__ __forceinline__ void angles(const bsa_rotary_plan &plan, const int32_t *pos, int t, int nrot,
                                       float (&cs)[8], float (&sn)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        cs[j] = 1.0f;
        sn[j] = 0.0f;
        if (j < nrot) {
            const uint64_t ph = plan.turns[8 * t + j] * static_cast<uint64_t>(static_cast<int64_t>(pos[plan.axis[8 * t + j]]));
            const float half_turns = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 4.656612873077393e-10f;  // 2^-31
            sincospif(half_turns, &sn[j], &cs[j]);
        }
    }
}

// Turns the 16 channels of a thread by its angles (DIR = 1) or back (DIR = -1). Channels that do not
// turn pass through as they are (no product with zero: an infinity stays one).
template <bool HALVES, int DIR>
__device__ __forceinline__ void turn(float (&u0)[8], float (&u1)[8], const float (&cs)[8], const float (&sn)[8], int nrot)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float &a = HALVES ? u0[j] : (j < 4 ? u0[2 * j] : u1[2 * j - 8]);
        float &b = HALVES ? u1[j] : (j < 4 ? u0[2 * j + 1] : u1[2 * j - 7]);
        const float s = DIR * sn[j];
        const float ya = a * cs[j] - b * s, yb = b * cs[j] + a * s;
        if (j < nrot) {
            a = ya;
            b = yb;
        }
    }
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void load_weight(const float *w, int c, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = w ? w[c + i] : 1.0f;
}

// Grid: x over tiles of tokens, y over runs of `per` of the token's heads (Q's, then K's, then V's).
template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a, int per)
{
    constexpr int LANES = D / 16;
    const int t = threadIdx.x % LANES;
    const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
    int64_t token = static_cast<int64_t>(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
    const bool live = token < tokens;
    if (!live) token = tokens - 1;  // shuffles below take whole warps
    const int b = static_cast<int>(token / a.N), n = static_cast<int>(token % a.N);
    const Lane l = lane_of<HALVES>(t, a.plan.rot);

    int lo = blockIdx.y * per, hi = lo + per;
    const int turning = a.t[0].heads + a.t[1].heads;
    float cs[8], sn[8];
    if (lo < turning) angles(a.plan, a.positions + b * a.pos_batch + static_cast<int64_t>(n) * a.plan.n_axes, t, l.nrot, cs, sn);

#pragma unroll
    for (int s = 0; s < 3; ++s) {
        const HeadsView &v = a.t[s];
        const int h0 = max(lo, 0), h1 = min(hi, v.heads);
        lo -= v.heads;
        hi -= v.heads;
        if (h0 >= h1) continue;
        const char *src = v.src + (b * v.src_b + n * v.src_n) * sizeof(T);
        char *dst = v.dst + (b * v.dst_b + n * v.dst_n) * sizeof(T);
        float w0[8], w1[8];
        const bool norm = s < 2 && a.norm;
        if (norm) {
            load_weight(v.weight, l.c0, w0);
            load_weight(v.weight, l.c1, w1);
        }
        for (int h = h0; h < h1; h += kUnroll) {
            Vec8<T> r0[kUnroll], r1[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int hh = min(h + i, h1 - 1);
                r0[i].load(src, hh * v.src_h + l.c0);
                r1[i].load(src, hh * v.src_h + l.c1);
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (s < 2) {
                    float u0[8], u1[8];
                    r0[i].unpack(u0);
                    r1[i].unpack(u1);
                    if (norm) {
                        float ss = 0.0f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) ss += u0[j] * u0[j] + u1[j] * u1[j];
                        const float r = rsqrtf(lanes_sum<LANES>(ss) * (1.0f / D) + a.eps);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            u0[j] *= r * w0[j];
                            u1[j] *= r * w1[j];
                        }
                    }
                    turn<HALVES, 1>(u0, u1, cs, sn, l.nrot);
                    r0[i].pack(u0);
                    r1[i].pack(u1);
                }
                if (live && h + i < h1) {
                    r0[i].store(dst, (h + i) * v.dst_h + l.c0);
                    r1[i].store(dst, (h + i) * v.dst_h + l.c1);
                }
            }
        }
    }
}

// Backward. A CTA takes the work items (tile of tokens, run of heads) blockIdx.x, + gridDim.x, ...;
// its threads keep the weight gradients of their 16 channels in registers over all of them.
template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads) rotary_backward_kernel(const __grid_constant__ RotaryArgs a, int per, int runs,
                                                                   int64_t items)
{
    constexpr int LANES = D / 16, TOKENS = kThreads / LANES;
    const int t = threadIdx.x % LANES;
    const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
    const Lane l = lane_of<HALVES>(t, a.plan.rot);
    float dw[2][16] = {};

    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        int64_t token = item / runs * TOKENS + threadIdx.x / LANES;
        const bool live = token < tokens;
        if (!live) token = tokens - 1;
        const int b = static_cast<int>(token / a.N), n = static_cast<int>(token % a.N);
        int lo = static_cast<int>(item % runs) * per, hi = lo + per;
        float cs[8], sn[8];
        if (lo < a.t[0].heads + a.t[1].heads)
            angles(a.plan, a.positions + b * a.pos_batch + static_cast<int64_t>(n) * a.plan.n_axes, t, l.nrot, cs, sn);
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            const HeadsView &v = a.t[s];
            const int h0 = max(lo, 0), h1 = min(hi, v.heads);
            lo -= v.heads;
            hi -= v.heads;
            if (h0 >= h1) continue;
            const char *src = v.src + (b * v.src_b + n * v.src_n) * sizeof(T);
            const char *x = v.x + (b * v.x_b + n * v.x_n) * sizeof(T);
            char *dst = v.dst + (b * v.dst_b + n * v.dst_n) * sizeof(T);
            float w0[8], w1[8];
            const bool norm = s < 2 && a.norm;
            if (norm) {
                load_weight(v.weight, l.c0, w0);
                load_weight(v.weight, l.c1, w1);
            }
            for (int h = h0; h < h1; h += 2) {
                Vec8<T> g0[2], g1[2], x0[2], x1[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int hh = min(h + i, h1 - 1);
                    g0[i].load(src, hh * v.src_h + l.c0);
                    g1[i].load(src, hh * v.src_h + l.c1);
                    if (norm) {
                        x0[i].load(x, hh * v.x_h + l.c0);
                        x1[i].load(x, hh * v.x_h + l.c1);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool write = live && h + i < h1;
                    if (s < 2) {
                        float u0[8], u1[8];
                        g0[i].unpack(u0);
                        g1[i].unpack(u1);
                        turn<HALVES, -1>(u0, u1, cs, sn, l.nrot);
                        if (norm) {
                            float y0[8], y1[8];
                            x0[i].unpack(y0);
                            x1[i].unpack(y1);
                            float ss = 0.0f, sv = 0.0f;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                ss += y0[j] * y0[j] + y1[j] * y1[j];
                                sv += u0[j] * w0[j] * y0[j] + u1[j] * w1[j] * y1[j];
                            }
                            const float r = rsqrtf(lanes_sum<LANES>(ss) * (1.0f / D) + a.eps);
                            const float m = lanes_sum<LANES>(sv) * (1.0f / D) * r * r;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if (write) {
                                    dw[s][j] += u0[j] * y0[j] * r;
                                    dw[s][8 + j] += u1[j] * y1[j] * r;
                                }
                                u0[j] = r * (u0[j] * w0[j] - y0[j] * m);
                                u1[j] = r * (u1[j] * w1[j] - y1[j] * m);
                            }
                        }
                        g0[i].pack(u0);
                        g1[i].pack(u1);
                    }
                    if (write) {
                        g0[i].store(dst, (h + i) * v.dst_h + l.c0);
                        g1[i].store(dst, (h + i) * v.dst_h + l.c1);
                    }
                }
            }
        }
    }

    if (a.partial == nullptr) return;
    // the CTA's sums per channel: over the warp's tokens by shuffles, over the warps in order
    __shared__ float sums[kThreads / 32][2][D];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float v = dw[s][j];
#pragma unroll
            for (int o = LANES; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (threadIdx.x % 32 < LANES) sums[threadIdx.x / 32][s][(j < 8 ? l.c0 : l.c1 - 8) + j] = v;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) v += sums[w][i / D][i % D];
        a.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = v;
    }
}

// dweight[c] = sum of the CTAs' partial sums: 32 channels per CTA, 32 slices of the CTAs each
__global__ void __launch_bounds__(1024) rotary_dweight_kernel(const float *partial, int ctas, int d, float *dwq, float *dwk)
{
    __shared__ float sums[32][33];
    grid_dependency_wait();
    const int c = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
    float v = 0.0f;
    for (int i = slice; i < ctas; i += 32) v += partial[static_cast<int64_t>(i) * 2 * d + c];
    sums[slice][threadIdx.x % 32] = v;
    __syncthreads();
    if (slice != 0) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][threadIdx.x];
    float *out = c < d ? dwq : dwk;
    if (out) out[c % d] = v;
}

// Heads per run: enough runs that every SM has its threads, a multiple of the unroll.
int heads_per_run(int64_t tiles, int heads, int sms, int unroll)
{
    const int64_t want = static_cast<int64_t>(sms) * (2048 / kThreads);
    const int64_t runs = (want + tiles - 1) / tiles;
    const int per = static_cast<int>((heads + runs - 1) / runs);
    return (per + unroll - 1) / unroll * unroll;
}

template <typename T, int D, bool HALVES>
bsa_status forward(const RotaryArgs &a, int sms, cudaStream_t st)
{
    const int tokens = kThreads / (D / 16);
    const int64_t tiles = (static_cast<int64_t>(a.B) * a.N + tokens - 1) / tokens;
    const int heads = a.t[0].heads + a.t[1].heads + a.t[2].heads;
    const int per = heads_per_run(tiles, heads, sms, kUnroll);
    const dim3 grid(static_cast<unsigned>(tiles), (heads + per - 1) / per);
    rotary_kernel<T, D, HALVES><<<grid, kThreads, 0, st>>>(a, per);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <typename T, int D, bool HALVES>
bsa_status backward(const RotaryArgs &a, int sms, cudaStream_t st)
{
    const int tokens = kThreads / (D / 16);
    const int64_t tiles = (static_cast<int64_t>(a.B) * a.N + tokens - 1) / tokens;
    const int heads = a.t[0].heads + a.t[1].heads + a.t[2].heads;
    const int per = heads_per_run(tiles, heads, sms, 2);
    const int runs = (heads + per - 1) / per;
    const int64_t items = tiles * runs;
    int64_t ctas = static_cast<int64_t>(sms) * 4;
    if (ctas > kRotaryMaxCtas) ctas = kRotaryMaxCtas;
    if (ctas > items) ctas = items;
    rotary_backward_kernel<T, D, HALVES><<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(a, per, runs, items);
    if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
    if (a.partial && !pdl_launch(rotary_dweight_kernel, dim3(2 * D / 32), 1024, 0, st, a.partial, static_cast<int>(ctas), D,
                                 a.t[0].dweight, a.t[1].dweight))
        return BSA_ERR_CUDA;
    return BSA_OK;
}

template <typename F>
bsa_status by_shape(const RotaryArgs &a, F &&run)
{
    const bool halves = a.plan.pairing == BSA_ROTARY_HALVES;
    auto by_d = [&](auto type) {
        using T = decltype(type);
        if (a.plan.d == 64) return halves ? run(T(), std::integral_constant<int, 64>(), std::true_type())
                                          : run(T(), std::integral_constant<int, 64>(), std::false_type());
        return halves ? run(T(), std::integral_constant<int, 128>(), std::true_type())
                      : run(T(), std::integral_constant<int, 128>(), std::false_type());
    };
    return a.dt == BSA_BF16 ? by_d(__nv_bfloat16()) : by_d(float());
}

}  // namespace

bsa_status launch_rotary(const RotaryArgs &a, cudaStream_t st)
{
    int sms = 0;
    const bsa_status s = current_sm_count(&sms);
    if (s != BSA_OK) return s;
    return by_shape(a, [&](auto t, auto d, auto halves) {
        return forward<decltype(t), decltype(d)::value, decltype(halves)::value>(a, sms, st);
    });
}

bsa_status launch_rotary_backward(const RotaryArgs &a, cudaStream_t st)
{
    int sms = 0;
    const bsa_status s = current_sm_count(&sms);
    if (s != BSA_OK) return s;
    return by_shape(a, [&](auto t, auto d, auto halves) {
        return backward<decltype(t), decltype(d)::value, decltype(halves)::value>(a, sms, st);
    });
}

}  // namespace bsa
