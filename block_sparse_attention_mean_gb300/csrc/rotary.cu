// rotary.cu -- rotary positions with several axes, the per-head RMS norm of Q and K, and the
// change from the projection's layout to the attention's, in one pass; and its backward pass.
//
// Per token n, head and channel pair (a, b) of axis s:
//   u = x * rsqrt(mean x^2 + eps) * w,  t = pos[n][s] * f,
//   y_a = u_a cos t - u_b sin t,  y_b = u_b cos t + u_a sin t.
// Each element is read once and written once and takes about ten operations: HBM bounds it.
//
// Split: a CTA of 256 threads takes a tile of tokens, d / 16 threads to a token, 16 channels (8 pairs) each, and
// walks over the heads of Q, then K, then V, so that a thread's eight angles, the one costly part, are computed once
// for all heads of its token. The work, (tiles) x (heads) in that order, is cut into equal ranges, one per CTA that
// fits on the device at once: no last wave that is only partly full.
//
// Loads: each thread copies its own 16 channels of the next heads to shared memory with cp.async, kStages heads
// ahead, and reads them back itself: loads stay in flight across heads and tiles, and no barrier guards the buffers.
//
// Angles: frequencies are 64-bit fixed point in turns, so pos * f modulo one turn is the low 64 bits of an integer
// product. Its top 32 bits, as a signed fraction of half turns, go to sincospif in fp32: the angle is off by at most
// 2^-25 half turns whatever the position, without fp64 or a slow argument reduction.
#include "block_internal.h"
#include "ptx.cuh"

#include <atomic>
#include <type_traits>

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kStages = 4;  // heads in flight per thread (a power of two)

// What a thread holds of a head: two groups of 8 channels from c0 and c1 on, in which its pairs are
//   INTERLEAVED: channels (2j, 2j + 1) of the groups (j < 4 of the first);  HALVES: channel j of the first and of the second
// and which of the 8 pairs turn (bits). Groups are dealt out so that a warp's 16-byte accesses are contiguous.
struct Lane {
    int c0, c1;
    unsigned turns;
};

template <int D, bool HALVES>
__device__ __forceinline__ int pair_of(int t, int j)
{
    return HALVES ? 8 * t + j : j < 4 ? 4 * t + j : D / 4 + 4 * t + j - 4;
}

template <int D, bool HALVES>
__device__ __forceinline__ Lane lane_of(int t, int rot)
{
    Lane l;
    l.turns = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) l.turns |= (pair_of<D, HALVES>(t, j) < rot / 2 ? 1u : 0u) << j;
    if (HALVES) {  // rot / 2 is a multiple of 8: all eight pairs turn, or none (then 16 channels past the turning ones)
        l.c0 = l.turns ? 8 * t : 16 * t;
        l.c1 = l.turns ? rot / 2 + 8 * t : 16 * t + 8;
    } else {
        l.c0 = 8 * t;
        l.c1 = D / 2 + 8 * t;
    }
    return l;
}

template <int D, bool HALVES>
__device__ __forceinline__ void angles(const bsa_rotary_plan &plan, const int32_t *pos, int t, unsigned turns,
                                       float (&cs)[8], float (&sn)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        cs[j] = 1.0f;
        sn[j] = 0.0f;
        if (turns >> j & 1u) {
            const int p = pair_of<D, HALVES>(t, j);
            const uint64_t ph = plan.turns[p] * static_cast<uint64_t>(static_cast<int64_t>(pos[plan.axis[p]]));
            const float half_turns = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 4.656612873077393e-10f;  // 2^-31
            sincospif(half_turns, &sn[j], &cs[j]);
        }
    }
}

// Turns the 16 channels of a thread by its angles (DIR = 1) or back (DIR = -1). Channels that do not
// turn pass through as they are (no product with zero: an infinity stays one).
template <bool HALVES, int DIR>
__device__ __forceinline__ void turn(float (&u0)[8], float (&u1)[8], const float (&cs)[8], const float (&sn)[8],
                                     unsigned turns)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float &a = HALVES ? u0[j] : (j < 4 ? u0[2 * j] : u1[2 * j - 8]);
        float &b = HALVES ? u1[j] : (j < 4 ? u0[2 * j + 1] : u1[2 * j - 7]);
        const float s = DIR * sn[j];
        const float ya = a * cs[j] - b * s, yb = b * cs[j] + a * s;
        if (turns >> j & 1u) {
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
    if (w) {
        Vec8<float> v;
        v.load(w, c);
        v.unpack(f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 1.0f;
    }
}

// A CTA's range of the work: units of one head of one tile of tokens, heads of Q, K, V in order within a tile.
struct Work {
    int64_t units;
    int heads;  // of Q, K and V together
};

// A thread's place in the work: the tile's token (clamped: shuffles take whole warps), the tensor and the head.
struct Place {
    int64_t tile;
    int s, h;  // tensor, head
    int b, n;
    bool live;

    __device__ __forceinline__ void tile_at(int64_t t, const RotaryArgs &a, int tokens, int mine)
    {
        tile = t;
        const int64_t all = static_cast<int64_t>(a.B) * a.N;
        int64_t token = t * tokens + mine;
        live = token < all;
        if (!live) token = all - 1;
        b = static_cast<int>(token) / a.N;
        n = static_cast<int>(token) % a.N;
    }
    __device__ __forceinline__ void start(int64_t unit, const Work &w, const RotaryArgs &a, int tokens, int mine)
    {
        tile_at(unit / w.heads, a, tokens, mine);
        h = static_cast<int>(unit % w.heads);
        s = 0;
        while (h >= a.t[s].heads) h -= a.t[s++].heads;
    }
    // to the next head; true where the tensor or the tile changed
    __device__ __forceinline__ bool next(const RotaryArgs &a, int tokens, int mine)
    {
        if (++h < a.t[s].heads) return false;
        h = 0;
        do {
            if (++s == 3) {
                s = 0;
                tile_at(tile + 1, a, tokens, mine);
            }
        } while (a.t[s].heads == 0);
        return true;
    }
};

// 16 channels of a thread, from global memory to its own place in a stage
template <typename T>
__device__ __forceinline__ void copy_groups(uint32_t to, const char *from, const Lane &l)
{
    constexpr int PIECES = sizeof(T) / 2;  // of 16 bytes, per group
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            cp_async16(to + (g * PIECES + i) * kThreads * 16, from + (g ? l.c1 : l.c0) * sizeof(T) + 16 * i);
    }
}

// one group of 8 channels from the thread's place in a stage
template <typename T>
__device__ __forceinline__ void read_group(const char *at, int g, float (&f)[8])
{
    constexpr int PIECES = sizeof(T) / 2;
    Vec8<T> v;
    if constexpr (PIECES == 1) {
        v.r = *reinterpret_cast<const uint4 *>(at + g * kThreads * 16);
    } else {
        v.a = *reinterpret_cast<const float4 *>(at + 2 * g * kThreads * 16);
        v.b = *reinterpret_cast<const float4 *>(at + (2 * g + 1) * kThreads * 16);
    }
    v.unpack(f);
}

template <typename T>
__device__ __forceinline__ void write_group(char *to, int c, const float (&f)[8])
{
    Vec8<T> v;
    v.pack(f);
    v.store(to, c);
}

template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const __grid_constant__ RotaryArgs a, Work w)
{
    constexpr int LANES = D / 16, TOKENS = kThreads / LANES, STAGE = kThreads * 16 * sizeof(T);
    extern __shared__ __align__(16) char ring[];
    const int t = threadIdx.x % LANES, mine = threadIdx.x / LANES;
    const Lane l = lane_of<D, HALVES>(t, a.plan.rot);
    const int64_t u0 = w.units * blockIdx.x / gridDim.x, u1 = w.units * (blockIdx.x + 1) / gridDim.x;
    const int count = static_cast<int>(u1 - u0);
    char *const own = ring + threadIdx.x * 16;

    Place ahead;
    ahead.start(u0, w, a, TOKENS, mine);
    const char *src = nullptr;
    auto enter_src = [&] {
        const HeadsView &v = a.t[ahead.s];
        src = v.src + (ahead.b * v.src_b + ahead.n * v.src_n + ahead.h * v.src_h) * sizeof(T);
    };
    enter_src();
    auto fetch = [&](int i) {  // a group of copies per head, empty past the end
        if (i < count) {
            copy_groups<T>(smem_u32(own + (i % kStages) * STAGE), src, l);
            src += a.t[ahead.s].src_h * sizeof(T);
            if (ahead.next(a, TOKENS, mine)) enter_src();
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    Place here;
    here.start(u0, w, a, TOKENS, mine);
    float cs[8], sn[8], w0[8], w1[8];
    char *dst = nullptr;
    int64_t tile = -1;  // the one whose angles are here
    auto enter = [&] {
        const HeadsView &v = a.t[here.s];
        dst = v.dst + (here.b * v.dst_b + here.n * v.dst_n + here.h * v.dst_h) * sizeof(T);
        if (here.s == 2) return;
        if (tile != here.tile) {
            tile = here.tile;
            angles<D, HALVES>(a.plan, a.positions + here.b * a.pos_batch + static_cast<int64_t>(here.n) * a.plan.n_axes, t,
                              l.turns, cs, sn);
        }
        if (a.norm) {
            load_weight(v.weight, l.c0, w0);
            load_weight(v.weight, l.c1, w1);
        }
    };
    enter();
    for (int i = 0; i < count; ++i) {
        fetch(i + kStages - 1);
        cp_async_wait_group<kStages - 1>();
        const char *at = own + (i % kStages) * STAGE;
        float x0[8], x1[8];
        read_group<T>(at, 0, x0);
        read_group<T>(at, 1, x1);
        if (here.s < 2) {
            if (a.norm) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += x0[j] * x0[j] + x1[j] * x1[j];
                const float r = rsqrtf(lanes_sum<LANES>(ss) * (1.0f / D) + a.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x0[j] *= r * w0[j];
                    x1[j] *= r * w1[j];
                }
            }
            turn<HALVES, 1>(x0, x1, cs, sn, l.turns);
        }
        if (here.live) {
            write_group<T>(dst, l.c0, x0);
            write_group<T>(dst, l.c1, x1);
        }
        dst += a.t[here.s].dst_h * sizeof(T);
        if (i + 1 < count && here.next(a, TOKENS, mine)) enter();
    }
}

// Backward. Two copies per head under the norm, dy and x. A thread sums the weight gradients of its 16 channels in
// registers over a run of heads, then in its own place in shared memory over its CTA's work.
template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads, 2) rotary_backward_kernel(const __grid_constant__ RotaryArgs a, Work w)
{
    constexpr int LANES = D / 16, TOKENS = kThreads / LANES, STAGE = kThreads * 16 * sizeof(T);
    extern __shared__ __align__(16) char ring[];  // [stage][dy, then x with norm], then the weight gradients' sums
    __shared__ float sums[kThreads / 32][D];
    const int t = threadIdx.x % LANES, mine = threadIdx.x / LANES;
    const Lane l = lane_of<D, HALVES>(t, a.plan.rot);
    const int64_t u0 = w.units * blockIdx.x / gridDim.x, u1 = w.units * (blockIdx.x + 1) / gridDim.x;
    const int count = static_cast<int>(u1 - u0), stage_bytes = a.norm ? 2 * STAGE : STAGE;
    char *const own = ring + threadIdx.x * 16;
    float4 *const dw_at = reinterpret_cast<float4 *>(ring + kStages * stage_bytes) + threadIdx.x;  // [2][4] pieces
    if (a.partial) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dw_at[i * kThreads] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }

    Place ahead;
    ahead.start(u0, w, a, TOKENS, mine);
    const char *src = nullptr, *xsrc = nullptr;
    auto enter_src = [&] {
        const HeadsView &v = a.t[ahead.s];
        src = v.src + (ahead.b * v.src_b + ahead.n * v.src_n + ahead.h * v.src_h) * sizeof(T);
        xsrc = v.x + (ahead.b * v.x_b + ahead.n * v.x_n + ahead.h * v.x_h) * sizeof(T);
    };
    enter_src();
    auto fetch = [&](int i) {
        if (i < count) {
            const HeadsView &v = a.t[ahead.s];
            const uint32_t to = smem_u32(own + (i % kStages) * stage_bytes);
            copy_groups<T>(to, src, l);
            if (a.norm && ahead.s < 2) copy_groups<T>(to + STAGE, xsrc, l);
            src += v.src_h * sizeof(T);
            xsrc += v.x_h * sizeof(T);
            if (ahead.next(a, TOKENS, mine)) enter_src();
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    Place here;
    here.start(u0, w, a, TOKENS, mine);
    float cs[8], sn[8], w0[8], w1[8], dw[16] = {};
    char *dst = nullptr;
    int64_t tile = -1;
    auto enter = [&] {
        const HeadsView &v = a.t[here.s];
        dst = v.dst + (here.b * v.dst_b + here.n * v.dst_n + here.h * v.dst_h) * sizeof(T);
        if (here.s == 2) return;
        if (tile != here.tile) {
            tile = here.tile;
            angles<D, HALVES>(a.plan, a.positions + here.b * a.pos_batch + static_cast<int64_t>(here.n) * a.plan.n_axes, t,
                              l.turns, cs, sn);
        }
        if (a.norm) {
            load_weight(v.weight, l.c0, w0);
            load_weight(v.weight, l.c1, w1);
        }
    };
    auto leave = [&](int s) {  // the end of a run of heads of one tensor
        if (!a.partial || s == 2) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 v = dw_at[(4 * s + i) * kThreads];
            v.x += dw[4 * i], v.y += dw[4 * i + 1], v.z += dw[4 * i + 2], v.w += dw[4 * i + 3];
            dw_at[(4 * s + i) * kThreads] = v;
            dw[4 * i] = dw[4 * i + 1] = dw[4 * i + 2] = dw[4 * i + 3] = 0.0f;
        }
    };
    enter();
    for (int i = 0; i < count; ++i) {
        fetch(i + kStages - 1);
        cp_async_wait_group<kStages - 1>();
        const char *at = own + (i % kStages) * stage_bytes;
        float g0[8], g1[8];
        read_group<T>(at, 0, g0);
        read_group<T>(at, 1, g1);
        if (here.s < 2) {
            turn<HALVES, -1>(g0, g1, cs, sn, l.turns);
            if (a.norm) {
                float x0[8], x1[8];
                read_group<T>(at + STAGE, 0, x0);
                read_group<T>(at + STAGE, 1, x1);
                float ss = 0.0f, sv = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ss += x0[j] * x0[j] + x1[j] * x1[j];
                    sv += g0[j] * w0[j] * x0[j] + g1[j] * w1[j] * x1[j];
                }
                const float r = rsqrtf(lanes_sum<LANES>(ss) * (1.0f / D) + a.eps);
                const float m = lanes_sum<LANES>(sv) * (1.0f / D) * r * r;
                const float rl = here.live ? r : 0.0f;  // the clamped token is not counted again
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (here.live) {
                        dw[j] += g0[j] * (x0[j] * rl);
                        dw[8 + j] += g1[j] * (x1[j] * rl);
                    }
                    g0[j] = r * (g0[j] * w0[j] - x0[j] * m);
                    g1[j] = r * (g1[j] * w1[j] - x1[j] * m);
                }
            }
        }
        if (here.live) {
            write_group<T>(dst, l.c0, g0);
            write_group<T>(dst, l.c1, g1);
        }
        dst += a.t[here.s].dst_h * sizeof(T);
        const int s = here.s;
        if (i + 1 == count || here.next(a, TOKENS, mine)) {
            leave(s);
            if (i + 1 < count) enter();
        }
    }

    if (a.partial == nullptr) return;
    // the CTA's sums per channel: over the warp's tokens by shuffles, over the warps in order
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 q = dw_at[(4 * s + i) * kThreads];
            float v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int o = LANES; o < 32; o <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
                const int j = 4 * i + e;
                if (threadIdx.x % 32 < LANES) sums[threadIdx.x / 32][(j < 8 ? l.c0 : l.c1 - 8) + j] = v[e];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += kThreads) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kThreads / 32; ++k) v += sums[k][c];
            a.partial[(static_cast<int64_t>(blockIdx.x) * 2 + s) * D + c] = v;
        }
        __syncthreads();
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

// The work, and the CTAs that share it: as many as are resident at once, at most one per unit.
template <int D>
int work_of(const RotaryArgs &a, int sms, int resident, Work *w)
{
    constexpr int TOKENS = kThreads / (D / 16);
    const int64_t tiles = (static_cast<int64_t>(a.B) * a.N + TOKENS - 1) / TOKENS;
    w->heads = a.t[0].heads + a.t[1].heads + a.t[2].heads;
    w->units = tiles * w->heads;
    const int64_t ctas = static_cast<int64_t>(sms) * resident;
    return static_cast<int>(w->units < ctas ? w->units : ctas);
}

// Leave to use more than 48 KB of shared memory, asked for once per kernel and device.
template <typename Kernel>
bsa_status allow_smem(Kernel kern, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return BSA_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
        return BSA_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_release);
    return BSA_OK;
}

template <typename T, int D, bool HALVES>
bsa_status forward(const RotaryArgs &a, int sms, cudaStream_t st)
{
    auto kern = rotary_kernel<T, D, HALVES>;
    constexpr int SMEM = kStages * kThreads * 16 * sizeof(T);
    static std::atomic<uint64_t> done{0};
    const bsa_status ok = allow_smem(kern, SMEM, done);
    if (ok != BSA_OK) return ok;
    Work w;
    const int ctas = work_of<D>(a, sms, 3, &w);
    kern<<<ctas, kThreads, SMEM, st>>>(a, w);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <typename T, int D, bool HALVES>
bsa_status backward(const RotaryArgs &a, int sms, cudaStream_t st)
{
    auto kern = rotary_backward_kernel<T, D, HALVES>;
    constexpr int STAGE = kThreads * 16 * sizeof(T), SUMS = kThreads * 128;
    static std::atomic<uint64_t> done{0};
    const bsa_status ok = allow_smem(kern, kStages * 2 * STAGE + SUMS, done);
    if (ok != BSA_OK) return ok;
    Work w;
    const int resident = sizeof(T) == 2 ? 2 : 1;  // fp32: 160 KB of shared memory per CTA
    int ctas = work_of<D>(a, sms, resident, &w);
    if (ctas > kRotaryMaxCtas) ctas = kRotaryMaxCtas;
    kern<<<ctas, kThreads, kStages * (a.norm ? 2 : 1) * STAGE + (a.partial ? SUMS : 0), st>>>(a, w);
    if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
    if (a.partial && !pdl_launch(rotary_dweight_kernel, dim3(2 * D / 32), 1024, 0, st, a.partial, ctas, D, a.t[0].dweight,
                                 a.t[1].dweight))
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
