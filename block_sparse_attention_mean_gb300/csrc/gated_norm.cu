// gated_norm.cu -- the step between two sub-blocks of a transformer block: norm of the branch,
// gate, residual add, norm of the sum, scale and shift, in one pass; and its backward pass.
//
//   u = post(y),  h = x + alpha * gate * u,  z = pre(h) * (1 + scale) + shift
//
// A row of C channels is read once, so that mean, variance and result come from one reading, and is
// written once. HBM bounds it.
//
// Split: a worker, the threads that hold one row, walks a contiguous range of the rows (in order of batch
// and token). A worker is a power of two of lanes of a warp (rows of up to 32 groups of 8 channels) or a CTA.
// Each thread holds 8 V channels of the row, in units of 16 bytes of the stream's dtype dealt out thread by
// thread, so that a warp reads contiguous memory.
//
// Every thread copies its own part of the next rows to shared memory with cp.async, STAGES rows ahead, and
// reads it back itself: loads stay in flight across the reductions of the rows before, no barrier or flag
// guards the buffers, and a row that is overwritten in place is read by the thread that writes it.
// What is constant over the rows that share a modulation (weight, bias, gate, scale, shift, alpha) is folded
// into at most two factors per channel and output, kept in registers until the group ends.
#include "block_internal.h"
#include "ptx.cuh"

#include <atomic>
#include <type_traits>

namespace bsa {
namespace {

constexpr int kMaxWarps = 16;  // CTAs of up to 512 threads

// Rows in flight per worker: three, fewer where a CTA of 512 threads would not find room for them (rows of more
// than 4096 channels of several fp32 tensors). `bytes`: what a thread copies per row.
__host__ __device__ constexpr int stages_for(int bytes)
{
    const int fit = 221184 / (512 * bytes);
    return fit > 3 ? 3 : fit < 1 ? 1 : fit;
}

__host__ __device__ constexpr int pow2_ceil(int v)
{
    int p = 1;
    while (p < v) p *= 2;
    return p;
}

// Threads that hold a row of `groups` groups of 8 channels, v of them per thread
__host__ __device__ inline int row_threads(int groups, int v)
{
    return groups <= 32 ? pow2_ceil(groups) : (groups + 32 * v - 1) / (32 * v) * 32;
}

// ------------------------------------------------------------ pairs of fp32
// Two channels per instruction: fp32 add, multiply and fused multiply-add on register pairs.
using f2 = unsigned long long;

__device__ __forceinline__ f2 pair(float a, float b)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 twice(float a) { return pair(a, a); }
__device__ __forceinline__ void split(f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ float both(f2 v)
{
    float a, b;
    split(v, a, b);
    return a + b;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// ------------------------------------------------------------ E channels of a row: a thread's unit
// E / 2 pairs from and to memory. Stores to bf16 round to nearest even: half a step per element.
__device__ __forceinline__ f2 widen(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t narrow(f2 v)
{
    float a, b;
    split(v, a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T, int P>  // P pairs
struct Unit;

template <>
struct Unit<__nv_bfloat16, 4> {
    static __device__ __forceinline__ void get(const void *p, f2 (&v)[4])
    {
        const uint4 r = *static_cast<const uint4 *>(p);
        v[0] = widen(r.x), v[1] = widen(r.y), v[2] = widen(r.z), v[3] = widen(r.w);
    }
    static __device__ __forceinline__ void put(void *p, const f2 (&v)[4])
    {
        *static_cast<uint4 *>(p) = make_uint4(narrow(v[0]), narrow(v[1]), narrow(v[2]), narrow(v[3]));
    }
};

template <>
struct Unit<__nv_bfloat16, 2> {
    static __device__ __forceinline__ void get(const void *p, f2 (&v)[2])
    {
        const uint2 r = *static_cast<const uint2 *>(p);
        v[0] = widen(r.x), v[1] = widen(r.y);
    }
    static __device__ __forceinline__ void put(void *p, const f2 (&v)[2])
    {
        *static_cast<uint2 *>(p) = make_uint2(narrow(v[0]), narrow(v[1]));
    }
};

template <int P>
struct Unit<float, P> {
    static __device__ __forceinline__ void get(const void *p, f2 (&v)[P])
    {
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            const float4 r = static_cast<const float4 *>(p)[i / 2];
            v[i] = pair(r.x, r.y), v[i + 1] = pair(r.z, r.w);
        }
    }
    static __device__ __forceinline__ void put(void *p, const f2 (&v)[P])
    {
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            float4 r;
            split(v[i], r.x, r.y);
            split(v[i + 1], r.z, r.w);
            static_cast<float4 *>(p)[i / 2] = r;
        }
    }
};

// channels of a modulation or of a weight (fp32)
template <int P>
__device__ __forceinline__ void load_mod(const void *p, int dt, int64_t at, f2 (&v)[P])
{
    if (dt == BSA_BF16)
        Unit<__nv_bfloat16, P>::get(static_cast<const char *>(p) + at * 2, v);
    else
        Unit<float, P>::get(static_cast<const char *>(p) + at * 4, v);
}

template <int P>
__device__ __forceinline__ void store_mod(char *p, int dt, int64_t at, const f2 (&v)[P])
{
    if (dt == BSA_BF16)
        Unit<__nv_bfloat16, P>::put(p + at * 2, v);
    else
        Unit<float, P>::put(p + at * 4, v);
}

// v *= m, v *= 1 + m, v += m, for a modulation's (or weight's) channels
template <int P>
__device__ __forceinline__ void times(const void *p, int dt, int64_t at, f2 (&v)[P])
{
    f2 m[P];
    load_mod(p, dt, at, m);
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = mul2(v[i], m[i]);
}
template <int P>
__device__ __forceinline__ void times_one_plus(const void *p, int dt, int64_t at, f2 (&v)[P])
{
    f2 m[P];
    load_mod(p, dt, at, m);
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = mul2(v[i], add2(twice(1.0f), m[i]));
}
template <int P>
__device__ __forceinline__ void plus(const void *p, int dt, int64_t at, f2 (&v)[P])
{
    f2 m[P];
    load_mod(p, dt, at, m);
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = add2(v[i], m[i]);
}
template <int P>
__device__ __forceinline__ void fill(float x, f2 (&v)[P])
{
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = twice(x);
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// ------------------------------------------------------------ rows and workers

// The rows, B * N in order, cut into `workers` ranges that differ by at most one row.
struct Ranges {
    int rows, workers, most;  // most: the longest range
    int per_group;            // rows that share a modulation

    __host__ __device__ int first(int64_t w) const { return static_cast<int>(w * rows / workers); }
    __host__ __device__ int worker_of(int64_t row) const
    {
        return static_cast<int>(((row + 1) * workers - 1) / rows);
    }
};

// A thread's place in a [B][N][C] tensor (byte strides), walked one row at a time
struct Walk {
    char *p;
    int64_t step, wrap;  // to the next token, to the next batch's first

    __device__ __forceinline__ Walk(const RowsView &v, int b, int n, int N, int size)
    {
        p = v.p + (b * v.b + n * v.n) * size;
        step = v.n * size;
        wrap = (v.b - (N - 1) * v.n) * size;
    }
    __device__ __forceinline__ void next(bool batch) { p += batch ? wrap : step; }
};

// What a thread knows of its row: its channels, and the CTA's exchange of the warps' sums. SUB: the row is held
// by `lanes` < 32 lanes of a warp; else by whole warps.
template <int K, int P, bool SUB>
struct Row {
    static constexpr int E = 2 * P;
    int C, lanes, warps, turn;
    bool on[K];
    int c[K];
    float *buf;   // [2][4][kMaxWarps]
    float *held;  // channels that each warp holds

    __device__ __forceinline__ Row(int C_, int tpr, float *buf_)
    {
        C = C_;
        lanes = SUB ? tpr : 32;
        warps = SUB ? 1 : tpr / 32;
        buf = buf_;
        held = buf + 8 * kMaxWarps;
        turn = 0;
        const int t = threadIdx.x % tpr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = E * (t + k * tpr);
            on[k] = at < C;
            c[k] = on[k] ? at : 0;
        }
        if (warps > 1) {
            for (int i = threadIdx.x; i < 9 * kMaxWarps; i += blockDim.x) {
                float n = 0.0f;  // the sums of warps that are not there stay zero, and they hold nothing
                const int w = i - 8 * kMaxWarps;
                if (w >= 0 && w < warps)
                    for (int k = 0; k < K; ++k) n += E * min(32, max(0, C / E - k * tpr - 32 * w));
                buf[i] = n;
            }
            __syncthreads();
        }
    }

    template <int M>
    __device__ __forceinline__ void lanes_sum(float (&v)[M]) const
    {
        if (SUB) {
            for (int o = lanes / 2; o > 0; o >>= 1) {
#pragma unroll
                for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
            }
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
                for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
            }
        }
    }

    // Puts each warp's M values where every thread can read them: one barrier. Two buffers in turn, so that a
    // warp that is ahead does not overwrite what others still read.
    template <int M>
    __device__ __forceinline__ const float *exchange(const float (&v)[M])
    {
        float *b = buf + turn * 4 * kMaxWarps;
        turn ^= 1;
        if (threadIdx.x % 32 == 0) {
#pragma unroll
            for (int m = 0; m < M; ++m) b[m * kMaxWarps + threadIdx.x / 32] = v[m];
        }
        __syncthreads();
        return b;
    }

    __device__ __forceinline__ float total(const float *b) const
    {
        float s = 0.0f;
#pragma unroll 1
        for (int w = 0; w < warps; w += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(b + w);
            s += (q.x + q.y) + (q.z + q.w);
        }
        return s;
    }

    // sums over the row, the same in every thread
    template <int M>
    __device__ __forceinline__ void sums(float (&v)[M])
    {
        lanes_sum(v);
        if (warps == 1) return;
        const float *b = exchange(v);
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] = total(b + m * kMaxWarps);
    }

    // Mean (0 but for LAYER) and mean square about it of M rows at once, one exchange. The spread is taken about
    // each warp's own mean and joined exactly: sum_w (spread_w + n_w (mean_w - mean)^2), no cancellation for rows
    // far from zero. Units that are off hold zeros.
    template <int M>
    __device__ __forceinline__ void stats(const f2 (&v)[M][K][P], const int (&kind)[M], float (&mean)[M], float (&square)[M])
    {
        const float inv_c = 1.0f / static_cast<float>(C);
        bool layer = false;
#pragma unroll
        for (int m = 0; m < M; ++m) layer = layer || kind[m] == BSA_NORM_LAYER;
        if (!layer) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
                f2 q = 0;
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int i = 0; i < P; ++i) q = fma2(v[m][k][i], v[m][k][i], q);
                }
                square[m] = both(q);
                mean[m] = 0.0f;
            }
            sums(square);
#pragma unroll
            for (int m = 0; m < M; ++m) square[m] *= inv_c;
            return;
        }
        const float mine = warps == 1 ? static_cast<float>(C) : held[threadIdx.x / 32];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            f2 q = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int i = 0; i < P; ++i) q = add2(q, v[m][k][i]);
            }
            mean[m] = both(q);
        }
        lanes_sum(mean);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            mean[m] = kind[m] == BSA_NORM_LAYER ? __fdividef(mean[m], mine) : 0.0f;
            const f2 off = twice(-mean[m]);
            f2 q = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                f2 p = 0;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const f2 x = add2(v[m][k][i], off);
                    p = fma2(x, x, p);
                }
                if (on[k]) q = add2(q, p);
            }
            square[m] = both(q);
        }
        lanes_sum(square);
        if (warps > 1) {
            float s[2 * M];
#pragma unroll
            for (int m = 0; m < M; ++m) s[m] = square[m], s[M + m] = mean[m];
            const float *b = exchange(s);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                square[m] = total(b + m * kMaxWarps);
                if (kind[m] != BSA_NORM_LAYER) continue;
                const float4 *means = reinterpret_cast<const float4 *>(b + (M + m) * kMaxWarps);
                const float4 *n = reinterpret_cast<const float4 *>(held);
                float all = 0.0f;
#pragma unroll 1
                for (int w = 0; w < warps; w += 4) {
                    const float4 a = means[w / 4], h = n[w / 4];
                    all += (a.x * h.x + a.y * h.y) + (a.z * h.z + a.w * h.w);
                }
                mean[m] = all * inv_c;
#pragma unroll 1
                for (int w = 0; w < warps; w += 4) {
                    float4 a = means[w / 4];
                    const float4 h = n[w / 4];
                    a.x -= mean[m], a.y -= mean[m], a.z -= mean[m], a.w -= mean[m];
                    square[m] += (a.x * a.x * h.x + a.y * a.y * h.y) + (a.z * a.z * h.z + a.w * a.w * h.w);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < M; ++m) square[m] *= inv_c;
    }
};

constexpr int kExchangeFloats = 9 * kMaxWarps;

// ------------------------------------------------------------ forward

template <typename TS, typename TB, int V, bool SUB>
__global__ void __launch_bounds__(512, 1) gated_norm_kernel(const __grid_constant__ NormArgs a, Ranges rg, int tpr)
{
    constexpr int E = 16 / sizeof(TS), P = E / 2, K = 8 * V / E, XB = E * sizeof(TS), YB = E * sizeof(TB);
    constexpr int STAGES = stages_for(8 * V * (sizeof(TS) + sizeof(TB)));
    __shared__ __align__(16) float buf[kExchangeFloats];
    extern __shared__ __align__(16) char ring[];  // [stage][x: K units of every thread, then y]
    const bsa_gated_norm_desc &d = a.d;
    const bool branch = a.y.p != nullptr, pre = d.pre.kind != BSA_NORM_NONE;
    const int threads = blockDim.x, at_y = K * threads * XB, stage_bytes = at_y + (branch ? K * threads * YB : 0);
    Row<K, P, SUB> rw(d.C, tpr, buf);

    const int64_t worker = static_cast<int64_t>(blockIdx.x) * (threads / tpr) + threadIdx.x / tpr;
    const bool some = worker < rg.workers;
    const int first = some ? rg.first(worker) : 0, count = some ? rg.first(worker + 1) - first : 0;
    const int b0 = first / d.N, n0 = first % d.N;
    Walk x(a.x, b0, n0, d.N, sizeof(TS)), y(a.y, b0, n0, d.N, sizeof(TB));
    Walk h(a.h, b0, n0, d.N, sizeof(TS)), z(a.z, b0, n0, d.N, sizeof(TB));
    int n_ahead = n0, n_here = n0;
    int left = rg.per_group - first % rg.per_group, group = first / rg.per_group;  // rows of the group still to come

    char *const mine_x = ring + threadIdx.x * XB, *const mine_y = ring + at_y + threadIdx.x * YB;
#pragma unroll
    for (int k = 0; k < K; ++k) {  // units that are off stay zero: they add nothing to a sum
        if (rw.on[k]) continue;
        const f2 zero[P] = {};
        for (int st = 0; st < STAGES; ++st) {
            Unit<TS, P>::put(mine_x + st * stage_bytes + k * threads * XB, zero);
            if (branch) Unit<TB, P>::put(mine_y + st * stage_bytes + k * threads * YB, zero);
        }
    }
    int to = 0, from = 0;  // stages
    auto fetch = [&](bool any) {  // copies the worker's next row; a group of copies per row, empty past the end
        if (any) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!rw.on[k]) continue;
                copy_async<XB>(smem_u32(mine_x + to * stage_bytes + k * threads * XB), x.p + rw.c[k] * sizeof(TS));
                if (branch) copy_async<YB>(smem_u32(mine_y + to * stage_bytes + k * threads * YB), y.p + rw.c[k] * sizeof(TB));
            }
            const bool batch = ++n_ahead == d.N;
            if (batch) n_ahead = 0;
            x.next(batch);
            if (branch) y.next(batch);
        }
        cp_async_commit();
        if (++to == STAGES) to = 0;
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i < count);

    f2 h1[K][P], h0[K][P], z1[K][P], z0[K][P];  // h = x + m h1 + h0, z = n z1 + z0
    const bool has_h0 = d.post.bias != nullptr, has_z0 = d.pre.bias || d.shift.ptr;
    auto factors = [&](int g) {
        const int b = g / d.F, f = g % d.F;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = rw.c[k];
            fill(d.alpha, h1[k]);
            fill(0.0f, h0[k]);
            fill(1.0f, z1[k]);
            fill(0.0f, z0[k]);
            if (d.post.weight) times(d.post.weight, BSA_FP32, c, h1[k]);
            if (d.post.bias) {
                fill(d.alpha, h0[k]);
                times(d.post.bias, BSA_FP32, c, h0[k]);
            }
            if (d.gate.ptr) {
                times(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c, h1[k]);
                times(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c, h0[k]);
            }
            if (d.pre.weight) load_mod(d.pre.weight, BSA_FP32, c, z1[k]);
            if (d.pre.bias) load_mod(d.pre.bias, BSA_FP32, c, z0[k]);
            if (d.scale.ptr) {
                times_one_plus(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c, z1[k]);
                times_one_plus(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c, z0[k]);
            }
            if (d.shift.ptr) plus(d.shift.ptr, d.mod_dt, b * d.shift.batch + f * d.shift.frame + c, z0[k]);
        }
    };
    if (count > 0) factors(group);

    // workers of whole warps end on their own; lanes that share a warp go on with it, writing nothing
    const int rounds = SUB ? rg.most : count;
    for (int i = 0; i < rounds; ++i) {
        fetch(i + STAGES - 1 < count);
        cp_async_wait_group<STAGES - 1>();  // row i is here
        const bool live = !SUB || i < count;
        if (live && left == 0) {
            left = rg.per_group;
            factors(++group);
        }
        --left;
        f2 t[1][K][P];
#pragma unroll
        for (int k = 0; k < K; ++k) Unit<TS, P>::get(mine_x + from * stage_bytes + k * threads * XB, t[0][k]);
        if (branch) {
            f2 m[1][K][P];
#pragma unroll
            for (int k = 0; k < K; ++k) Unit<TB, P>::get(mine_y + from * stage_bytes + k * threads * YB, m[0][k]);
            f2 r = twice(1.0f);
            if (d.post.kind != BSA_NORM_NONE) {
                float mean[1], square[1];
                const int kind[1] = {d.post.kind};
                rw.stats(m, kind, mean, square);
                r = twice(rsqrtf(square[0] + d.post.eps));
                if (d.post.kind == BSA_NORM_LAYER) {
                    const f2 off = twice(-mean[0]);
#pragma unroll
                    for (int k = 0; k < K; ++k) {
#pragma unroll
                        for (int j = 0; j < P; ++j) m[0][k][j] = add2(m[0][k][j], off);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int j = 0; j < P; ++j) t[0][k][j] = fma2(m[0][k][j], mul2(r, h1[k][j]), t[0][k][j]);
                if (has_h0) {
#pragma unroll
                    for (int j = 0; j < P; ++j) t[0][k][j] = add2(t[0][k][j], h0[k][j]);
                }
                if (live && rw.on[k]) Unit<TS, P>::put(h.p + rw.c[k] * sizeof(TS), t[0][k]);
                if (!rw.on[k]) fill(0.0f, t[0][k]);
            }
        }
        if (pre) {  // of h before its rounding: the norm sees the exact sum
            float mean[1], square[1];
            const int kind[1] = {d.pre.kind};
            rw.stats(t, kind, mean, square);
            const f2 r = twice(rsqrtf(square[0] + d.pre.eps)), off = twice(-mean[0]);
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (d.pre.kind == BSA_NORM_LAYER) t[0][k][j] = add2(t[0][k][j], off);
                    const f2 w = mul2(r, z1[k][j]);
                    t[0][k][j] = has_z0 ? fma2(t[0][k][j], w, z0[k][j]) : mul2(t[0][k][j], w);
                }
                if (live && rw.on[k]) Unit<TB, P>::put(z.p + rw.c[k] * sizeof(TB), t[0][k]);
            }
        }
        if (live) {
            const bool batch = ++n_here == d.N;
            if (batch) n_here = 0;
            if (branch) h.next(batch);
            if (pre) z.next(batch);
        }
        if (++from == STAGES) from = 0;
    }
}

// ------------------------------------------------------------ backward
//
// A worker keeps four sums per channel in registers while it walks its rows,
//   A = sum dz,  S = sum dz n,  P = sum dx,  Q = sum dx m      (m = y without a post norm),
// from which every parameter's gradient follows by factors that are constant over the rows that share a
// modulation (a group):
//   dshift = A,  dscale = w S + b A,  dgate = alpha (w2 Q + b2 P),
//   dpre_weight = sum_g (1 + scale_g) S_g,  dpre_bias = sum_g (1 + scale_g) A_g,
//   dpost_weight = alpha sum_g gate_g Q_g,  dpost_bias = alpha sum_g gate_g P_g.
// At the end of a group the worker writes the group's gradients itself if it held the whole group, else the
// four sums into one of its two slots (groups that its range's ends cut); the weights' sums go on in its
// third. A second kernel adds the slots in the order of the workers, so that results do not depend on timing.

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

// o = one * w + zero * b for a norm's weight and bias at channels c ..
template <int P>
__device__ __forceinline__ void join(const bsa_norm &n, int c, const f2 (&one)[P], const f2 (&zero)[P], f2 (&o)[P])
{
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] = one[i];
    if (n.weight) times(n.weight, BSA_FP32, c, o);
    if (n.bias) {
        f2 b[P];
        load_mod(n.bias, BSA_FP32, c, b);
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = fma2(zero[i], b[i], o[i]);
    }
}

// the gradients of a group's modulations from its four sums, at channels c ..
template <int P>
__device__ __forceinline__ void write_group(const NormArgs &a, int64_t g, int c, const f2 (&sA)[P], const f2 (&sS)[P],
                                            const f2 (&sP)[P], const f2 (&sQ)[P])
{
    const bsa_gated_norm_desc &d = a.d;
    const int64_t at = g * d.C + c;
    f2 o[P];
    if (a.dshift) store_mod(a.dshift, d.mod_dt, at, sA);
    if (a.dscale) {
        join(d.pre, c, sS, sA, o);
        store_mod(a.dscale, d.mod_dt, at, o);
    }
    if (a.dgate) {
        join(d.post, c, sQ, sP, o);
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = mul2(o[i], twice(d.alpha));
        store_mod(a.dgate, d.mod_dt, at, o);
    }
}

template <typename TS, typename TB, int V, bool SUB>
__global__ void __launch_bounds__(512, 1) gated_norm_backward_kernel(const __grid_constant__ NormArgs a, Ranges rg, int tpr)
{
    constexpr int E = 16 / sizeof(TS), P = E / 2, K = 8 * V / E, SB = E * sizeof(TS), BB = E * sizeof(TB);
    constexpr int STAGES = stages_for(16 * V * (sizeof(TS) + sizeof(TB)));
    __shared__ __align__(16) float buf[kExchangeFloats];
    extern __shared__ __align__(16) char ring[];  // [stage][h, dh, dz, y: K units of every thread each]
    const bsa_gated_norm_desc &d = a.d;
    const bool pre = d.pre.kind != BSA_NORM_NONE, post = d.post.kind != BSA_NORM_NONE, has_y = a.y.p != nullptr,
               has_dh = a.dh.p != nullptr;
    const int threads = blockDim.x, C = d.C;
    const float inv_c = 1.0f / static_cast<float>(C);
    // where each tensor's units lie within a stage
    const int at_dh = pre ? K * threads * SB : 0, at_dz = at_dh + (has_dh ? K * threads * SB : 0),
              at_y = at_dz + (pre ? K * threads * BB : 0), stage_bytes = at_y + (has_y ? K * threads * BB : 0);
    Row<K, P, SUB> rw(C, tpr, buf);
    const Wants want = wants_of(a);

    const int64_t worker = static_cast<int64_t>(blockIdx.x) * (threads / tpr) + threadIdx.x / tpr;
    const bool some = worker < rg.workers;
    const int first = some ? rg.first(worker) : 0, count = some ? rg.first(worker + 1) - first : 0;
    const int b0 = first / d.N, n0 = first % d.N;
    Walk ph(a.h, b0, n0, d.N, sizeof(TS)), pdh(a.dh, b0, n0, d.N, sizeof(TS)), pdx(a.dx, b0, n0, d.N, sizeof(TS));
    Walk pdz(a.dz, b0, n0, d.N, sizeof(TB)), py(a.y, b0, n0, d.N, sizeof(TB)), pdy(a.dy, b0, n0, d.N, sizeof(TB));
    int n_ahead = n0, n_here = n0;
    const int first_group = first / rg.per_group;
    int left = rg.per_group - first % rg.per_group, group = first_group;
    float *const slots = a.partial + worker * gated_norm_worker_floats(C);
    bool weighed = false;  // the worker's third slot holds sums

    char *const mine_s = ring + threadIdx.x * SB, *const mine_b = ring + threadIdx.x * BB;
#pragma unroll
    for (int k = 0; k < K; ++k) {  // units that are off stay zero: they add nothing to a sum
        if (rw.on[k]) continue;
        const f2 zero[P] = {};
        for (int st = 0; st < STAGES; ++st) {
            const int s_at = st * stage_bytes + k * threads * SB, b_at = st * stage_bytes + k * threads * BB;
            if (pre) Unit<TS, P>::put(mine_s + s_at, zero), Unit<TB, P>::put(mine_b + at_dz + b_at, zero);
            if (has_dh) Unit<TS, P>::put(mine_s + at_dh + s_at, zero);
            if (has_y) Unit<TB, P>::put(mine_b + at_y + b_at, zero);
        }
    }
    int to = 0, from = 0;  // stages
    auto fetch = [&](bool any) {
        if (any) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!rw.on[k]) continue;
                const uint32_t s_at = smem_u32(mine_s + to * stage_bytes + k * threads * SB);
                const uint32_t b_at = smem_u32(mine_b + to * stage_bytes + k * threads * BB);
                if (pre) {
                    copy_async<SB>(s_at, ph.p + rw.c[k] * sizeof(TS));
                    copy_async<BB>(b_at + at_dz, pdz.p + rw.c[k] * sizeof(TB));
                }
                if (has_dh) copy_async<SB>(s_at + at_dh, pdh.p + rw.c[k] * sizeof(TS));
                if (has_y) copy_async<BB>(b_at + at_y, py.p + rw.c[k] * sizeof(TB));
            }
            const bool batch = ++n_ahead == d.N;
            if (batch) n_ahead = 0;
            ph.next(batch);
            pdz.next(batch);
            pdh.next(batch);
            py.next(batch);
        }
        cp_async_commit();
        if (++to == STAGES) to = 0;
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i < count);

    f2 sA[K][P] = {}, sS[K][P] = {}, sP[K][P] = {}, sQ[K][P] = {};
    f2 z1[K][P], h1[K][P];  // what dz and dx are multiplied by on their way to n and m
    auto factors = [&](int g) {
        const int b = g / d.F, f = g % d.F;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = rw.c[k];
            fill(1.0f, z1[k]);
            fill(d.alpha, h1[k]);
            if (d.pre.weight) load_mod(d.pre.weight, BSA_FP32, c, z1[k]);
            if (d.scale.ptr) times_one_plus(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c, z1[k]);
            if (d.post.weight) times(d.post.weight, BSA_FP32, c, h1[k]);
            if (d.gate.ptr) times(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c, h1[k]);
        }
    };
    if (count > 0) factors(group);

    const int rounds = SUB ? rg.most : count;
    for (int i = 0; i < rounds; ++i) {
        fetch(i + STAGES - 1 < count);
        cp_async_wait_group<STAGES - 1>();
        const bool live = !SUB || i < count;
        const char *const here_s = mine_s + from * stage_bytes, *const here_b = mine_b + from * stage_bytes;
        if (++from == STAGES) from = 0;
        f2 v[2][K][P];  // h, then n; y, then m
#pragma unroll
        for (int k = 0; k < K; ++k) {
            fill(0.0f, v[0][k]);
            fill(0.0f, v[1][k]);
            if (pre) Unit<TS, P>::get(here_s + k * threads * SB, v[0][k]);
            if (has_y) Unit<TB, P>::get(here_b + at_y + k * threads * BB, v[1][k]);
        }
        float r[2] = {1.0f, 1.0f};
        if (pre || post) {
            float mean[2], square[2];
            const int kind[2] = {d.pre.kind, d.post.kind};
            rw.stats(v, kind, mean, square);
            if (pre) r[0] = rsqrtf(square[0] + d.pre.eps);
            if (post) r[1] = rsqrtf(square[1] + d.post.eps);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const f2 off = twice(-mean[m]), rr = twice(r[m]);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (kind[m] == BSA_NORM_LAYER) {
#pragma unroll
                        for (int j = 0; j < P; ++j) v[m][k][j] = add2(v[m][k][j], off);
                        if (!rw.on[k]) fill(0.0f, v[m][k]);
                    }
#pragma unroll
                    for (int j = 0; j < P; ++j) v[m][k][j] = mul2(v[m][k][j], rr);
                }
            }
        }
        f2 g[K][P];  // the gradient at h, then at u
#pragma unroll
        for (int k = 0; k < K; ++k) {
            fill(0.0f, g[k]);
            if (has_dh) Unit<TS, P>::get(here_s + at_dh + k * threads * SB, g[k]);
        }
        if (pre) {
            f2 q[K][P], s0 = 0, s1 = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                Unit<TB, P>::get(here_b + at_dz + k * threads * BB, q[k]);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (live) {
                        sA[k][j] = add2(sA[k][j], q[k][j]);
                        sS[k][j] = fma2(q[k][j], v[0][k][j], sS[k][j]);
                    }
                    q[k][j] = mul2(q[k][j], z1[k][j]);
                    s0 = fma2(q[k][j], v[0][k][j], s0);
                    s1 = add2(s1, q[k][j]);
                }
            }
            float s[2] = {both(s0), both(s1)};
            rw.sums(s);
            const f2 along = twice(-s[0] * inv_c), mean = twice(d.pre.kind == BSA_NORM_LAYER ? -s[1] * inv_c : 0.0f);
            const f2 rr = twice(r[0]);
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int j = 0; j < P; ++j)
                    g[k][j] = fma2(rr, fma2(v[0][k][j], along, add2(q[k][j], mean)), g[k][j]);
                if (!rw.on[k]) fill(0.0f, g[k]);
            }
        }
        if (a.dx.p && live) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (rw.on[k]) Unit<TS, P>::put(pdx.p + rw.c[k] * sizeof(TS), g[k]);
        }
        if (has_y) {
            f2 s0 = 0, s1 = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (live) {
                        sP[k][j] = add2(sP[k][j], g[k][j]);
                        sQ[k][j] = fma2(g[k][j], v[1][k][j], sQ[k][j]);
                    }
                    g[k][j] = mul2(g[k][j], h1[k][j]);
                    s0 = fma2(g[k][j], v[1][k][j], s0);
                    s1 = add2(s1, g[k][j]);
                }
            }
            if (post) {
                float s[2] = {both(s0), both(s1)};
                rw.sums(s);
                const f2 along = twice(-s[0] * inv_c), mean = twice(d.post.kind == BSA_NORM_LAYER ? -s[1] * inv_c : 0.0f);
                const f2 rr = twice(r[1]);
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int j = 0; j < P; ++j) g[k][j] = mul2(rr, fma2(v[1][k][j], along, add2(g[k][j], mean)));
                }
            }
            if (a.dy.p && live) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (rw.on[k]) Unit<TB, P>::put(pdy.p + rw.c[k] * sizeof(TB), g[k]);
            }
        }
        if (!live) continue;
        const bool batch = ++n_here == d.N;
        if (batch) n_here = 0;
        pdx.next(batch);
        pdy.next(batch);
        if (--left > 0 && i + 1 < count) continue;
        // the end of a group, or of the range
        if (want.pre_sums || want.post_sums) {
            const int64_t begin = static_cast<int64_t>(group) * rg.per_group;
            const bool whole = begin >= first && begin + rg.per_group <= static_cast<int64_t>(first) + count;
            float *const slot = slots + (group == first_group ? 0 : 4 * C);
            const int b = group / d.F, f = group % d.F;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!rw.on[k]) continue;
                const int c = rw.c[k];
                if (whole) {
                    write_group(a, group, c, sA[k], sS[k], sP[k], sQ[k]);
                } else {
                    Unit<float, P>::put(slot + c, sA[k]);
                    Unit<float, P>::put(slot + C + c, sS[k]);
                    Unit<float, P>::put(slot + 2 * C + c, sP[k]);
                    Unit<float, P>::put(slot + 3 * C + c, sQ[k]);
                }
                if (want.weights) {  // weighted for the parameters that all groups share, and added up
                    if (d.scale.ptr) {
                        times_one_plus(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c, sA[k]);
                        times_one_plus(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c, sS[k]);
                    }
                    if (d.gate.ptr) {
                        times(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c, sP[k]);
                        times(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c, sQ[k]);
                    }
                    float *const sum = slots + 8 * C + c;
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        sP[k][j] = mul2(sP[k][j], twice(d.alpha));
                        sQ[k][j] = mul2(sQ[k][j], twice(d.alpha));
                    }
                    if (weighed) {
                        plus(sum, BSA_FP32, 0, sA[k]);
                        plus(sum + C, BSA_FP32, 0, sS[k]);
                        plus(sum + 2 * C, BSA_FP32, 0, sP[k]);
                        plus(sum + 3 * C, BSA_FP32, 0, sQ[k]);
                    }
                    Unit<float, P>::put(sum, sA[k]);
                    Unit<float, P>::put(sum + C, sS[k]);
                    Unit<float, P>::put(sum + 2 * C, sP[k]);
                    Unit<float, P>::put(sum + 3 * C, sQ[k]);
                }
                fill(0.0f, sA[k]);
                fill(0.0f, sS[k]);
                fill(0.0f, sP[k]);
                fill(0.0f, sQ[k]);
            }
            weighed = true;
        }
        if (i + 1 < count) {
            left = rg.per_group;
            factors(++group);
        }
    }
}

// Adds the workers' slots, 32 channels per CTA, kSumSlices slices of the workers each. blockIdx.y == 0: the
// weights' sums over all workers; blockIdx.y > 0: one group that several workers share.
constexpr int kSumSlices = 32;

__global__ void __launch_bounds__(32 * kSumSlices) gated_norm_sums_kernel(const __grid_constant__ NormArgs a, Ranges rg,
                                                                          int64_t n_groups)
{
    __shared__ float part[kSumSlices][32][5];
    grid_dependency_wait();
    const bsa_gated_norm_desc &d = a.d;
    const int C = d.C;
    const int64_t stride = gated_norm_worker_floats(C);
    const Wants want = wants_of(a);
    int64_t w0 = 0, w1 = rg.workers - 1, group = -1;
    if (blockIdx.y == 0) {
        if (!want.weights) return;
    } else {
        // the group itself where there are at most as many groups as workers; else the one that worker y - 1's
        // range begins inside
        const int64_t i = blockIdx.y - 1;
        group = n_groups <= rg.workers ? i : rg.first(i) / rg.per_group;
        w0 = rg.worker_of(group * rg.per_group);
        w1 = rg.worker_of((group + 1) * rg.per_group - 1);
        if (w0 == w1) return;                              // written by its worker
        if (n_groups > rg.workers && i != w0 + 1) return;  // one CTA per group
    }
    const int c = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < C) {
        for (int64_t w = w0 + slice; w <= w1; w += kSumSlices) {
            const int slot = group < 0 ? 8 : (rg.first(w) / rg.per_group == group ? 0 : 4);
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

// vectors of 8 channels per thread
int vectors(int C) { return C > 4096 ? 2 : 1; }

// What a launch needs to know of a kernel, looked up once: registers, and (once per device) leave to use all of
// the shared memory.
template <typename Kernel>
bsa_status ready(Kernel kern, int smem, std::atomic<uint64_t> &done, std::atomic<int> &regs)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return BSA_OK;
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, kern) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
        return BSA_ERR_CUDA;
    regs.store(at.numRegs, std::memory_order_relaxed);
    done.fetch_or(bit, std::memory_order_release);
    return BSA_OK;
}

struct Shape {
    int tpr, threads, ctas;
    size_t smem;
    Ranges rg;
};

// Workers: as many as fit on the device at once, each with an equal share of the rows; at most one per row.
Shape shape_of(const bsa_gated_norm_desc &d, int v, int regs, int sms, int stages, int thread_bytes)
{
    Shape s;
    s.tpr = row_threads(d.C / 8, v);
    s.threads = s.tpr <= 32 ? 128 : s.tpr;
    s.smem = static_cast<size_t>(stages) * s.threads * thread_bytes;
    const int by_regs = 65536 / ((regs + 7) / 8 * 8 * s.threads);
    const int by_smem = static_cast<int>((228 * 1024) / (s.smem + 4096));
    int resident = by_regs < by_smem ? by_regs : by_smem;
    if (resident > 2048 / s.threads) resident = 2048 / s.threads;
    if (resident < 1) resident = 1;
    const int per_cta = s.threads / s.tpr;
    s.rg.rows = d.B * d.N;
    s.rg.per_group = d.N / d.F;
    const int64_t fill = static_cast<int64_t>(sms) * resident * per_cta, most = gated_norm_max_workers(s.rg.rows, d.C);
    s.rg.workers = static_cast<int>(fill < most ? fill : most);
    s.rg.most = (s.rg.rows + s.rg.workers - 1) / s.rg.workers;
    s.ctas = (s.rg.workers + per_cta - 1) / per_cta;
    return s;
}

template <typename TS, typename TB, int V, bool SUB>
bsa_status forward(const NormArgs &a, int sms, cudaStream_t st)
{
    auto kern = gated_norm_kernel<TS, TB, V, SUB>;
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> regs{0};
    constexpr int BYTES = 8 * V * (sizeof(TS) + sizeof(TB)), STAGES = stages_for(BYTES);
    const bsa_status ok = ready(kern, STAGES * 512 * BYTES, done, regs);
    if (ok != BSA_OK) return ok;
    const Shape s = shape_of(a.d, V, regs.load(std::memory_order_relaxed), sms, STAGES,
                             8 * V * static_cast<int>(sizeof(TS) + (a.y.p ? sizeof(TB) : 0)));
    kern<<<s.ctas, s.threads, s.smem, st>>>(a, s.rg, s.tpr);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <typename TS, typename TB, int V, bool SUB>
bsa_status backward(const NormArgs &a, int sms, cudaStream_t st)
{
    auto kern = gated_norm_backward_kernel<TS, TB, V, SUB>;
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> regs{0};
    constexpr int BYTES = 16 * V * (sizeof(TS) + sizeof(TB)), STAGES = stages_for(BYTES);
    const bsa_status ok = ready(kern, STAGES * 512 * BYTES, done, regs);
    if (ok != BSA_OK) return ok;
    const int pre = a.d.pre.kind != BSA_NORM_NONE;
    const Shape s = shape_of(a.d, V, regs.load(std::memory_order_relaxed), sms, STAGES,
                             8 * V * static_cast<int>(sizeof(TS) * (pre + (a.dh.p ? 1 : 0)) + sizeof(TB) * (pre + (a.y.p ? 1 : 0))));
    kern<<<s.ctas, s.threads, s.smem, st>>>(a, s.rg, s.tpr);
    if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
    if (a.partial == nullptr) return BSA_OK;
    const int64_t n_groups = static_cast<int64_t>(a.d.B) * a.d.F;
    const int64_t items = n_groups < s.rg.workers ? n_groups : s.rg.workers;
    const dim3 grid((a.d.C + 31) / 32, static_cast<unsigned>(items + 1));
    return pdl_launch(gated_norm_sums_kernel, grid, 32 * kSumSlices, 0, st, a, s.rg, n_groups) ? BSA_OK : BSA_ERR_CUDA;
}

template <typename F>
bsa_status by_kernel(const bsa_gated_norm_desc &d, F &&run)
{
    auto by_width = [&](auto ts, auto tb) {
        if (d.C >= 256) {
            if (vectors(d.C) == 2) return run(ts, tb, std::integral_constant<int, 2>(), std::false_type());
            return run(ts, tb, std::integral_constant<int, 1>(), std::false_type());
        }
        return row_threads(d.C / 8, 1) < 32 ? run(ts, tb, std::integral_constant<int, 1>(), std::true_type())
                                            : run(ts, tb, std::integral_constant<int, 1>(), std::false_type());
    };
    if (d.stream_dt == BSA_BF16) return by_width(__nv_bfloat16(), __nv_bfloat16());
    if (d.branch_dt == BSA_BF16) return by_width(float(), __nv_bfloat16());
    return by_width(float(), float());
}

}  // namespace

int64_t gated_norm_max_workers(int64_t rows, int C)
{
    const int64_t w = kNormMaxThreads / row_threads(C / 8, vectors(C));
    return rows < w ? rows : w;
}

bsa_status launch_gated_norm(const NormArgs &a, cudaStream_t st)
{
    int sms = 0;
    const bsa_status s = current_sm_count(&sms);
    if (s != BSA_OK) return s;
    return by_kernel(a.d, [&](auto ts, auto tb, auto v, auto sub) {
        return forward<decltype(ts), decltype(tb), decltype(v)::value, decltype(sub)::value>(a, sms, st);
    });
}

bsa_status launch_gated_norm_backward(const NormArgs &a, cudaStream_t st)
{
    int sms = 0;
    const bsa_status s = current_sm_count(&sms);
    if (s != BSA_OK) return s;
    return by_kernel(a.d, [&](auto ts, auto tb, auto v, auto sub) {
        return backward<decltype(ts), decltype(tb), decltype(v)::value, decltype(sub)::value>(a, sms, st);
    });
}

}  // namespace bsa
