// gated_norm.cuh -- what the forward (gated_norm.cu) and backward (gated_norm_backward.cu) kernels of the gated norm
// share: a thread's part of a row, the sums over a row, and how the rows are dealt out.
#pragma once

#include <atomic>
#include <type_traits>

#include "block_internal.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int kMaxWarps = 16;  // CTAs of up to 512 threads

// Threads of a CTA at most: of several rows, of a row in that many registers (by_kernel)
__host__ __device__ constexpr int most_threads(int regs, bool multi, int branch_size)
{
    return multi ? 128 : regs == 128 ? 512 : branch_size == 4 ? 320 : 384;
}

// Rows in flight per worker, forward: more of them are slower (65536 rows of 2048 channels: three 182 us, four 197 us).
// Backward two, which have more tensors each (16384 rows of 2048 channels bf16: one 110.8 us, two 87.4, three 87.9), or one
// where the largest CTA has no room for two of `bytes` a thread beside the `kept` bytes.
constexpr int kStages = 3;
__host__ __device__ constexpr int stages_for(int threads, int bytes, int kept)
{
    return threads * (2 * bytes + kept) <= 221184 ? 2 : 1;
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
    return groups <= 32 * v ? pow2_ceil((groups + v - 1) / v) : (groups + 32 * v - 1) / (32 * v) * 32;
}

// ------------------------------------------------------------ a thread's unit of a row
// P pairs of channels from and to memory. Stores to bf16 round to nearest even: half a step per element.
template <typename T, int P>
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

// channels of a modulation or of a weight (fp32): nothing writes them while the kernel runs, so that their loads need not
// wait for one another's uses
template <int P>
__device__ __forceinline__ void load_mod(const void *p, int dt, int64_t at, f2 (&v)[P])
{
    if (dt == BSA_BF16) {
        const char *from = static_cast<const char *>(p) + at * 2;
        uint32_t r[P];
        if constexpr (P == 4) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(from));
            r[0] = q.x, r[1] = q.y, r[2] = q.z, r[3] = q.w;
        } else {
            const uint2 q = __ldg(reinterpret_cast<const uint2 *>(from));
            r[0] = q.x, r[1] = q.y;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = widen(r[i]);
    } else {
        const float4 *from = reinterpret_cast<const float4 *>(static_cast<const char *>(p) + at * 4);
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            const float4 r = __ldg(from + i / 2);
            v[i] = pair(r.x, r.y), v[i + 1] = pair(r.z, r.w);
        }
    }
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

// Vectors of 8 channels per thread. What a row costs a thread apart from its channels (the sums over the row, addresses,
// the loop) is about as much as eight channels cost: with one vector, twice as many warps pay it (2048 channels bf16:
// 193 against 182 us forward, 65536 rows; 153 against 87 us backward, 16384 rows). With more there are too few
// registers for the sums of the backward pass.
constexpr int V = 2;

// ------------------------------------------------------------ rows and workers

// The rows, B * N in order, cut into `workers` ranges of nearly equal length: range w begins at row
// floor(w * step / 2^32), step = ceil(rows * 2^32 / workers). Longer and shorter ranges alternate: with the longer ones
// first, most workers stand the same number of rows apart, and meet a little more often in the same memory channels
// (65536 rows of 2048 channels: 183.3 against 181.9 us).
struct Ranges {
    int rows, workers;
    uint64_t step, per_step;
    int per_group;    // rows that share a modulation
    int long_groups;  // no range is longer than a group: it touches two groups at most

    __host__ __device__ int first(int w) const { return static_cast<int>(static_cast<uint64_t>(w) * step >> 32); }
    __host__ __device__ int most() const { return static_cast<int>(step >> 32) + 1; }  // no range is longer
    // floor(x / step) for x = (row + 1) 2^32 - 1, by the reciprocal floor(2^64 / step): at most one too small
    __device__ int worker_of(int row) const
    {
        const int w = static_cast<int>(__umul64hi((static_cast<uint64_t>(row) + 1 << 32) - 1, per_step));
        return w + (first(w + 1) <= row);
    }
};

// A thread's place in a [B][N][C] tensor, walked one row at a time
struct Walk {
    char *p;

    __device__ __forceinline__ Walk(const RowsView &v, int b, int n, int size) : p(v.p + (b * v.b + n * v.n) * size) {}
    __device__ __forceinline__ void next(const RowsView &v, int size, int rows = 1) { p += rows * v.n * size; }
    // after the last token's next(): to the next batch's first
    __device__ __forceinline__ void wrap(const RowsView &v, int N, int size) { p += (v.b - N * v.n) * size; }
};

// What a thread knows of its row: its channels, and the CTA's exchange of the warps' sums. MULTI: the CTA may hold
// several rows, each in `lanes` lanes of a warp or in up to two warps; else one. LN: a layer norm is among the norms (RMS
// alone needs no means).
template <int K, int P, bool MULTI, bool LN>
struct Row {
    static constexpr int E = 2 * P;
    int C, lanes, warps, turn;
    float inv_c, inv_held;  // 1 / channels of the row, of this warp's part of it
    bool on[K];
    unsigned c[K];
    float *buf;   // [2][4][kMaxWarps]: the warps' sums
    float *held;  // channels that each warp holds
    int base, warp;  // where the row's warps are in these (rows of up to two warps: four places each), this warp there

    __device__ __forceinline__ Row(int C_, int tpr, float *buf_)
    {
        C = C_;
        lanes = MULTI ? min(tpr, 32) : 32;
        warps = MULTI ? max(1, tpr / 32) : tpr / 32;
        const int t = MULTI ? threadIdx.x % tpr : threadIdx.x, rows = MULTI ? blockDim.x / tpr : 1;
        base = MULTI && rows > 1 && warps > 1 ? 4 * (threadIdx.x / tpr) : 0;
        warp = t / 32;
        buf = buf_ + base;
        held = buf_ + 8 * kMaxWarps + base;
        turn = 0;
        inv_c = inv_held = 1.0f / static_cast<float>(C);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = E * (t + k * tpr);
            on[k] = at < C;
            c[k] = at;  // not looked at where the unit is off
        }
        if (warps > 1) {
            for (int i = threadIdx.x; i < 9 * kMaxWarps; i += blockDim.x) {
                float n = 0.0f;  // the sums of warps that are not there stay zero, and they hold nothing
                const int w = rows > 1 ? (i - 8 * kMaxWarps) % 4 : i - 8 * kMaxWarps;
                if (i >= 8 * kMaxWarps && w < warps)
                    for (int k = 0; k < K; ++k) n += E * min(32, max(0, C / E - k * tpr - 32 * w));
                buf_[i] = n;
            }
            __syncthreads();
            inv_held = 1.0f / held[warp];
        }
    }

    template <int M>
    __device__ __forceinline__ void lanes_sum(float (&v)[M]) const
    {
        if (MULTI) {
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
            for (int m = 0; m < M; ++m) b[m * kMaxWarps + warp] = v[m];
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

    // -mean where a unit is on, 0 where it is off: adding it leaves units that are off at zero
    __device__ __forceinline__ f2 minus(float mean, int k) const { return twice(on[k] ? -mean : 0.0f); }
    // v - mean, for a mean's minus(); nothing to do without a layer norm
    static __device__ __forceinline__ f2 centred(f2 v, f2 off) { return LN ? add2(v, off) : v; }

    // Mean (0 but for LAYER) and mean square about it of M rows at once, one exchange; read(m, k, v) gives unit k of row
    // m, zeros where it is off. The spread is taken about each warp's own mean and joined exactly:
    // sum_w (spread_w + n_w (mean_w - mean)^2), no cancellation for rows far from zero.
    template <int M, typename Read>
    __device__ __forceinline__ void stats(const Read &read, const int (&kind)[M], float (&mean)[M], float (&square)[M])
    {
#pragma unroll
        for (int m = 0; m < M; ++m) mean[m] = 0.0f;
        if (LN) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
                f2 q = twice(0.0f);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    f2 v[P];
                    read(m, k, v);
#pragma unroll
                    for (int i = 0; i < P; ++i) q = add2(q, v[i]);
                }
                mean[m] = two(q);
            }
            lanes_sum(mean);
#pragma unroll
            for (int m = 0; m < M; ++m) mean[m] = kind[m] == BSA_NORM_LAYER ? mean[m] * inv_held : 0.0f;
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            f2 q = twice(0.0f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const f2 off = minus(mean[m], k);
                f2 v[P];
                read(m, k, v);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const f2 x = centred(v[i], off);
                    q = fma2(x, x, q);
                }
            }
            square[m] = two(q);
        }
        lanes_sum(square);
        if (warps > 1) {
            float s[LN ? 2 * M : M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                s[m] = square[m];
                if (LN) s[(LN ? M : 0) + m] = mean[m];
            }
            const float *b = exchange(s);
#pragma unroll
            for (int m = 0; m < M; ++m) square[m] = total(b + m * kMaxWarps);
            if (LN) {
#pragma unroll
                for (int m = 0; m < M; ++m) {
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
        }
#pragma unroll
        for (int m = 0; m < M; ++m) square[m] *= inv_c;
    }
};

constexpr int kExchangeFloats = 9 * kMaxWarps;

// ------------------------------------------------------------ host

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

// Workers: as many as fit on the device at once, each with an equal share of the rows; at most one per row. A worker is
// a row's threads, or (teams) a CTA: several rows of up to 1024 channels side by side in up to 128 threads, no more of them
// than a group has rows.
inline Shape shape_of(const bsa_gated_norm_desc &d, int regs, int sms, int stages, int thread_bytes, int kept_bytes = 0,
                      bool teams = false)
{
    Shape s;
    s.rg.rows = d.B * d.N;
    s.rg.per_group = d.N / d.F;
    s.tpr = row_threads(d.C / 8, V);
    s.threads = s.tpr < (teams ? 128 : 32) ? 128 / s.tpr * s.tpr : s.tpr;
    if (teams) {
        while (s.threads / s.tpr > s.rg.per_group && s.threads > 32) s.threads /= 2;
        if (s.threads > s.tpr) kept_bytes += 32 * V;  // where the teams' sums meet
    }
    s.smem = static_cast<size_t>(s.threads) * (stages * thread_bytes + kept_bytes);
    const int by_regs = 65536 / ((regs + 7) / 8 * 8 * s.threads);
    const int by_smem = static_cast<int>((228 * 1024) / (s.smem + 4096));
    int resident = by_regs < by_smem ? by_regs : by_smem;
    if (resident > 2048 / s.threads) resident = 2048 / s.threads;
    if (resident > 32) resident = 32;
    if (resident < 1) resident = 1;
    const int per_cta = teams ? 1 : s.threads / s.tpr;
    const int64_t fill = static_cast<int64_t>(sms) * resident * per_cta,
                  most = teams ? gated_norm_max_workers(s.rg.rows, d.C) : s.rg.rows;
    s.rg.workers = static_cast<int>(fill < most ? fill : most);
    s.rg.step = ((static_cast<uint64_t>(s.rg.rows) << 32) + s.rg.workers - 1) / s.rg.workers;
    s.rg.per_step = UINT64_MAX / s.rg.step;
    s.rg.long_groups = s.rg.per_group >= s.rg.most();
    s.ctas = (s.rg.workers + per_cta - 1) / per_cta;
    return s;
}

// run(stream dtype, branch dtype, registers per thread, whether the CTA holds several rows, whether there is a post norm,
// whether a layer norm is among the norms) for the kernel that a desc needs. Rows of up to MULTI threads share a CTA.
// Registers: 168, or 128 where 168 do not fit (more than 384 threads; 320 with an fp32 branch, so that the backward pass
// has room for two rows in flight) or, mostly, where they leave room for only half as many CTAs (224 and 256 threads, that
// is 3080 to 4096 channels). The backward pass of an fp32 stream with a post norm has the fewest registers to spare, and
// takes fewer CTAs there. us with 168 and with 128, 4096 channels: forward, 32768 rows bf16, 206 and 195, layer norms 328
// and 225; backward, 8192 rows, bf16 119 and 121, layer norms 154 and 150, no post norm 94 and 79; fp32 stream 132 and 147,
// no post norm 119 and 120. 320 threads, backward, 4096 rows: 89 and 117.
template <int MULTI, bool BACKWARD, typename F>
bsa_status by_kernel(const bsa_gated_norm_desc &d, F &&run)
{
    auto by_width = [&](auto ts, auto tb, auto post, auto ln) {
        const int threads = row_threads(d.C / 8, V);
        const std::integral_constant<int, 168> regs;
        const bool halved = 65536 / (128 * threads) >= 2 * (65536 / (168 * threads)),
                   rather = BACKWARD && post.value && sizeof(ts) == 4;
        if (threads > most_threads(168, false, sizeof(tb)) || (threads > 128 && halved && !rather))
            return run(ts, tb, std::integral_constant<int, 128>(), std::false_type(), post, ln);
        return threads <= MULTI ? run(ts, tb, regs, std::true_type(), post, ln) : run(ts, tb, regs, std::false_type(), post, ln);
    };
    auto by_norms = [&](auto ts, auto tb) {
        const bool ln = d.post.kind == BSA_NORM_LAYER || d.pre.kind == BSA_NORM_LAYER;
        if (d.post.kind != BSA_NORM_NONE)
            return ln ? by_width(ts, tb, std::true_type(), std::true_type()) : by_width(ts, tb, std::true_type(), std::false_type());
        return ln ? by_width(ts, tb, std::false_type(), std::true_type()) : by_width(ts, tb, std::false_type(), std::false_type());
    };
    if (d.stream_dt == BSA_BF16) return by_norms(__nv_bfloat16(), __nv_bfloat16());
    if (d.branch_dt == BSA_BF16) return by_norms(float(), __nv_bfloat16());
    return by_norms(float(), float());
}

}  // namespace
}  // namespace bsa
