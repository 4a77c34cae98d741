// cache_rows.cu -- rows of keys and values into the pages of a cache (bsa_cache_write) and back (bsa_cache_read).
//
// Both move each row once and compute next to nothing: memory bounds them. A row of d channels belongs to d / 8
// lanes, 16 bytes of bf16 each; a unit of work is HEADS rows (heads) of one token, of K or of V, all loaded before
// the first is used, so that a thread has 64 bytes in flight and finds its token's sequence and page once for them: four
// rows, and eight of a large 8-bit call, whose arithmetic weighs more (65536 tokens, 16 heads of 128: 173 us written
// with four, 163 us with eight; bf16 loses 6% with eight, and a call of 64 tokens 0.5 us).
//
// 8-bit rows: the exponent of a row is that of its largest magnitude a, found with log2(d / 8) shuffles on the bits of
// |x| (the order of floats of one sign is that of their bits), two channels in a word (15717 tokens, 8 heads of 128: 25.4 us
// with one at a time). a = m 2^E with 1 <= m < 2, and 448 = 1.75 * 2^8, so
// the least e with a <= 448 * 2^e is E - 8 where m <= 1.75, else E - 7. x * 2^-e is exact in fp32 (all its bits stay,
// |x * 2^-e| <= 448 and e4m3's least step is 2^-9: what falls below fp32's range rounds to zero either way) and is
// rounded once, by cvt.rn.satfinite.e4m3x2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cache_internal.h"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kCheckCtas = 64;  // that look at the sequences, at most

// tokens that a sequence's row of the table has room for
__device__ __forceinline__ int64_t room(const CacheRowsArgs &a) { return static_cast<int64_t>(a.table.width) << a.cache.page_shift; }

// Reports sequences that are malformed: a token finds one sequence, and what is wrong with others (those between that decrease,
// those that no token falls in) shows nowhere else. The first `ctas` of the launch do nothing else, so that short calls do not
// wait for it. WRITE: the lengths too.
template <bool WRITE>
__device__ __forceinline__ void check_sequences(const CacheRowsArgs &a, int ctas)
{
    for (int64_t b = blockIdx.x * kThreads + threadIdx.x; b < a.table.B; b += ctas * kThreads) {
        const int begin = a.cu ? __ldg(a.cu + b) : 0, end = a.cu ? __ldg(a.cu + b + 1) : 1;
        bool ok = begin >= 0 && end >= begin && end <= a.T;
        const int64_t n = static_cast<int64_t>(end) - begin, len = WRITE ? __ldg(a.kv_lens + b) : n;
        ok = ok && len >= n && len <= room(a);
        if (!ok) raise_error(a.err, BSA_ERR_INVALID_ARG);
    }
}

// Sequence of packed token t: the last b with cu[b] <= t (of an ordered cu). False for a token of no sequence, and of a
// malformed one. [t - cu[b], cu[b + 1] - cu[b]) is returned as (at, n).
__device__ __forceinline__ bool find_sequence(const int32_t *cu, int B, int T, int t, int &b, int &at, int &n)
{
    int lo = 0, hi = B;  // cu[lo] <= t < cu[hi], if at all
    if (t < __ldg(cu) || t >= __ldg(cu + B)) return false;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid;
        else hi = mid;
    }
    const int begin = __ldg(cu + lo), end = __ldg(cu + lo + 1);
    b = lo;
    at = t - begin;
    n = end - begin;
    return begin >= 0 && end <= T && begin <= t && end > t;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 2^e for e in [-126, 127]
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// two values to e4m3 (lo in the low byte)
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Exponent of a row whose largest finite magnitude has the bf16 bits a
__device__ __forceinline__ int row_exp(uint32_t a)
{
    const int E = static_cast<int>(a >> 7) - 127;  // a below 2^-126 has E = -127: clamped all the same
    const int e = E - ((a & 0x7Fu) <= 0x60u ? 8 : 7);
    return max(-100, min(119, e));
}

// The unit (token, K or V, group of heads) of a thread, and its lane within a row
template <int D, int HEADS>
struct Unit {
    int t, kv, h0, lane;
    bool any;
    __device__ __forceinline__ Unit(unsigned cta, int64_t T, int groups)
    {
        constexpr int LPR = D / 8;
        const int64_t u = (static_cast<int64_t>(cta) * kThreads + threadIdx.x) / LPR;
        lane = threadIdx.x % LPR;
        any = u < T * 2 * groups;
        const int64_t r = u / groups;
        h0 = static_cast<int>(u - r * groups) * HEADS;
        t = static_cast<int>(r >> 1);
        kv = static_cast<int>(r & 1);
    }
};

// element offset of row `row` of a page's head, in rows
__device__ __forceinline__ int64_t row_of(const CacheView &c, int page, int head, int row)
{
    return ((static_cast<int64_t>(page) * c.heads + head) << c.page_shift) + row;
}

template <int D, bool E4M3, int HEADS>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheRowsArgs a, int groups, int check_ctas)
{
    if (static_cast<int>(blockIdx.x) < check_ctas) {
        check_sequences<true>(a, check_ctas);
        return;
    }
    constexpr int LPR = D / 8;
    const Unit<D, HEADS> u(blockIdx.x - check_ctas, a.T, groups);
    // the rows are on their way while their place is looked up: the tensor has them, whether a sequence does or not
    const PackedView &src = u.kv ? a.v : a.k;
    int heads = u.any ? min(HEADS, a.cache.heads - u.h0) : 0;
    uint4 x[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (i < heads)
            x[i] = __ldg(reinterpret_cast<const uint4 *>(src.p + u.t * src.token + (u.h0 + i) * src.head) + u.lane);
    }
    bool ok = u.any;
    int b = 0, at = 0, n = 1, page = 0, row = 0;
    if (ok) {
        if (a.cu) ok = find_sequence(a.cu, a.table.B, a.T, u.t, b, at, n);
        else b = u.t;
    }
    if (ok) {
        const int len = __ldg(a.kv_lens + b);
        const int64_t place = static_cast<int64_t>(len) - n + at;
        ok = len >= n && len <= room(a);
        if (ok) {
            page = __ldg(a.table.pages + b * a.table.stride + (place >> a.cache.page_shift));
            row = static_cast<int>(place & ((1 << a.cache.page_shift) - 1));
            ok = page >= 0 && page < a.cache.n_pages;
            if (!ok) raise_error(a.err, BSA_ERR_INVALID_ARG);
        }
    }
    if (!ok) heads = 0;
    char *data = u.kv ? a.cache.v : a.cache.k;
    if constexpr (!E4M3) {
#pragma unroll
        for (int i = 0; i < HEADS; ++i)
            if (i < heads) reinterpret_cast<uint4 *>(data)[row_of(a.cache, page, u.h0 + i, row) * LPR + u.lane] = x[i];
    } else {
        uint8_t *exps = u.kv ? a.cache.v_exp : a.cache.k_exp;
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
            uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            // magnitudes by their bits, two channels at a time; what is not finite counts as zero
            uint32_t big = 0u, odd = 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t mag = w[k] & 0x7FFF7FFFu, bad = __vcmpgeu2(mag, 0x7F807F80u);
                odd |= bad;
                big = __vmaxu2(big, mag & ~bad);
            }
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) big = __vmaxu2(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
            const int e = row_exp(max(big & 0xFFFFu, big >> 16));
            const float unit = exp2_int(-e);
            const uint64_t none = f2_pack(-0.0f, -0.0f);  // the addend that keeps a zero's sign
            if (odd) {  // infinities to NaN: the conversion would make them 448
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] |= __vcmpgeu2(w[k] & 0x7FFF7FFFu, 0x7F807F80u) & 0x7FFF7FFFu;
            }
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo, hi;  // subnormals as zeros: at most 2^-26 after the product, far below the least step
                f2_unpack(f2_fma(f2_pack(bf16_lo(w[k]), bf16_hi(w[k])), f2_pack(unit, unit), none), lo, hi);
                q[k] = to_e4m3x2(lo, hi);
            }
            if (i < heads) {
                const int64_t r = row_of(a.cache, page, u.h0 + i, row);
                reinterpret_cast<uint2 *>(data)[r * LPR + u.lane] = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
                if (u.lane == 0) exps[r] = static_cast<uint8_t>(e + 127);
            }
        }
    }
}

// two e4m3 values (the low half of w) times `unit`, as bf16x2
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t w, float unit)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return pack_bf16x2(lo * unit, hi * unit);
}

template <int D, bool E4M3, int HEADS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheRowsArgs a, int groups, int check_ctas)
{
    if (static_cast<int>(blockIdx.x) < check_ctas) {
        check_sequences<false>(a, check_ctas);
        return;
    }
    constexpr int LPR = D / 8;
    const Unit<D, HEADS> u(blockIdx.x - check_ctas, a.T, groups);
    if (!u.any) return;
    int b = 0, at = 0, n = 0, page = 0, row = 0;
    if (!find_sequence(a.cu, a.table.B, a.T, u.t, b, at, n) || n > room(a)) return;
    page = __ldg(a.table.pages + b * a.table.stride + (at >> a.cache.page_shift));
    row = at & ((1 << a.cache.page_shift) - 1);
    const bool there = page >= 0 && page < a.cache.n_pages;
    if (!there) raise_error(a.err, BSA_ERR_INVALID_ARG);
    const PackedView &dst = u.kv ? a.v : a.k;
    const char *data = u.kv ? a.cache.v : a.cache.k;
    const uint8_t *exps = u.kv ? a.cache.v_exp : a.cache.k_exp;
    const int heads = min(HEADS, a.cache.heads - u.h0);
    uint4 x[HEADS];
    uint2 w[HEADS];
    int e[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        w[i] = make_uint2(0u, 0u);
        e[i] = 127;
        if (i < heads && there) {
            const int64_t r = row_of(a.cache, page, u.h0 + i, row);
            if constexpr (E4M3) {
                w[i] = __ldg(reinterpret_cast<const uint2 *>(data) + r * LPR + u.lane);
                e[i] = __ldg(exps + r);
            } else {
                x[i] = __ldg(reinterpret_cast<const uint4 *>(data) + r * LPR + u.lane);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        if (i >= heads) continue;
        if constexpr (E4M3) {
            // bytes of 0, 255 and others that no row written by this library has are taken as they stand
            const float unit = e[i] == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(e[i]) << 23);
            x[i] = make_uint4(e4m3x2_to_bf16x2(w[i].x & 0xFFFFu, unit), e4m3x2_to_bf16x2(w[i].x >> 16, unit),
                              e4m3x2_to_bf16x2(w[i].y & 0xFFFFu, unit), e4m3x2_to_bf16x2(w[i].y >> 16, unit));
        }
        *(reinterpret_cast<uint4 *>(dst.p + u.t * dst.token + (u.h0 + i) * dst.head) + u.lane) = x[i];
    }
}

template <int HEADS, typename Kernel>
bsa_status launch_rows(Kernel kern, const CacheRowsArgs &a, cudaStream_t st)
{
    const int groups = (a.cache.heads + HEADS - 1) / HEADS;
    const int64_t threads = static_cast<int64_t>(a.T) * 2 * groups * (a.d / 8);
    const int check = std::min((a.table.B - 1) / kThreads + 1, kCheckCtas);
    const int64_t ctas = (threads + kThreads - 1) / kThreads + check;
    if (ctas > INT32_MAX) return BSA_ERR_SHAPE;
    kern<<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(a, groups, check);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

// eight rows a thread: 8-bit rows, enough of them to fill the device (152 SMs of 1024 threads) all the same
bool eight(const CacheRowsArgs &a)
{
    return a.cache.e4m3 && static_cast<int64_t>(a.T) * 2 * ((a.cache.heads + 7) / 8) * (a.d / 8) >= 152 * 1024;
}

template <int D>
bsa_status launch_write(const CacheRowsArgs &a, cudaStream_t st)
{
    if (eight(a)) return launch_rows<8>(cache_write_kernel<D, true, 8>, a, st);
    return a.cache.e4m3 ? launch_rows<4>(cache_write_kernel<D, true, 4>, a, st) : launch_rows<4>(cache_write_kernel<D, false, 4>, a, st);
}

template <int D>
bsa_status launch_read(const CacheRowsArgs &a, cudaStream_t st)
{
    if (eight(a)) return launch_rows<8>(cache_read_kernel<D, true, 8>, a, st);
    return a.cache.e4m3 ? launch_rows<4>(cache_read_kernel<D, true, 4>, a, st) : launch_rows<4>(cache_read_kernel<D, false, 4>, a, st);
}

}  // namespace

bsa_status launch_cache_write(const CacheRowsArgs &a, cudaStream_t st) { return a.d == 128 ? launch_write<128>(a, st) : launch_write<64>(a, st); }

bsa_status launch_cache_read(const CacheRowsArgs &a, cudaStream_t st) { return a.d == 128 ? launch_read<128>(a, st) : launch_read<64>(a, st); }

}  // namespace bsa
