// cache_attention.cu -- attention of one new token per sequence over a paged cache (bsa_cache_attention).
//
// Every key and value is used by the H / Hk query heads of its head and by nothing else: one pass over the cache
// bounds the call (2 * d multiplications per byte-pair and head are far below the tensor cores' rate), so the
// kernel is built around keeping loads in flight everywhere at once.
//
//   * The tokens of all sequences and key heads form one row of units of 64 or 128 tokens, which is cut evenly over the
//     resident CTAs, whatever the lengths; the end of each (sequence, key head) counts as kEnd units more. Where a cut
//     falls inside a (sequence, key head), its pieces leave partial results (O, max, sums) in the workspace and the CTA
//     that finishes last joins them in the order of the tokens: in groups of kGroup, then over the groups, so that no
//     CTA reads many.
//   * Each of a CTA's four warps takes 16 or 32 tokens of a unit through a ring of its own in shared memory, filled with
//     16-byte cp.async far ahead and across the ends of sequences. Warps meet only at the end of a (sequence, head).
//   * The products run on mma.sync.m16n8k16 with the 16 tokens (then 16 channels) as rows and 8 query heads as
//     columns, S^T = K Q^T and O^T = V^T P^T: 8 heads fill the narrow side, as many as share a key head in practice, and the
//     softmax's result moves from one product to the next by transposing 8 x 8 blocks in registers. tcgen05 wants 64 or
//     more rows and operands in shared memory; at one query the tensor cores are a quarter busy at most either way.
//   * The running maximum is raised, and O rescaled, only when a score passes it by 2^8 (fp32 sums, P at most 2^8).
//   * 8-bit rows become fp16 (exact: e4m3 has 4 bits and fp16 its range). Q is scaled by a power of two to below 2
//     and rounded to fp16 (exact for all of its 8 bits down to 2^-17 of the largest); the key's exponent multiplies
//     the fp32 score, the value's is added to it in log2, so that P 2^e is what is rounded, to 11 bits, with a maximum
//     of its own near one. The softmax's sum is that of the scores alone, with a running maximum of its own: beside a value
//     of 2^40 the product of a weight and a row of zeros vanishes, the weight does not.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "cache_internal.h"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 8;              // partial results that one CTA joins at a time
constexpr int kMaxJoin = (kCacheMaxCtas + kGroup - 1) / kGroup;  // groups of one (sequence, key head), at most
static_assert(kMaxJoin >= kGroup, "room for a group's weights");
// What the end of a (sequence, key head) costs, in units: the warps' results put together, Q of the next one, the join
// (64 sequences of 100 to 8192 tokens, 8 key heads: 57 us without, 46 us with one to three of them)
constexpr int kEnd = 2;
constexpr int kSlotHeads = 16;         // query heads of a partial result
constexpr float kRaise = 8.0f;         // log2 of how far a score may pass the running maximum
constexpr float kRaiseSum = 256.0f;    // and of an 8-bit cache's weights, a thread's sum over a tile

struct Params {
    CacheView cache;
    TableView table;
    PackedView q, o;
    const int32_t *kv_lens;
    float *lse;
    int H, g, chunks, HH;  // query heads per key head; chunks of them; chunks of all key heads
    float scale;
    uint32_t *err;
    uint32_t *tickets;  // [3][kCacheMaxCtas]
    float *part_o;      // [slot][kSlotHeads][D]
    float4 *part_s;     // [slot][kSlotHeads]: Stats
};

template <int D, bool E4M3>
struct Ring {
    static constexpr int kRow = E4M3 ? D : 2 * D;  // bytes of a row
    static constexpr int kChunks = kRow / 16;
    // Tokens of a warp at a time: 32 where two rings of three stages fit an SM. The chain of one tile (page, loads, products,
    // maxima) costs about the same for 16.
    static constexpr int kTile = kRow <= 128 ? 32 : 16;
    static constexpr int kUnit = kWarps * kTile;   // tokens of a unit
    static constexpr int kData = kTile * kRow;     // K of a tile, or V
    static constexpr int kStage = 2 * kData + (E4M3 ? 2 * kTile : 0);
    static constexpr int kStages = 24576 / (2 * kData) > 6 ? 6 : 24576 / (2 * kData);
    static constexpr int kWarpBytes = kStages * kStage;
    // Floats between heads where warps join, and between a thread's runs of channels there (8-bit rows: a thread has D / 8
    // channels next to each other): no two of the threads that write together share a bank more than twice
    static constexpr int kRun = E4M3 ? D / 8 + 2 : 8;
    static constexpr int kPad = 8 * kRun * (E4M3 ? 1 : D / 64) + 4;
    static __device__ __forceinline__ int channel_at(int ch) { return E4M3 ? ch / (D / 8) * kRun + ch % (D / 8) : ch; }
    static constexpr int kJoin = kWarps * kWarpBytes;
    static constexpr int kBytes = kJoin + 2 * 8 * kPad * 4;
    // 16-byte chunk ch of row r lies at chunk swizzle(ch, r): without it the readers' rows share banks
    static __device__ __forceinline__ int k_swizzle(int ch, int r) { return E4M3 ? (D == 128 ? ch ^ ((r & 1) << 2) : ch) : ch ^ (r & 7); }
    static __device__ __forceinline__ int v_swizzle(int ch, int r)
    {
        return E4M3 ? (D == 128 ? ch ^ (((r >> 1) & 3) << 1) : ch ^ ((r >> 1) & 3)) : ch ^ (r & 7);
    }
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// c += a b: rows x 16 times 16 x 8, 16-bit operands of one type
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the two e4m3 values of a 16-bit half of w, as f16x2
__device__ __forceinline__ uint32_t half2_lo(uint32_t w)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    return h;
}
__device__ __forceinline__ uint32_t half2_hi(uint32_t w) { return half2_lo(w >> 16); }

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// tokens of sequence b in the cache; a malformed length (reported) counts as none
__device__ __forceinline__ int valid_len(const Params &p, int b)
{
    const int n = __ldg(p.kv_lens + b);
    if (n < 0 || n > (static_cast<int64_t>(p.table.width) << p.cache.page_shift)) {
        raise_error(p.err, BSA_ERR_INVALID_ARG);
        return 0;
    }
    return n;
}

// A place among the units: unit `tile` of (sequence b, chunk of heads hu)
template <int kUnit>
struct Place {
    int b, hu, tile, len;
    __device__ __forceinline__ int tiles() const { return (len + kUnit - 1) / kUnit; }
    __device__ __forceinline__ bool at_end() const { return tile + 1 >= tiles(); }
    // the next unit, or the first one of the next (sequence, chunk of heads); only called where there is one
    __device__ __forceinline__ void next(const Params &p)
    {
        if (++tile < tiles()) return;
        tile = 0;
        if (++hu < p.HH) return;
        hu = 0;
        do {
            ++b;
            len = b < p.table.B ? valid_len(p, b) : 1;
        } while (len == 0);
    }
};

// `units` cut over `ctas`: the first units % ctas of them have one more
struct Cut {
    int base, rem;
    __device__ __forceinline__ Cut(int units, int ctas) : base(units / ctas), rem(units % ctas) {}
    __device__ __forceinline__ int begin(int cta) const { return cta * base + min(cta, rem); }
    __device__ __forceinline__ int cta_of(int u) const
    {
        const int longer = rem * (base + 1);
        return u < longer ? u / (base + 1) : rem + (u - longer) / base;
    }
};

__device__ __forceinline__ size_t slot_of(int c0, int part) { return part == 0 ? 2 * c0 + 1 : 2 * (c0 + part); }

// x 2^e in two steps: 2^e alone may vanish, or be infinite, where the product is neither
__device__ __forceinline__ float scaled(float x, float e)
{
    const float h = ex2_approx(0.5f * e);
    return x * h * h;
}
// 2^(x - m), one where both are the same infinity
__device__ __forceinline__ float rescale(float x, float m) { return x == m ? 1.0f : ex2_approx(x - m); }

// What a partial result O (fp32, relative to 2^m) is divided by. bf16 cache: l the sum of the weights, lp of the rounded
// ones, both relative to 2^m. 8-bit cache: l the sum of the weights relative to 2^lm, the maximum of the scores alone, where
// m is that of the scores with their values' exponents.
struct Stats {
    float m, l, lp, lm;
};
__device__ __forceinline__ Stats load_stats(const float4 *p)
{
    const float4 v = __ldcg(p);
    return Stats{v.x, v.y, v.z, v.w};
}
// nothing
__device__ __forceinline__ Stats no_stats() { return Stats{-CUDART_INF_F, 0.0f, 0.0f, -CUDART_INF_F}; }
// the maxima of both
template <bool E4M3>
__device__ __forceinline__ void raise_stats(Stats &a, float m, float lm)
{
    a.m = fmaxf(a.m, m);
    if constexpr (E4M3) a.lm = fmaxf(a.lm, lm);
}
// adds b's sums to a's, whose maxima are b's at least
template <bool E4M3>
__device__ __forceinline__ void add_stats(Stats &a, const Stats &b)
{
    const float from = E4M3 ? b.lm : b.m, to = E4M3 ? a.lm : a.m, e = from == to ? 0.0f : from - to;
    a.l += scaled(b.l, e);
    if constexpr (!E4M3) a.lp += scaled(b.lp, e);
}

// One thread's share of a joined result: 8 channels of a head
struct Joined {
    float o[8];
    Stats s;
};

// Weights and sums of the partial results 0, step, 2 step, ... (count of them) of the parts that begin at CTA c0, left in
// shared memory for join_parts. All threads.
struct Weights {
    float w[kMaxJoin][kSlotHeads];
    Stats s[kSlotHeads];
};
template <bool E4M3>
__device__ __forceinline__ void weigh_parts(const Params &p, Weights &ws, int c0, int first, int step, int count, int heads)
{
    // eight threads a head, which take every eighth part
    static_assert(kThreads == 8 * kSlotHeads, "a thread's head and parts");
    constexpr int kEach = (kMaxJoin + 7) / 8;
    const int head = threadIdx.x / 8, j = threadIdx.x % 8;
    Stats s[kEach], all = no_stats();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = k * 8 + j;
        s[k] = no_stats();
        if (i < count && head < heads) s[k] = load_stats(p.part_s + slot_of(c0, first + i * step) * kSlotHeads + head);
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) raise_stats<E4M3>(all, s[k].m, s[k].lm);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
        raise_stats<E4M3>(all, __shfl_xor_sync(0xFFFFFFFFu, all.m, o), __shfl_xor_sync(0xFFFFFFFFu, all.lm, o));
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = k * 8 + j;
        if (i >= count || head >= heads) continue;
        ws.w[i][head] = rescale(s[k].m, all.m);
        add_stats<E4M3>(all, s[k]);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        all.l += __shfl_xor_sync(0xFFFFFFFFu, all.l, o);
        if constexpr (!E4M3) all.lp += __shfl_xor_sync(0xFFFFFFFFu, all.lp, o);
    }
    if (j == 0) ws.s[head] = all;
    __syncthreads();
}

// ... and their sum for one head and 8 channels
template <int D>
__device__ __forceinline__ Joined join_parts(const Params &p, const Weights &ws, int c0, int first, int step, int count, int head, int ch)
{
    Joined r;
    r.s = ws.s[head];
#pragma unroll
    for (int k = 0; k < 8; ++k) r.o[k] = 0.0f;
    for (int i0 = 0; i0 < count; i0 += 8) {
        float4 a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            a[k] = b[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i0 + k >= count) continue;
            const float4 *src = reinterpret_cast<const float4 *>(
                p.part_o + (slot_of(c0, first + (i0 + k) * step) * kSlotHeads + head) * D + ch);
            a[k] = __ldcg(src), b[k] = __ldcg(src + 1);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i0 + k >= count) continue;
            const float w = ws.w[i0 + k][head];
            r.o[0] += w * a[k].x, r.o[1] += w * a[k].y, r.o[2] += w * a[k].z, r.o[3] += w * a[k].w;
            r.o[4] += w * b[k].x, r.o[5] += w * b[k].y, r.o[6] += w * b[k].z, r.o[7] += w * b[k].w;
        }
    }
    return r;
}

template <bool E4M3>
__device__ __forceinline__ void write_result(const Params &p, int b, int h, int ch, const Joined &r)
{
    const Stats &s = r.s;
    const float sum = E4M3 ? s.l : s.lp, inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    float o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        o[k] = r.o[k] * inv;
        if constexpr (E4M3) o[k] = scaled(o[k], s.m == s.lm ? 0.0f : s.m - s.lm);  // (equal: also without a score)
    }
    *reinterpret_cast<uint4 *>(p.o.p + b * p.o.token + h * p.o.head + ch * 2) =
        make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
    if (ch == 0 && p.lse)
        p.lse[static_cast<int64_t>(b) * p.H + h] = ((E4M3 ? s.lm : s.m) + log2f(s.l)) * 0.69314718055994530942f;
}

template <int D, bool E4M3, int NH>
__global__ void __launch_bounds__(kThreads, 2) cache_attention_kernel(const Params p)
{
    using R = Ring<D, E4M3>;
    constexpr int KS = D / 16;  // steps of 16 channels
    constexpr int kTile = R::kTile, kUnit = R::kUnit, kHalves = kTile / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int scan[kWarps];
    __shared__ int found[3];  // sequence, unit within it, length
    __shared__ Stats st[kWarps][8 * NH];
    __shared__ uint32_t arrived;
    __shared__ Weights weights;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, j = lane & 3;
    const int cta = blockIdx.x;

    // units in front of each thread's run of sequences, and of all (the host keeps them below 2^31)
    const int run = (p.table.B + kThreads - 1) / kThreads;
    const int b_lo = min(p.table.B, tid * run), b_hi = min(p.table.B, b_lo + run);
    const int own_len = cta < p.table.B ? valid_len(p, cta) : 1;  // see the end: started with the other loads
    int mine = 0, len = 0;
    auto cost = [&](int n) { return n > 0 ? (n + kUnit - 1) / kUnit + kEnd : 0; };
    for (int b = b_lo; b < b_hi; ++b) {
        len = valid_len(p, b);
        mine += cost(len);
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int units = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scan[w];
        units += scan[w];
    }
    units *= p.HH;
    before *= p.HH;
    // sequences without tokens
    for (int b = cta; b < p.table.B; b += gridDim.x) {
        if ((b == cta ? own_len : valid_len(p, b)) != 0) continue;
        for (int i = tid; i < p.H * (D / 8); i += kThreads)
            *reinterpret_cast<uint4 *>(p.o.p + b * p.o.token + (i / (D / 8)) * p.o.head + (i % (D / 8)) * 16) = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse)
            for (int h = tid; h < p.H; h += kThreads) p.lse[static_cast<int64_t>(b) * p.H + h] = -CUDART_INF_F;
    }
    // every CTA that takes part has a unit, so that the parts of a (sequence, head) belong to consecutive ones
    const int ctas = min(static_cast<int>(gridDim.x), units);
    if (cta >= ctas) return;
    const Cut cut(units, ctas);
    const int u_lo = cut.begin(cta), u_hi = cut.begin(cta + 1);
    if (u_lo >= before && u_lo < before + mine * p.HH) {
        int at = before;
        for (int b = b_lo; b < b_hi; ++b) {
            if (run > 1) len = valid_len(p, b);
            const int n = cost(len) * p.HH;
            if (u_lo < at + n) {
                found[0] = b, found[1] = u_lo - at, found[2] = len;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    Place<kUnit> here;
    here.b = found[0];
    here.len = found[2];
    here.hu = found[1] / (here.tiles() + kEnd);
    here.tile = found[1] - here.hu * (here.tiles() + kEnd);
    int u = u_lo;  // where `here` is in the row
    if (here.tile >= here.tiles()) {  // the cut is in the end of one: the next one begins behind it
        u += here.tiles() + kEnd - here.tile;
        if (u >= u_hi) return;
        here.tile = here.tiles() - 1;
        here.next(p);
    }

    // ---- Q of a (sequence, chunk of heads): loads first, the rest when they are needed
    uint32_t qf[NH][KS][2];
    float qs[NH][2];  // scale of the scores of heads 2j and 2j + 1
    auto load_q = [&](const Place<kUnit> &w) {
        const int kh = w.hu / p.chunks, head0 = (w.hu % p.chunks) * 8 * NH;  // of the group
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const int head = head0 + n * 8 + r;
            const bool real = head < p.g;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(
                p.q.p + w.b * p.q.token + static_cast<int64_t>(kh * p.g + (real ? head : 0)) * p.q.head);
#pragma unroll
            for (int t = 0; t < KS; ++t) {
                qf[n][t][0] = qf[n][t][1] = 0u;
                if (!real) continue;
                if constexpr (E4M3) {  // channels c .. c + 3, as the thread reads them from K's rows
                    const int c = D == 128 ? (j + 4 * (t >> 2)) * 16 + 4 * (t & 3) : j * 16 + 4 * t;
                    const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src + c / 2));
                    qf[n][t][0] = x.x, qf[n][t][1] = x.y;
                } else {
                    qf[n][t][0] = __ldg(src + t * 8 + j), qf[n][t][1] = __ldg(src + t * 8 + j + 4);
                }
            }
        }
    };
    auto ready_q = [&]() {
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            qs[n][0] = qs[n][1] = p.scale;
            if constexpr (E4M3) {
                uint32_t big = 0u;
#pragma unroll
                for (int t = 0; t < KS; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) big = max(big, max((qf[n][t][k] << 16) & 0x7FFFFFFFu, qf[n][t][k] & 0x7FFF0000u));
                big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                // |q| < 2 after division by 2^E; a row below 2^-126 keeps its values (they are zero in fp16)
                const int E = max(-126, min(126, static_cast<int>(big >> 23) - 127));
                const float down = __uint_as_float(static_cast<uint32_t>(127 - E) << 23);
                const float up = p.scale * __uint_as_float(static_cast<uint32_t>(127 + E) << 23);
#pragma unroll
                for (int t = 0; t < KS; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        qf[n][t][k] = pack_half2(__uint_as_float(qf[n][t][k] << 16) * down,
                                                 __uint_as_float(qf[n][t][k] & 0xFFFF0000u) * down);
                qs[n][0] = __shfl_sync(0xFFFFFFFFu, up, 8 * j);
                qs[n][1] = __shfl_sync(0xFFFFFFFFu, up, 8 * j + 4);
            }
        }
    };
    load_q(here);

    // ---- the warp's ring: `ahead` runs kStages - 1 units in front of `here`
    const uint32_t ring = smem_u32(smem) + warp * R::kWarpBytes;
    Place<kUnit> ahead = here;
    int issued = u;  // where `ahead` is
    const int page_mask = (1 << p.cache.page_shift) - 1;
    auto page_of = [&](const Place<kUnit> &w, int half) -> int {
        const int tok = w.tile * kUnit + warp * kTile + half * 16;
        if (tok >= w.len) return 0;  // no page is looked up; its rows become zeros
        return __ldg(p.table.pages + w.b * p.table.stride + (tok >> p.cache.page_shift));
    };
    // a tile of 32 tokens may lie in two pages of 16
    auto pages_of = [&](const Place<kUnit> &w, int (&page)[kHalves]) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) page[h] = page_of(w, h);
    };
    auto copy = [&](int stage, const Place<kUnit> &w, const int (&page)[kHalves]) {
        const int tok = w.tile * kUnit + warp * kTile;
        const int left = w.len - tok;  // tokens of the tile that exist
        if (left > 0) {
            const int kh = w.hu / p.chunks;
            const uint32_t at = ring + stage * R::kStage;
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const bool ok = page[h] >= 0 && page[h] < p.cache.n_pages;
                if (!ok) raise_error(p.err, BSA_ERR_INVALID_ARG);
                const int64_t row =
                    ok ? ((static_cast<int64_t>(page[h]) * p.cache.heads + kh) << p.cache.page_shift) + ((tok + h * 16) & page_mask) : 0;
                const char *ks = p.cache.k + row * R::kRow, *vs = p.cache.v + row * R::kRow;
#pragma unroll
                for (int i = 0; i < R::kChunks / 2; ++i) {
                    const int idx = i * 32 + lane, rr = idx / R::kChunks + h * 16, ch = idx % R::kChunks;
                    const uint32_t bytes = ok && rr < left ? 16u : 0u;  // rows that do not exist become zeros
                    cp_async16(at + rr * R::kRow + R::k_swizzle(ch, rr) * 16, ks + idx * 16, bytes);
                    cp_async16(at + R::kData + rr * R::kRow + R::v_swizzle(ch, rr) * 16, vs + idx * 16, bytes);
                }
                if constexpr (E4M3)
                    if (lane < 2)
                        cp_async16(at + 2 * R::kData + lane * kTile + h * 16, (lane ? p.cache.v_exp : p.cache.k_exp) + row, ok ? 16u : 0u);
            }
        }
    };
    int page[kHalves];  // of `ahead`
    auto advance = [&]() -> bool {  // of `ahead`
        issued += ahead.at_end() ? 1 + kEnd : 1;
        if (issued >= u_hi) return false;
        ahead.next(p);
        return true;
    };
    auto load = [&](int stage) {
        if (issued < u_hi) {
            copy(stage, ahead, page);
            if (advance()) pages_of(ahead, page);
        }
        cp_async_commit();
    };
    {  // the first stages: all page numbers are on their way before the first is needed
        Place<kUnit> first[R::kStages - 1];
        int first_page[R::kStages - 1][kHalves];
        bool there[R::kStages - 1];
#pragma unroll
        for (int s = 0; s < R::kStages - 1; ++s) {
            first[s] = ahead;
            there[s] = issued < u_hi;
            if (there[s]) {
                pages_of(ahead, first_page[s]);
                advance();
            }
        }
        if (issued < u_hi) pages_of(ahead, page);
#pragma unroll
        for (int s = 0; s < R::kStages - 1; ++s) {
            if (there[s]) copy(s, first[s], first_page[s]);
            cp_async_commit();
        }
    }

    float m[NH][2], l[NH][2], lp[NH][2], lm[NH][2];  // as in Stats
    float o[KS][NH][4];        // O^T: rows are channels, columns heads 2j and 2j + 1
    int stage = 0;
    while (u < u_hi) {
        // ---- a (sequence, chunk of heads): its units in this CTA are [here.tile, end)
        const int tiles = here.tiles(), first = here.tile;
        const int whole = u - first;  // its first unit
        const int end = min(tiles, u_hi - whole);
        const int b = here.b, kh = here.hu / p.chunks, head0 = (here.hu % p.chunks) * 8 * NH;  // of the group
        ready_q();
#pragma unroll
        for (int n = 0; n < NH; ++n) {
#pragma unroll
            for (int k = 0; k < 2; ++k) m[n][k] = lm[n][k] = -CUDART_INF_F, l[n][k] = lp[n][k] = 0.0f;
#pragma unroll
            for (int t = 0; t < KS; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[t][n][k] = 0.0f;
        }

        for (int tile = first; tile < end; ++tile, ++u) {
            load((stage + R::kStages - 1) % R::kStages);
            cp_async_wait_group<R::kStages - 1>();
            __syncwarp();
            const int left = here.len - tile * kUnit - warp * kTile;
            if (left > 0) {
                const uint32_t ka = ring + stage * R::kStage, va = ka + R::kData;
                float s[kHalves][NH][4];  // S^T: rows are tokens, columns heads
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    float s2[NH][2][4];  // two sums, of every other step
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) s2[n][0][k] = s2[n][1][k] = 0.0f;
                    if constexpr (E4M3) {
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            const int r0 = h * 16 + r;
                            const uint4 lo = lds128(ka + r0 * R::kRow + R::k_swizzle(j + 4 * c, r0) * 16);
                            const uint4 hi = lds128(ka + (r0 + 8) * R::kRow + R::k_swizzle(j + 4 * c, r0 + 8) * 16);
                            const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                            for (int t = 0; t < 4; ++t) {
                                const uint32_t a[4] = {half2_lo(wl[t]), half2_lo(wh[t]), half2_hi(wl[t]), half2_hi(wh[t])};
#pragma unroll
                                for (int n = 0; n < NH; ++n) mma16816<true>(s2[n][t & 1], a, qf[n][4 * c + t][0], qf[n][4 * c + t][1]);
                            }
                        }
                    } else {
                        const int row = h * 16 + (lane & 15);
#pragma unroll
                        for (int t = 0; t < KS; ++t) {
                            uint32_t a[4];
                            ldmatrix4(a, ka + row * R::kRow + R::k_swizzle(2 * t + (lane >> 4), row) * 16);
#pragma unroll
                            for (int n = 0; n < NH; ++n) mma16816<false>(s2[n][t & 1], a, qf[n][t][0], qf[n][t][1]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) s[h][n][k] = s2[n][0][k] + s2[n][1][k];
                }
                // scores in log2, of tokens r and r + 8 of each half
                float ve[kHalves][2];  // exponents of the values
                auto product = [&](int h, int n, int k) { return E4M3 ? s[h][n][k] + ve[h][k >> 1] : s[h][n][k]; };
                bool pass = false;
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    const bool in[2] = {h * 16 + r < left, h * 16 + r + 8 < left};
                    float ke[2] = {1.0f, 1.0f};
                    if constexpr (E4M3) {
                        const uint32_t ea = ka + 2 * R::kData + h * 16 + r;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            ke[t] = __uint_as_float(lds8(ea + 8 * t) << 23);
                            ve[h][t] = static_cast<float>(static_cast<int>(lds8(ea + kTile + 8 * t)) - 127);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float x = s[h][n][k] * (E4M3 ? qs[n][k & 1] * ke[k >> 1] : qs[n][k & 1]);
                            x = in[k >> 1] ? x : -CUDART_INF_F;
                            s[h][n][k] = x;
                            pass |= product(h, n, k) > m[n][k & 1] + kRaise;
                        }
                }
                // the maximum of the scores alone, and the sum relative to it
                auto raise_sums = [&]() {
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float x = lm[n][c];
#pragma unroll
                            for (int h = 0; h < kHalves; ++h) x = fmax3(x, s[h][n][c], s[h][n][2 + c]);
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, w));
                            l[n][c] *= rescale(lm[n][c], x);
                            lm[n][c] = x;
                        }
                };
                if (__any_sync(0xFFFFFFFFu, pass)) {
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float x = m[n][c];
#pragma unroll
                            for (int h = 0; h < kHalves; ++h) x = fmax3(x, product(h, n, c), product(h, n, 2 + c));
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, w));
                            const float a = rescale(m[n][c], x);
                            m[n][c] = x;
                            if constexpr (!E4M3) l[n][c] *= a, lp[n][c] *= a;
#pragma unroll
                            for (int t = 0; t < KS; ++t) o[t][n][c] *= a, o[t][n][2 + c] *= a;
                        }
                    if constexpr (E4M3) raise_sums();
                }
                if constexpr (E4M3) {
                    float sum[NH][2];
                    auto weights = [&]() -> bool {  // false: some are far above the maximum that they are relative to
                        bool small = true;
#pragma unroll
                        for (int n = 0; n < NH; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float base = lm[n][c] == -CUDART_INF_F ? 0.0f : lm[n][c];
                                sum[n][c] = 0.0f;
#pragma unroll
                                for (int h = 0; h < kHalves; ++h)
                                    sum[n][c] += ex2_approx(s[h][n][c] - base) + ex2_approx(s[h][n][2 + c] - base);
                                small &= !(sum[n][c] > kRaiseSum);  // NaN stays
                            }
                        return __all_sync(0xFFFFFFFFu, small);
                    };
                    if (!weights()) {  // the scores rise while the values' exponents fall
                        raise_sums();
                        weights();
                    }
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) l[n][c] += sum[n][c];
                }
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    uint32_t pf[NH][2];
#pragma unroll
                    for (int n = 0; n < NH; ++n) {
                        float w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float base = m[n][k & 1] == -CUDART_INF_F ? 0.0f : m[n][k & 1];
                            w[k] = ex2_approx(product(h, n, k) - base);
                            if constexpr (!E4M3) l[n][k & 1] += w[k];
                        }
                        if constexpr (E4M3) {
                            pf[n][0] = pack_half2(w[0], w[1]);
                            pf[n][1] = pack_half2(w[2], w[3]);
                        } else {
                            pf[n][0] = pack_bf16x2(w[0], w[1]);
                            pf[n][1] = pack_bf16x2(w[2], w[3]);
                            add_bf16x2_to_f32(lp[n][0], lp[n][1], pf[n][0]);
                            add_bf16x2_to_f32(lp[n][0], lp[n][1], pf[n][1]);
                        }
                        pf[n][0] = transpose8x8(pf[n][0]);
                        pf[n][1] = transpose8x8(pf[n][1]);
                    }
                    if constexpr (E4M3) {
                        // thread r has channels [r * D / 8, (r + 1) * D / 8) of tokens 2j, 2j + 1, 2j + 8, 2j + 9
                        uint32_t w[4][D / 32];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int row = h * 16 + 2 * j + (k & 1) + 8 * (k >> 1);
                            if constexpr (D == 128) {
                                const uint4 v = lds128(va + row * R::kRow + R::v_swizzle(r, row) * 16);
                                w[k][0] = v.x, w[k][1] = v.y, w[k][2] = v.z, w[k][3] = v.w;
                            } else {
                                const uint2 v = lds64(va + row * R::kRow + R::v_swizzle(r >> 1, row) * 16 + (r & 1) * 8);
                                w[k][0] = v.x, w[k][1] = v.y;
                            }
                        }
#pragma unroll
                        for (int q = 0; q < D / 32; ++q) {
                            const uint32_t a01 = __byte_perm(w[0][q], w[1][q], 0x5140), a23 = __byte_perm(w[0][q], w[1][q], 0x7362);
                            const uint32_t b01 = __byte_perm(w[2][q], w[3][q], 0x5140), b23 = __byte_perm(w[2][q], w[3][q], 0x7362);
                            const uint32_t t0[4] = {half2_lo(a01), half2_hi(a01), half2_lo(b01), half2_hi(b01)};
                            const uint32_t t1[4] = {half2_lo(a23), half2_hi(a23), half2_lo(b23), half2_hi(b23)};
#pragma unroll
                            for (int n = 0; n < NH; ++n) {
                                mma16816<true>(o[2 * q][n], t0, pf[n][0], pf[n][1]);
                                mma16816<true>(o[2 * q + 1][n], t1, pf[n][0], pf[n][1]);
                            }
                        }
                    } else {
                        const int row = h * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                        for (int t = 0; t < KS; ++t) {
                            uint32_t a[4];
                            ldmatrix4_trans(a, va + row * R::kRow + R::v_swizzle(2 * t + ((lane >> 3) & 1), row) * 16);
#pragma unroll
                            for (int n = 0; n < NH; ++n) mma16816<false>(o[t][n], a, pf[n][0], pf[n][1]);
                        }
                    }
                }
            }
            __syncwarp();  // the stage is read: the next load may overwrite it
            stage = stage + 1 == R::kStages ? 0 : stage + 1;
        }

        if (end == tiles) u += kEnd;
        if (u < u_hi) {  // the next one's Q is on its way while this one's results are put together
            here.tile = tiles - 1;
            here.next(p);
            load_q(here);
        }

        // ---- the four warps' results become one
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) {
                    l[n][h] += __shfl_xor_sync(0xFFFFFFFFu, l[n][h], w);
                    lp[n][h] += __shfl_xor_sync(0xFFFFFFFFu, lp[n][h], w);
                }
                if (r == 0) st[warp][n * 8 + 2 * j + h] = Stats{m[n][h], l[n][h], lp[n][h], lm[n][h]};
            }
        __syncthreads();
        const bool is_whole = first == 0 && end == tiles;
        const int c0 = cut.cta_of(whole), c1 = cut.cta_of(whole + tiles - 1);
        const int parts = c1 - c0 + 1, part = cta - c0;
        float *join = reinterpret_cast<float *>(smem + R::kJoin);
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            if (head0 + n * 8 >= p.g) break;
            float wt[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = n * 8 + 2 * j + h;
                const float M = fmaxf(fmaxf(st[0][c].m, st[1][c].m), fmaxf(st[2][c].m, st[3][c].m));
                wt[h] = rescale(m[n][h], M);
            }
            for (int w = 0; w < 2; ++w) {  // warps 0 and 1, then 2 and 3 into their buffers: the sum has one order
                if (w == warp >> 1) {
                    float *to = join + ((warp & 1) * 8 + 2 * j) * R::kPad;
#pragma unroll
                    for (int t = 0; t < KS; ++t)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {  // heads 2j and 2j + 1
                            const float x = o[t][n][c] * wt[c], y = o[t][n][2 + c] * wt[c];
                            if constexpr (E4M3) {
                                float2 *at = reinterpret_cast<float2 *>(to + c * R::kPad + r * R::kRun + 2 * t);
                                const float2 old = w == 0 ? make_float2(0.0f, 0.0f) : *at;
                                *at = make_float2(old.x + x, old.y + y);
                            } else {
                                float *at = to + c * R::kPad + 16 * t + r;
                                at[0] = w == 0 ? x : at[0] + x;
                                at[8] = w == 0 ? y : at[8] + y;
                            }
                        }
                }
                __syncthreads();
            }
            for (int i = tid; i < D; i += kThreads) {  // 8 heads, D / 8 lanes of 8 channels
                const int hd = i / (D / 8), ch = (i % (D / 8)) * 8, c = n * 8 + hd;
                if (head0 + c >= p.g) continue;
                Joined res;
                res.s = no_stats();
#pragma unroll
                for (int w = 0; w < kWarps; ++w) raise_stats<E4M3>(res.s, st[w][c].m, st[w][c].lm);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) add_stats<E4M3>(res.s, st[w][c]);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int at = hd * R::kPad + R::channel_at(ch + k);
                    res.o[k] = join[at] + join[8 * R::kPad + at];
                }
                if (is_whole) {
                    write_result<E4M3>(p, b, kh * p.g + head0 + c, ch, res);
                } else {
                    const size_t row = slot_of(c0, part) * kSlotHeads + c;
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + row * D + ch);
                    dst[0] = make_float4(res.o[0], res.o[1], res.o[2], res.o[3]);
                    dst[1] = make_float4(res.o[4], res.o[5], res.o[6], res.o[7]);
                    if (ch == 0) p.part_s[row] = make_float4(res.s.m, res.s.l, res.s.lp, res.s.lm);
                }
            }
            __syncthreads();
        }
        if (!is_whole) {
            // The last of a group of kGroup parts joins them, the last group joins the groups. A ticket is indexed by the
            // CTA of the group's first part; the first group's and the final ones have rows of their own, since a CTA
            // can be in the middle of one (sequence, head) and begin another.
            const int group = part / kGroup, groups = (parts + kGroup - 1) / kGroup;
            const int members = min(kGroup, parts - group * kGroup);
            auto last_of = [&](uint32_t *ticket, int count) -> bool {
                __syncthreads();  // the CTA's results are written; what one thread releases and acquires holds for all
                if (tid == 0) {
                    uint32_t before_me;
                    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before_me) : "l"(ticket) : "memory");
                    if (before_me == static_cast<uint32_t>(count - 1)) *ticket = 0u;  // for the next call
                    arrived = before_me;
                }
                __syncthreads();
                const bool last = arrived == static_cast<uint32_t>(count - 1);
                __syncthreads();  // `arrived` may be written again
                return last;
            };
            const int heads = min(8 * NH, p.g - head0);
            if (last_of(p.tickets + (group == 0 ? 0 : kCacheMaxCtas) + c0 + group * kGroup, members)) {
                const bool final_join = groups == 1;
                weigh_parts<E4M3>(p, weights, c0, group * kGroup, 1, members, heads);
                constexpr int kRounds = 8 * NH * (D / 8) / kThreads > 0 ? 8 * NH * (D / 8) / kThreads : 1;
                Joined res[kRounds];
#pragma unroll
                for (int k = 0; k < kRounds; ++k) {  // all loads first
                    const int i = k * kThreads + tid, hd = i / (D / 8), ch = (i % (D / 8)) * 8;
                    if (hd < heads) res[k] = join_parts<D>(p, weights, c0, group * kGroup, 1, members, hd, ch);
                }
                // the group's result takes the place of its first part, which has been read
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kRounds; ++k) {
                    const int i = k * kThreads + tid, hd = i / (D / 8), ch = (i % (D / 8)) * 8;
                    if (hd >= heads) continue;
                    if (final_join) {
                        write_result<E4M3>(p, b, kh * p.g + head0 + hd, ch, res[k]);
                        continue;
                    }
                    const size_t row = slot_of(c0, group * kGroup) * kSlotHeads + hd;
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + row * D + ch);
                    dst[0] = make_float4(res[k].o[0], res[k].o[1], res[k].o[2], res[k].o[3]);
                    dst[1] = make_float4(res[k].o[4], res[k].o[5], res[k].o[6], res[k].o[7]);
                    if (ch == 0) p.part_s[row] = make_float4(res[k].s.m, res[k].s.l, res[k].s.lp, res[k].s.lm);
                }
                if (!final_join && last_of(p.tickets + 2 * kCacheMaxCtas + c0, groups)) {
                    weigh_parts<E4M3>(p, weights, c0, 0, kGroup, groups, heads);
                    for (int i = tid; i < heads * (D / 8); i += kThreads) {
                        const int hd = i / (D / 8), ch = (i % (D / 8)) * 8;
                        write_result<E4M3>(p, b, kh * p.g + head0 + hd, ch, join_parts<D>(p, weights, c0, 0, kGroup, groups, hd, ch));
                    }
                }
            }
        }
    }
    cp_async_wait_group<0>();
}

template <int D, bool E4M3, int NH>
bsa_status launch(const CacheAttentionArgs &a, cudaStream_t st)
{
    using R = Ring<D, E4M3>;
    auto kern = cache_attention_kernel<D, E4M3, NH>;
    static_assert(2 * (R::kBytes + 1024 + 6528) <= 233472, "two CTAs per SM");
    static std::atomic<uint64_t> ready{0};
    if (!allow_shared_memory(kern, R::kBytes, ready)) return BSA_ERR_CUDA;
    int sms = 0;
    const bsa_status s = current_sm_count(&sms);
    if (s != BSA_OK) return s;
    Params p;
    p.cache = a.cache;
    p.table = a.table;
    p.q = a.q;
    p.o = a.o;
    p.kv_lens = a.kv_lens;
    p.lse = a.lse;
    p.H = a.H;
    p.g = a.H / a.cache.heads;
    p.chunks = (p.g + 8 * NH - 1) / (8 * NH);
    p.HH = p.chunks * a.cache.heads;
    p.scale = a.scale * 1.44269504088896340736f;
    p.err = reinterpret_cast<uint32_t *>(a.ws);
    p.tickets = reinterpret_cast<uint32_t *>(a.ws + kCacheTickets);
    p.part_s = reinterpret_cast<float4 *>(a.ws + kCacheScratch);
    p.part_o = reinterpret_cast<float *>(a.ws + kCacheScratch + sizeof(float4) * 2 * kCacheMaxCtas * kSlotHeads);
    const int ctas = 2 * sms < kCacheMaxCtas ? 2 * sms : kCacheMaxCtas;
    kern<<<ctas, kThreads, R::kBytes, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <int D, bool E4M3>
bsa_status launch_heads(const CacheAttentionArgs &a, cudaStream_t st)
{
    return a.H / a.cache.heads <= 8 ? launch<D, E4M3, 1>(a, st) : launch<D, E4M3, 2>(a, st);
}

}  // namespace

size_t cache_attention_workspace(int d)
{
    return sizeof(float4) * 2 * kCacheMaxCtas * kSlotHeads + sizeof(float) * 2 * kCacheMaxCtas * kSlotHeads * d;
}

bsa_status launch_cache_attention(const CacheAttentionArgs &a, cudaStream_t st)
{
    if (a.d == 128) return a.cache.e4m3 ? launch_heads<128, true>(a, st) : launch_heads<128, false>(a, st);
    return a.cache.e4m3 ? launch_heads<64, true>(a, st) : launch_heads<64, false>(a, st);
}

}  // namespace bsa
