// rotary.cu -- rotary positions with several axes, the per-head RMS norm of Q and K, and the
// change from the projection's layout to the attention's, in one pass; and its backward pass.
//
// Per token n, head and channel pair (a, b) of axis s:
//   u = x * rsqrt(mean x^2 + eps) * w,  t = pos[n][s] * f,
//   y_a = u_a cos t - u_b sin t,  y_b = u_b cos t + u_a sin t.
// Each element is read once and written once and takes about ten operations: HBM bounds it. 16640 tokens of 24 heads of
// 128 bf16: 102 us forward, 133 us backward with the norm, 6.0 and 6.2 TB/s (89% and 90% of a plain copy's rate).
//
// Split: d / 16 threads hold one head of one token, 16 channels (8 pairs) each. A CTA of 256 threads takes a tile of
// tokens and `together` heads at a time, and walks over the heads of Q, then K, then V, so that a thread's eight
// angles, the one costly part, are computed once for all its heads of a token. Heads are taken together so that both
// layouts are met in long runs: per token `together` heads side by side, per head the tile's tokens side by side.
// The work, (tiles) x (groups of heads) in that order, is cut into equal ranges, one per CTA that fits on the device
// at once: no last wave that is only partly full.
//
// Loads: each thread copies its own 16 channels of the next heads to shared memory with cp.async, some steps
// ahead, and reads them back itself: loads stay in flight across heads and tiles, and no barrier guards the buffers.
//
// Angles: frequencies are 64-bit fixed point in turns, so pos * f modulo one turn is the low 64 bits of an integer
// product. The nearest quarter turn is taken off its top 32 bits as they are, and what remains, an eighth of a turn at
// most, goes to fp32: the conversion is off by at most 2^-27 half turns, the bits left out by 2^-31, whatever the
// position, without fp64 or a slow argument reduction. (Converted before the quarter is taken off, the angle would be off
// by four times as much.) On top comes the plan's rounding of the frequency times the position: |pos * f| 2^-51 radians
// and |pos| 2^-65 turns, 2^-34 turns at most.
#include "block_internal.h"
#include "pairs.cuh"
#include "ptx.cuh"

#include <atomic>
#include <type_traits>

namespace bsa {
namespace {

constexpr int kThreads = 256;
// CTAs per SM, and steps in flight per thread, forward and backward. More of either is slower although the kernels
// wait for memory: what is asked for at once then comes from more places than the memory keeps open (16640 tokens of 24
// heads of 128 bf16, us: forward two CTAs of three, four, five stages 105.3, 101.9, 104.6, three CTAs of four 117.0,
// one of eight 139.6; backward two CTAs of three and four stages 133.8 and 139.7, one of six 166.5).
constexpr int kResident = 2, kForwardStages = 4, kBackwardStages = 3;

// Heads side by side in a step: the largest power of two up to kTogether that divides all the head counts, as long as
// there are kSteps steps of Q and K to a tile. With one, a token's row is read 256 bytes at a time, with eight, a head's
// rows are written 1 KB at a time, and either way the memory's pages are opened more often (d = 128 bf16, 16640 tokens of
// 24 heads, us forward and backward: one 115.6 and 152.5, two 111.8 and 145.8, four 101.9 and 133.2, eight 113.1 and
// 149.7). But each of the threads that share a token computes its angles, and few steps do not make up for that (three
// batches of 57314 tokens, two heads: two together 169, one 117; 65536 tokens of 16 heads: four together 264, two 254).
constexpr int kTogether = 4, kSteps = 12;

// What a thread holds of a head: 16 channels in groups of 16 bytes (GROUP channels), from c[g] on, dealt out so that a
// warp's accesses are contiguous; and which of its 8 pairs turn (bits). Pair j is
//   INTERLEAVED: channels 2i and 2i + 1 of a group;  HALVES: channel i of a group of the first half, and of its partner
template <typename T>
struct Lane {
    static constexpr int GROUP = 16 / sizeof(T), GROUPS = 16 / GROUP;
    int c[GROUPS];
    unsigned turns;
};

// the index of pair j
template <typename T, bool HALVES>
__device__ __forceinline__ int pair_of(const Lane<T> &l, int j)
{
    constexpr int G = Lane<T>::GROUP;
    return HALVES ? l.c[j / G] + j % G : l.c[j / (G / 2)] / 2 + j % (G / 2);
}

template <typename T, int D, bool HALVES>
__device__ __forceinline__ Lane<T> lane_of(int t, int rot)
{
    constexpr int G = Lane<T>::GROUP, N = Lane<T>::GROUPS;
    Lane<T> l;
    // HALVES: rot is a multiple of 16, so that all pairs of a thread turn, or none
    const int turning = HALVES ? rot / 16 : D / 16;
    const bool first = t < turning;
#pragma unroll
    for (int g = 0; g < N; ++g) {
        if (!HALVES)
            l.c[g] = G * t + g * (D / N);
        else if (first)
            l.c[g] = G * t + g % (N / 2) * G * turning + g / (N / 2) * (rot / 2);
        else
            l.c[g] = rot + G * (t - turning) + g * G * (D / 16 - turning);
    }
    l.turns = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) l.turns |= (first && pair_of<T, HALVES>(l, j) < rot / 2 ? 1u : 0u) << j;
    return l;
}

// sin and cos of r half turns, |r| <= 1 / 4: their Taylor series, coefficients pi^k / k!, pi itself in two parts. The first
// terms left out are below 1.8e-9; cos is off by at most 1.2 units of 2^-24 and sin by 0.9, apart from r's own rounding.
// sincospif would take a quarter turn off again (three batches of 57314 tokens, two heads: 121 against 117 us).
__device__ __forceinline__ void sin_cos(float r, float &s, float &c)
{
    const float q = r * r;
    s = fmaf(fmaf(fmaf(0.0821458866f, q, -0.599264529f), q, 2.55016404f), q, -5.16771278f);
    s = fmaf(r, 3.14159274f, r * fmaf(s, q, -8.74227801e-08f));
    c = fmaf(fmaf(fmaf(-0.0258068914f, q, 0.23533063f), q, -1.33526277f), q, 4.05871213f);
    c = fmaf(fmaf(c, q, -4.9348022f), q, 1.0f);
}

template <typename T, int D, bool HALVES>
__device__ __forceinline__ void angles(const bsa_rotary_plan &plan, const int *pos, const Lane<T> &l, float (&cs)[8],
                                       float (&sn)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        cs[j] = 1.0f;
        sn[j] = 0.0f;
        if (l.turns >> j & 1u) {
            const int p = pair_of<T, HALVES>(l, j);
            const uint64_t ph = plan.turns[p] * static_cast<uint64_t>(static_cast<int64_t>(pos[plan.axis[p] * (kThreads * 16 / D)]));
            // the nearest of four quarter turns in the top two bits, what lies beyond it in the others, from -2^29 on
            const uint32_t v = static_cast<uint32_t>(ph >> 32) + 0x20000000u;
            const int32_t rest = static_cast<int32_t>(v & 0x3fffffffu) - 0x20000000;
            float s, c;
            sin_cos(static_cast<float>(rest) * 4.656612873077393e-10f, s, c);  // 2^-31 half turns
            const bool swap = v & 0x40000000u;
            sn[j] = __uint_as_float(__float_as_uint(swap ? c : s) ^ (v & 0x80000000u));
            cs[j] = __uint_as_float(__float_as_uint(swap ? s : c) ^ (v + 0x40000000u & 0x80000000u));
        }
    }
}

// A thread's 16 channels are held as pairs of neighbours, group after group. The channels of its pair j among them:
template <bool HALVES>
__host__ __device__ constexpr int a_of(int j)
{
    return HALVES ? j : 2 * j;
}
template <bool HALVES>
__host__ __device__ constexpr int b_of(int j)
{
    return HALVES ? 8 + j : 2 * j + 1;
}

__device__ __forceinline__ void channels_of(const f2 (&u)[8], float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) split(u[i], x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ void pairs_of(const float (&x)[16], f2 (&u)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = pair(x[2 * i], x[2 * i + 1]);
}

// Turns the thread's eight pairs by their angles (DIR = 1) or back (DIR = -1). Channels that do not turn pass through
// as they are (no product with zero: an infinity stays one).
template <bool HALVES, int DIR>
__device__ __forceinline__ void turn(f2 (&u)[8], const float (&cs)[8], const float (&sn)[8], unsigned turns)
{
    float x[16], y[16];
    channels_of(u, x);
    if (turns == 0xffu) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int a = a_of<HALVES>(j), b = b_of<HALVES>(j);
            y[a] = x[a] * cs[j] - x[b] * (DIR * sn[j]);
            y[b] = x[b] * cs[j] + x[a] * (DIR * sn[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int a = a_of<HALVES>(j), b = b_of<HALVES>(j);
            const bool on = turns >> j & 1u;
            y[a] = on ? x[a] * cs[j] - x[b] * (DIR * sn[j]) : x[a];
            y[b] = on ? x[b] * cs[j] + x[a] * (DIR * sn[j]) : x[b];
        }
    }
    pairs_of(y, u);
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ f2 sum_squares(const f2 (&u)[8])
{
    f2 q = mul2(u[0], u[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) q = fma2(u[i], u[i], q);
    return q;
}

// What a CTA keeps in shared memory besides the stages: the weights of Q and K (ones where there is none), and the
// positions of the tokens of the tiles in flight, copied ahead like the heads by the threads that share the token.
template <int D, int STAGES>
struct Side {
    float weight[2][D];
    int pos[STAGES][BSA_ROTARY_MAX_AXES][kThreads * 16 / D];

    __device__ __forceinline__ void weights(const RotaryArgs &a)
    {
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            const float *w = a.norm ? a.t[i / D].weight : nullptr;
            weight[i / D][i % D] = w ? w[i % D] : 1.0f;
        }
    }
    __device__ __forceinline__ void positions(const RotaryArgs &a, int tile, int b, int n)
    {
        const int axis = threadIdx.x % (D / 16);  // at least four threads to a token
        if (axis >= a.plan.n_axes) return;
        const int32_t *from = a.positions + b * a.pos_batch + static_cast<int64_t>(n) * a.plan.n_axes + axis;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                         smem_u32(&pos[tile % STAGES][axis][threadIdx.x / (D / 16)])),
                     "l"(from)
                     : "memory");
    }
    // the positions of the thread's token, one axis every kThreads * 16 / D entries
    __device__ __forceinline__ const int *at(int tile) const { return &pos[tile % STAGES][0][threadIdx.x / (D / 16)]; }
    // 16 channels of a tensor's weight
    template <typename T>
    __device__ __forceinline__ void read(int s, const Lane<T> &l, f2 (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            constexpr int G = Lane<T>::GROUP;
            const float4 v = *reinterpret_cast<const float4 *>(&weight[s][l.c[2 * i / G] + 2 * i % G]);
            f[i] = pair(v.x, v.y);
            f[i + 1] = pair(v.z, v.w);
        }
    }
};

// The work: units of `together` heads of one tile of `tokens` tokens, heads of Q, K, V in order within a tile.
struct Work {
    int64_t units;
    int groups;  // of heads, of Q, K and V
    int together, tokens;
};

// A place in the work, the same for the whole CTA: tile, tensor, first head of the group.
struct Place {
    int tile, s, h;

    __device__ __forceinline__ Place(int64_t unit, const Work &w, const RotaryArgs &a)
    {
        tile = static_cast<int>(unit / w.groups);
        h = static_cast<int>(unit % w.groups) * w.together;
        s = 0;
        while (h >= a.t[s].heads) h -= a.t[s++].heads;
    }
    // to the next group; true where the tensor or the tile changed
    __device__ __forceinline__ bool next(const Work &w, const RotaryArgs &a)
    {
        h += w.together;
        if (h < a.t[s].heads) return false;
        h = 0;
        do {
            if (++s == 3) {
                s = 0;
                ++tile;
            }
        } while (a.t[s].heads == 0);
        return true;
    }
};

// A thread's token of a tile: (b, n), the last one for threads past it (shuffles take whole warps; they are not live)
struct Token {
    int b, n;
    bool live;

    __device__ __forceinline__ Token(int tile, int tokens, int mine, const RotaryArgs &a)
    {
        const int64_t at = static_cast<int64_t>(tile) * tokens + mine;
        const int all = a.B * a.N;
        live = at < all;
        const int token = live ? static_cast<int>(at) : all - 1;
        b = token / a.N;
        n = token % a.N;
    }
};

// 16 channels of a thread, from global memory to its own place in a stage
template <typename T>
__device__ __forceinline__ void copy_groups(uint32_t to, const char *from, const Lane<T> &l)
{
#pragma unroll
    for (int g = 0; g < Lane<T>::GROUPS; ++g) cp_async16(to + g * kThreads * 16, from + l.c[g] * sizeof(T));
}

// from there
template <typename T>
__device__ __forceinline__ void read_groups(const char *at, f2 (&u)[8])
{
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const uint4 r = *reinterpret_cast<const uint4 *>(at + g * kThreads * 16);
            u[4 * g] = widen(r.x), u[4 * g + 1] = widen(r.y), u[4 * g + 2] = widen(r.z), u[4 * g + 3] = widen(r.w);
        }
    } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 r = *reinterpret_cast<const float4 *>(at + g * kThreads * 16);
            u[2 * g] = pair(r.x, r.y), u[2 * g + 1] = pair(r.z, r.w);
        }
    }
}

// and to global memory; rounded to nearest even where T is bf16
template <typename T>
__device__ __forceinline__ void write_groups(char *to, const Lane<T> &l, const f2 (&u)[8])
{
#pragma unroll
    for (int g = 0; g < Lane<T>::GROUPS; ++g) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4 *>(to + l.c[g] * 2) =
                make_uint4(narrow(u[4 * g]), narrow(u[4 * g + 1]), narrow(u[4 * g + 2]), narrow(u[4 * g + 3]));
        } else {
            float4 r;
            split(u[2 * g], r.x, r.y);
            split(u[2 * g + 1], r.z, r.w);
            *reinterpret_cast<float4 *>(to + l.c[g] * 4) = r;
        }
    }
}

template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads, kResident) rotary_kernel(const __grid_constant__ RotaryArgs a, Work work)
{
    constexpr int STAGES = kForwardStages, LANES = D / 16, STAGE = kThreads * 16 * sizeof(T);
    extern __shared__ __align__(16) char ring[];
    const int t = threadIdx.x % LANES, mine = threadIdx.x / LANES % work.tokens, head = threadIdx.x / LANES / work.tokens;
    const Lane<T> l = lane_of<T, D, HALVES>(t, a.plan.rot);
    const int64_t u0 = work.units * blockIdx.x / gridDim.x, u1 = work.units * (blockIdx.x + 1) / gridDim.x;
    const int count = static_cast<int>(u1 - u0);
    char *const own = ring + threadIdx.x * 16;
    __shared__ __align__(16) Side<D, STAGES> side;

    Place ahead(u0, work, a);
    const char *src = nullptr;
    int tile_ahead = -1;
    auto enter_src = [&] {
        const HeadsView &v = a.t[ahead.s];
        const Token k(ahead.tile, work.tokens, mine, a);
        if (ahead.s < 2 && ahead.tile != tile_ahead) {
            __syncwarp();  // every thread of the token has read the positions that are overwritten
            side.positions(a, tile_ahead = ahead.tile, k.b, k.n);
        }
        src = v.src + (k.b * v.src_b + k.n * v.src_n + (ahead.h + head) * v.src_h) * sizeof(T);
    };
    bool fresh = true;  // src is to be found anew
    auto fetch = [&](int i) {  // a group of copies per step, empty past the end; a tile's positions come with its first
        if (i < count) {
            if (fresh) enter_src();
            copy_groups<T>(smem_u32(own + (i % STAGES) * STAGE), src, l);
            src += work.together * a.t[ahead.s].src_h * sizeof(T);
            fresh = ahead.next(work, a);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i);

    Place here(u0, work, a);
    bool live = false;
    float cs[8], sn[8];
    char *dst = nullptr;
    int tile = -1;  // the one whose angles are here
    auto enter = [&] {
        const HeadsView &v = a.t[here.s];
        const Token k(here.tile, work.tokens, mine, a);
        live = k.live;
        dst = v.dst + (k.b * v.dst_b + k.n * v.dst_n + (here.h + head) * v.dst_h) * sizeof(T);
        if (here.s == 2 || tile == here.tile) return;
        tile = here.tile;
        __syncwarp();  // the token's positions were copied by its other threads
        angles<T, D, HALVES>(a.plan, side.at(tile), l, cs, sn);
    };
    side.weights(a);
    __syncthreads();
    bool entered = false;
    for (int i = 0; i < count; ++i) {
        fetch(i + STAGES - 1);
        cp_async_wait_group<STAGES - 1>();
        if (!entered) enter();
        entered = true;
        f2 u[8];
        read_groups<T>(own + (i % STAGES) * STAGE, u);
        if (here.s < 2) {
            if (a.norm) {
                const f2 r = twice(rsqrtf(lanes_sum<LANES>(two(sum_squares(u))) * (1.0f / D) + a.eps));
                f2 w[8];
                side.read(here.s, l, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = mul2(u[j], mul2(r, w[j]));
            }
            turn<HALVES, 1>(u, cs, sn, l.turns);
        }
        if (live) write_groups<T>(dst, l, u);
        dst += work.together * a.t[here.s].dst_h * sizeof(T);
        entered = !here.next(work, a);
    }
}

// Backward. Two copies per head under the norm, dy and x. A thread sums the weight gradients of its 16 channels in
// registers over a run of heads, then in its own place in shared memory over its CTA's work.
template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads, kResident) rotary_backward_kernel(const __grid_constant__ RotaryArgs a, Work work)
{
    constexpr int STAGES = kBackwardStages, LANES = D / 16, STAGE = kThreads * 16 * sizeof(T);
    extern __shared__ __align__(16) char ring[];  // [stage][dy, then x with norm], then the weight gradients' sums
    __shared__ float sums[kThreads / 32][D];
    const int t = threadIdx.x % LANES, mine = threadIdx.x / LANES % work.tokens, head = threadIdx.x / LANES / work.tokens;
    const Lane<T> l = lane_of<T, D, HALVES>(t, a.plan.rot);
    const int64_t u0 = work.units * blockIdx.x / gridDim.x, u1 = work.units * (blockIdx.x + 1) / gridDim.x;
    const int count = static_cast<int>(u1 - u0), stage_bytes = a.norm ? 2 * STAGE : STAGE;
    char *const own = ring + threadIdx.x * 16;
    float4 *const dw_at = reinterpret_cast<float4 *>(ring + STAGES * stage_bytes) + threadIdx.x;  // [2][4] pieces
    if (a.partial) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dw_at[i * kThreads] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __shared__ __align__(16) Side<D, STAGES> side;

    Place ahead(u0, work, a);
    const char *src = nullptr, *xsrc = nullptr;
    int tile_ahead = -1;
    auto enter_src = [&] {
        const HeadsView &v = a.t[ahead.s];
        const Token k(ahead.tile, work.tokens, mine, a);
        if (ahead.s < 2 && ahead.tile != tile_ahead) {
            __syncwarp();  // every thread of the token has read the positions that are overwritten
            side.positions(a, tile_ahead = ahead.tile, k.b, k.n);
        }
        src = v.src + (k.b * v.src_b + k.n * v.src_n + (ahead.h + head) * v.src_h) * sizeof(T);
        xsrc = v.x + (k.b * v.x_b + k.n * v.x_n + (ahead.h + head) * v.x_h) * sizeof(T);
    };
    bool fresh = true;  // src is to be found anew
    auto fetch = [&](int i) {
        if (i < count) {
            if (fresh) enter_src();
            const HeadsView &v = a.t[ahead.s];
            const uint32_t to = smem_u32(own + (i % STAGES) * stage_bytes);
            copy_groups<T>(to, src, l);
            if (a.norm && ahead.s < 2) copy_groups<T>(to + STAGE, xsrc, l);
            src += work.together * v.src_h * sizeof(T);
            xsrc += work.together * v.x_h * sizeof(T);
            fresh = ahead.next(work, a);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i);

    Place here(u0, work, a);
    bool live = false;
    float cs[8], sn[8];
    f2 w[8], dw[8] = {};
    char *dst = nullptr;
    int tile = -1;
    auto enter = [&] {
        const HeadsView &v = a.t[here.s];
        const Token k(here.tile, work.tokens, mine, a);
        live = k.live;
        dst = v.dst + (k.b * v.dst_b + k.n * v.dst_n + (here.h + head) * v.dst_h) * sizeof(T);
        if (here.s == 2) return;
        if (tile != here.tile) {
            tile = here.tile;
            __syncwarp();  // the token's positions were copied by its other threads
            angles<T, D, HALVES>(a.plan, side.at(tile), l, cs, sn);
        }
        side.read(here.s, l, w);
    };
    auto leave = [&](int s) {  // the end of a run of heads of one tensor
        if (!a.partial || s == 2) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 v = dw_at[(4 * s + i) * kThreads];
            float d[4];
            split(dw[2 * i], d[0], d[1]);
            split(dw[2 * i + 1], d[2], d[3]);
            v.x += d[0], v.y += d[1], v.z += d[2], v.w += d[3];
            dw_at[(4 * s + i) * kThreads] = v;
            dw[2 * i] = dw[2 * i + 1] = twice(0.0f);
        }
    };
    side.weights(a);
    __syncthreads();
    bool entered = false;
    for (int i = 0; i < count; ++i) {
        fetch(i + STAGES - 1);
        cp_async_wait_group<STAGES - 1>();
        if (!entered) enter();
        entered = true;
        const char *at = own + (i % STAGES) * stage_bytes;
        f2 g[8];
        read_groups<T>(at, g);
        if (here.s < 2) {
            turn<HALVES, -1>(g, cs, sn, l.turns);
            if (a.norm) {
                f2 x[8], sv = twice(0.0f);
                read_groups<T>(at + STAGE, x);
                const float ss = two(sum_squares(x));
                f2 p[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    p[j] = mul2(g[j], x[j]);
                    sv = fma2(p[j], w[j], sv);
                }
                const float r = rsqrtf(lanes_sum<LANES>(ss) * (1.0f / D) + a.eps);
                const float m = lanes_sum<LANES>(two(sv)) * (1.0f / D) * r * r;
                const f2 rr = twice(r), mr = twice(-m * r);
                if (live) {  // the clamped token is not counted again
#pragma unroll
                    for (int j = 0; j < 8; ++j) dw[j] = fma2(p[j], rr, dw[j]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = fma2(mul2(g[j], w[j]), rr, mul2(x[j], mr));
            }
        }
        if (live) write_groups<T>(dst, l, g);
        dst += work.together * a.t[here.s].dst_h * sizeof(T);
        const int s = here.s;
        entered = !here.next(work, a);
        if (i + 1 == count || !entered) leave(s);
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
                if (threadIdx.x % 32 < LANES) sums[threadIdx.x / 32][l.c[j / Lane<T>::GROUP] + j % Lane<T>::GROUP] = v[e];
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
    w->together = kTogether;
    for (const HeadsView &t : a.t)
        while (t.heads % w->together != 0) w->together /= 2;
    while (w->together > 1 && a.t[0].heads + a.t[1].heads < kSteps * w->together) w->together /= 2;
    w->tokens = kThreads / (D / 16) / w->together;
    const int64_t tiles = (static_cast<int64_t>(a.B) * a.N + w->tokens - 1) / w->tokens;
    w->groups = (a.t[0].heads + a.t[1].heads + a.t[2].heads) / w->together;
    w->units = tiles * w->groups;
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
    constexpr int SMEM = kThreads * kForwardStages * 16 * sizeof(T);
    static std::atomic<uint64_t> done{0};
    const bsa_status ok = allow_smem(kern, SMEM, done);
    if (ok != BSA_OK) return ok;
    Work w;
    const int ctas = work_of<D>(a, sms, kResident, &w);
    kern<<<ctas, kThreads, SMEM, st>>>(a, w);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <typename T, int D, bool HALVES>
bsa_status backward(const RotaryArgs &a, int sms, cudaStream_t st)
{
    auto kern = rotary_backward_kernel<T, D, HALVES>;
    constexpr int STAGE = kThreads * 16 * sizeof(T), SUMS = kThreads * 128;
    static std::atomic<uint64_t> done{0};
    // fp32 with the norm and a dweight takes 128 KB of shared memory, which leaves one CTA per SM (16640 tokens of 24
    // heads of 128: 272 us, 6.0 TB/s). The forms that take less, 48 KB without the norm, go by the same rule (190 us, 6.5).
    constexpr int RESIDENT = sizeof(T) == 2 ? kResident : 1;
    const bsa_status ok = allow_smem(kern, kBackwardStages * 2 * STAGE + SUMS, done);
    if (ok != BSA_OK) return ok;
    Work w;
    int ctas = work_of<D>(a, sms, RESIDENT, &w);
    if (ctas > kRotaryMaxCtas) ctas = kRotaryMaxCtas;
    kern<<<ctas, kThreads, kBackwardStages * (a.norm ? 2 : 1) * STAGE + (a.partial ? SUMS : 0), st>>>(a, w);
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
