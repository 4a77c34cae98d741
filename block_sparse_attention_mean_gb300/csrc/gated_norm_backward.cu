// gated_norm_backward.cu -- the backward pass of the gated norm (gated_norm.cu), in one pass over the rows.
// A CTA walks a contiguous range of the rows, its teams (the threads that hold a row; one team for rows of more than
// 1024 channels) side by side, never past the end of a group (the rows that share a modulation) in one step. A thread keeps
// four sums per channel in registers,
//   A = sum dz,  S = sum dz n,  P = sum dx,  Q = sum dx m      (m = y without a post norm),
// from which every parameter's gradient follows by factors that are constant over the group:
//   dshift = A,  dscale = w S + b A,  dgate = alpha (w2 Q + b2 P),
//   dpre_weight = sum_g (1 + scale_g) S_g,  dpre_bias = sum_g (1 + scale_g) A_g,
//   dpost_weight = alpha sum_g gate_g Q_g,  dpost_bias = alpha sum_g gate_g P_g.
// At the end of a group the CTA adds its teams' sums and writes them into one of its two slots; a second kernel adds the
// slots in the order of the CTAs, so that results do not depend on timing. Where groups are shorter than the longest
// range (long_groups == 0), a CTA that held a whole group writes its modulations' gradients itself, and adds up the sums
// for the weights in a third slot.
//
// 16384 rows of 2048 channels bf16, RMS norms before and after, all gradients, 16 groups: 88 us, 4.6 TB/s (68% of a plain
// copy's rate). Each further row costs 4.1 ns, 89% of that rate; the rest is the start, the slots (8 KB a CTA and sum) and the
// second kernel, 20 us together. The four sums take 64 registers per thread, which leaves 12 warps per SM; kept in tensor
// memory they leave 16, but each row then waits for them four times (111 against 93 us).
#include "gated_norm.cuh"

namespace bsa {
namespace {

// Which of the sums A, S, P, Q (bits 0 to 3) the gradients that are asked for need, and whether those of weights are among
// them. The others are neither written nor read: most blocks have no norm with a bias behind the branch, and need no P.
struct Wants {
    unsigned sums;
    bool weights;

    __device__ __forceinline__ explicit Wants(const NormArgs &a)
    {
        const bool A = a.dshift || a.dpre_b || (a.dscale && a.d.pre.bias), S = a.dscale || a.dpre_w,
                   P = a.dpost_b || (a.dgate && a.d.post.bias), Q = a.dgate || a.dpost_w;
        sums = A | S << 1 | P << 2 | Q << 3;
        weights = a.dpre_w || a.dpre_b || a.dpost_w || a.dpost_b;
    }
    __device__ __forceinline__ bool has(int k) const { return sums >> k & 1u; }
};

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

// a group's sums, weighted for the parameters that all groups share
template <int P>
__device__ __forceinline__ void weight(const bsa_gated_norm_desc &d, int g, int c, f2 (&sA)[P], f2 (&sS)[P], f2 (&sP)[P],
                                       f2 (&sQ)[P])
{
    const int b = g / d.F, f = g % d.F;
    if (d.scale.ptr) {
        times_one_plus(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c, sA);
        times_one_plus(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c, sS);
    }
    if (d.gate.ptr) {
        times(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c, sP);
        times(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c, sQ);
    }
#pragma unroll
    for (int j = 0; j < P; ++j) sP[j] = mul2(sP[j], twice(d.alpha)), sQ[j] = mul2(sQ[j], twice(d.alpha));
}

// Adds one of the sums over the teams, in their order, into the first team's registers. shared: C floats per team.
template <int K, int P, typename R>
__device__ __forceinline__ void join_teams(f2 (&v)[K][P], const R &rw, int team, int teams, float *shared)
{
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (rw.on[k]) Unit<float, P>::put(shared + team * rw.C + rw.c[k], v[k]);
    __syncthreads();
    for (int c = 4 * threadIdx.x; c < rw.C; c += 4 * blockDim.x) {
        float4 s = *reinterpret_cast<const float4 *>(shared + c);
        for (int t = 1; t < teams; ++t) {
            const float4 q = *reinterpret_cast<const float4 *>(shared + t * rw.C + c);
            s.x += q.x, s.y += q.y, s.z += q.z, s.w += q.w;
        }
        *reinterpret_cast<float4 *>(shared + c) = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (rw.on[k] && team == 0) Unit<float, P>::get(shared + rw.c[k], v[k]);
    __syncthreads();
}

template <typename TS, typename TB, int REGS, bool MULTI, bool POST, bool LN>
__global__ void __maxnreg__(REGS) gated_norm_backward_kernel(const __grid_constant__ NormArgs a, Ranges rg, int tpr)
{
    constexpr int E = 16 / sizeof(TS), P = E / 2, K = 8 * V / E, SB = E * sizeof(TS), BB = E * sizeof(TB);
    constexpr int STAGES = stages_for(most_threads(REGS, MULTI, sizeof(TB)), 16 * V * (sizeof(TS) + sizeof(TB)), 64 * V);
    __shared__ __align__(16) float buf[kExchangeFloats];
    extern __shared__ __align__(16) char ring[];  // [stage][h, dh, dz, y: K units of every thread each]
    const bsa_gated_norm_desc &d = a.d;
    const bool pre = d.pre.kind != BSA_NORM_NONE, has_y = a.y.p != nullptr, has_dh = a.dh.p != nullptr;
    const int threads = blockDim.x, C = d.C;
    // where each tensor's units lie within a stage
    const int at_dh = pre ? K * threads * SB : 0, at_dz = at_dh + (has_dh ? K * threads * SB : 0),
              at_y = at_dz + (pre ? K * threads * BB : 0), stage_bytes = at_y + (has_y ? K * threads * BB : 0);
    Row<K, P, MULTI, LN> rw(C, tpr, buf);
    const Wants want(a);

    // all that depends on the CTA's rows alone is uniform
    const int worker = blockIdx.x, teams = MULTI ? threads / tpr : 1, team = MULTI ? threadIdx.x / tpr : 0;
    const int first = rg.first(worker), end = rg.first(worker + 1);
    const int b0 = first / d.N, n0 = first % d.N;
    Walk ph(a.h, b0, n0, sizeof(TS)), pdh(a.dh, b0, n0, sizeof(TS)), pdx(a.dx, b0, n0, sizeof(TS));
    Walk pdz(a.dz, b0, n0, sizeof(TB)), py(a.y, b0, n0, sizeof(TB)), pdy(a.dy, b0, n0, sizeof(TB));
    // a step: `teams` rows of one group, fewer at its end and at the end of the range
    struct Steps {
        int row, n, stop;  // first row of the step, its token; the end of its group within the range
    };
    const int first_group = first / rg.per_group;
    Steps ahead{first, n0, min(end, (first_group + 1) * rg.per_group)}, here = ahead;
    auto next_stop = [&](int stop) { return end - stop < rg.per_group ? end : stop + rg.per_group; };
    int group = first_group;
    float *const slots = a.partial + int64_t(worker) * gated_norm_worker_floats(C);
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
    auto fetch = [&] {  // copies the rows of the next step; a group of copies per step, empty past the end
        if (ahead.row < end) {
            const int rows = MULTI ? min(teams, ahead.stop - ahead.row) : 1;
            if (team < rows) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (!rw.on[k]) continue;
                    const uint32_t s_at = smem_u32(mine_s + to * stage_bytes + k * threads * SB);
                    const uint32_t b_at = smem_u32(mine_b + to * stage_bytes + k * threads * BB);
                    if (pre) {
                        copy_async<SB>(s_at, ph.p + team * a.h.n * sizeof(TS) + rw.c[k] * unsigned(sizeof(TS)));
                        copy_async<BB>(b_at + at_dz, pdz.p + team * a.dz.n * sizeof(TB) + rw.c[k] * unsigned(sizeof(TB)));
                    }
                    if (has_dh) copy_async<SB>(s_at + at_dh, pdh.p + team * a.dh.n * sizeof(TS) + rw.c[k] * unsigned(sizeof(TS)));
                    if (has_y) copy_async<BB>(b_at + at_y, py.p + team * a.y.n * sizeof(TB) + rw.c[k] * unsigned(sizeof(TB)));
                }
            }
            ph.next(a.h, sizeof(TS), rows);
            pdh.next(a.dh, sizeof(TS), rows);
            pdz.next(a.dz, sizeof(TB), rows);
            py.next(a.y, sizeof(TB), rows);
            ahead.row += rows;
            if ((ahead.n += rows) == d.N) {
                ahead.n = 0;
                ph.wrap(a.h, d.N, sizeof(TS));
                pdh.wrap(a.dh, d.N, sizeof(TS));
                pdz.wrap(a.dz, d.N, sizeof(TB));
                py.wrap(a.y, d.N, sizeof(TB));
            }
            if (ahead.row == ahead.stop) ahead.stop = next_stop(ahead.stop);
        }
        cp_async_commit();
        if (++to == STAGES) to = 0;
    };
    if (STAGES == 2) fetch();

    f2 sA[K][P] = {}, sS[K][P] = {}, sP[K][P] = {}, sQ[K][P] = {};
    // what dz and dx are multiplied by on their way to n and m: the thread's own 16-byte pieces of shared memory
    float4 *const kept = reinterpret_cast<float4 *>(ring + STAGES * stage_bytes) + threadIdx.x;
    float *const shared = reinterpret_cast<float *>(ring + STAGES * stage_bytes + threads * 64 * V);  // for several teams
    auto keep = [&](int which, int k, const f2(&v)[P]) {
#pragma unroll
        for (int j = 0; j < P; j += 2) {
            f2 two_pairs[2] = {v[j], v[j + 1]};
            Unit<float, 2>::put(kept + ((which * K + k) * (P / 2) + j / 2) * threads, two_pairs);
        }
    };
    auto kept_times = [&](int which, int k, f2(&v)[P]) {
#pragma unroll
        for (int j = 0; j < P; j += 2) {
            f2 m[2];
            Unit<float, 2>::get(kept + ((which * K + k) * (P / 2) + j / 2) * threads, m);
            v[j] = mul2(v[j], m[0]);
            v[j + 1] = mul2(v[j + 1], m[1]);
        }
    };
    auto factors = [&](int g) {
        const int b = g / d.F, f = g % d.F;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!rw.on[k]) {  // nothing is there to be read; the sums stay as they are
                const f2 none[P] = {};
                keep(0, k, none);
                keep(1, k, none);
                continue;
            }
            const int c = rw.c[k];
            f2 m[P];
            fill(1.0f, m);
            if (d.pre.weight) load_mod(d.pre.weight, BSA_FP32, c, m);
            if (d.scale.ptr) times_one_plus(d.scale.ptr, d.mod_dt, b * d.scale.batch + f * d.scale.frame + c, m);
            keep(0, k, m);
            fill(d.alpha, m);
            if (d.post.weight) times(d.post.weight, BSA_FP32, c, m);
            if (d.gate.ptr) times(d.gate.ptr, d.mod_dt, b * d.gate.batch + f * d.gate.frame + c, m);
            keep(1, k, m);
        }
    };
    factors(group);

    while (here.row < end) {
        fetch();
        cp_async_wait_group<STAGES - 1>();
        const int rows = MULTI ? min(teams, here.stop - here.row) : 1;
        const bool live = team < rows;
        const char *const here_s = mine_s + from * stage_bytes, *const here_b = mine_b + from * stage_bytes;
        if (++from == STAGES) from = 0;
        constexpr int M = POST ? 2 : 1;
        f2 v[K][P];  // h, then n; later y, then m (read from the ring a second time: registers are what is scarce)
        float mean[M], r[M];
        if (pre || POST) {
            if (LN) {
                f2 both_rows[M][K][P];
                int kind[M];
                kind[0] = d.pre.kind;
                if (POST) kind[M - 1] = d.post.kind;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    fill(0.0f, both_rows[0][k]);
                    if (pre) Unit<TS, P>::get(here_s + k * threads * SB, both_rows[0][k]);
                    if (POST) Unit<TB, P>::get(here_b + at_y + k * threads * BB, both_rows[M - 1][k]);
                }
                rw.stats(
                    [&](int m, int k, f2(&x)[P]) {
#pragma unroll
                        for (int j = 0; j < P; ++j) x[j] = both_rows[m][k][j];
                    },
                    kind, mean, r);
                r[0] = rsqrtf(r[0] + d.pre.eps);
                if (POST) r[M - 1] = rsqrtf(r[M - 1] + d.post.eps);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const f2 off = rw.minus(mean[0], k), rr = twice(r[0]);
#pragma unroll
                    for (int j = 0; j < P; ++j) v[k][j] = mul2(rw.centred(both_rows[0][k][j], off), rr);
                }
            } else {
                // one row after the other, to hold only one of them
                float square[M];
                if (POST) {
                    f2 s = twice(0.0f);
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        Unit<TB, P>::get(here_b + at_y + k * threads * BB, v[k]);
#pragma unroll
                        for (int j = 0; j < P; ++j) s = fma2(v[k][j], v[k][j], s);
                    }
                    square[M - 1] = two(s);
                    asm volatile("" ::: "memory");
                }
                f2 s = twice(0.0f);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    fill(0.0f, v[k]);
                    if (pre) Unit<TS, P>::get(here_s + k * threads * SB, v[k]);
#pragma unroll
                    for (int j = 0; j < P; ++j) s = fma2(v[k][j], v[k][j], s);
                }
                square[0] = two(s);
                rw.sums(square);
                r[0] = rsqrtf(square[0] * rw.inv_c + d.pre.eps);
                mean[0] = mean[M - 1] = 0.0f;
                if (POST) r[M - 1] = rsqrtf(square[M - 1] * rw.inv_c + d.post.eps);
                const f2 rr = twice(r[0]);
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int j = 0; j < P; ++j) v[k][j] = mul2(v[k][j], rr);
                }
            }
        }
        f2 g[K][P];  // the gradient at h, then at u
        if (pre) {
            f2 q[K][P], s0 = twice(0.0f), s1 = twice(0.0f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                Unit<TB, P>::get(here_b + at_dz + k * threads * BB, q[k]);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (live) {
                        sA[k][j] = add2(sA[k][j], q[k][j]);
                        sS[k][j] = fma2(q[k][j], v[k][j], sS[k][j]);
                    }
                }
                kept_times(0, k, q[k]);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    s0 = fma2(q[k][j], v[k][j], s0);
                    if (LN) s1 = add2(s1, q[k][j]);
                }
            }
            float s[LN ? 2 : 1] = {two(s0)};
            if (LN) s[LN ? 1 : 0] = two(s1);
            rw.sums(s);
            const f2 along = twice(-s[0] * rw.inv_c), rr = twice(r[0]);
            const float m = LN && d.pre.kind == BSA_NORM_LAYER ? s[LN ? 1 : 0] * rw.inv_c : 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const f2 off = rw.minus(m, k);
                fill(0.0f, g[k]);
                if (has_dh) Unit<TS, P>::get(here_s + at_dh + k * threads * SB, g[k]);
#pragma unroll
                for (int j = 0; j < P; ++j) g[k][j] = fma2(rr, fma2(v[k][j], along, rw.centred(q[k][j], off)), g[k][j]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) Unit<TS, P>::get(here_s + at_dh + k * threads * SB, g[k]);
        }
        if (a.dx.p && live) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (rw.on[k]) Unit<TS, P>::put(pdx.p + team * a.dx.n * sizeof(TS) + rw.c[k] * unsigned(sizeof(TS)), g[k]);
        }
        if (has_y) {
            f2 s0 = twice(0.0f), s1 = twice(0.0f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                Unit<TB, P>::get(here_b + at_y + k * threads * BB, v[k]);
                if (POST) {
                    const f2 off = rw.minus(mean[M - 1], k), rr = twice(r[M - 1]);
#pragma unroll
                    for (int j = 0; j < P; ++j) v[k][j] = mul2(rw.centred(v[k][j], off), rr);
                }
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (live) {
                        sP[k][j] = add2(sP[k][j], g[k][j]);
                        sQ[k][j] = fma2(g[k][j], v[k][j], sQ[k][j]);
                    }
                }
                kept_times(1, k, g[k]);
                if (POST) {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        s0 = fma2(g[k][j], v[k][j], s0);
                        if (LN) s1 = add2(s1, g[k][j]);
                    }
                }
            }
            if (POST) {
                float s[LN ? 2 : 1] = {two(s0)};
                if (LN) s[LN ? 1 : 0] = two(s1);
                rw.sums(s);
                const f2 along = twice(-s[0] * rw.inv_c), rr = twice(r[M - 1]);
                const float m = LN && d.post.kind == BSA_NORM_LAYER ? s[LN ? 1 : 0] * rw.inv_c : 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const f2 off = rw.minus(m, k);
#pragma unroll
                    for (int j = 0; j < P; ++j) g[k][j] = mul2(rr, fma2(v[k][j], along, rw.centred(g[k][j], off)));
                }
            }
            if (a.dy.p && live) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (rw.on[k]) Unit<TB, P>::put(pdy.p + team * a.dy.n * sizeof(TB) + rw.c[k] * unsigned(sizeof(TB)), g[k]);
            }
        }
        pdx.next(a.dx, sizeof(TS), rows);
        pdy.next(a.dy, sizeof(TB), rows);
        here.row += rows;
        if ((here.n += rows) == d.N) {
            here.n = 0;
            pdx.wrap(a.dx, d.N, sizeof(TS));
            pdy.wrap(a.dy, d.N, sizeof(TB));
        }
        if (here.row < here.stop) continue;
        // the end of a group, or of the range
        if (want.sums) {
            if (teams > 1) {
                join_teams<K, P>(sA, rw, team, teams, shared);
                join_teams<K, P>(sS, rw, team, teams, shared);
                join_teams<K, P>(sP, rw, team, teams, shared);
                join_teams<K, P>(sQ, rw, team, teams, shared);
            }
            const int64_t begin = static_cast<int64_t>(group) * rg.per_group;
            const bool whole = !rg.long_groups && begin >= first && begin + rg.per_group <= end;
            float *const slot = slots + (group == first_group ? 0 : 4 * C);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!rw.on[k]) continue;
                const int c = rw.c[k];
                if (team > 0) {
                    // the first team has their sums
                } else if (whole) {
                    write_group(a, group, c, sA[k], sS[k], sP[k], sQ[k]);
                } else {
                    if (want.has(0)) Unit<float, P>::put(slot + c, sA[k]);
                    if (want.has(1)) Unit<float, P>::put(slot + C + c, sS[k]);
                    if (want.has(2)) Unit<float, P>::put(slot + 2 * C + c, sP[k]);
                    if (want.has(3)) Unit<float, P>::put(slot + 3 * C + c, sQ[k]);
                }
                // weighted for the parameters that all groups share, and added up
                if (want.weights && !rg.long_groups && team == 0) {
                    weight(d, group, c, sA[k], sS[k], sP[k], sQ[k]);
                    float *const sum = slots + 8 * C + c;
                    if (weighed) {
                        f2 before[4][P];
#pragma unroll
                        for (int m = 0; m < 4; ++m) Unit<float, P>::get(sum + m * C, before[m]);
#pragma unroll
                        for (int j = 0; j < P; ++j) {
                            sA[k][j] = add2(sA[k][j], before[0][j]);
                            sS[k][j] = add2(sS[k][j], before[1][j]);
                            sP[k][j] = add2(sP[k][j], before[2][j]);
                            sQ[k][j] = add2(sQ[k][j], before[3][j]);
                        }
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
        here.stop = next_stop(here.stop);
        if (here.row < end) factors(++group);
    }
}

// Adds the workers' slots, kStrip channels per CTA: a warp takes four quads of channels from eight slots at a time.
//   few long groups   the warps are split into as many teams as there are groups (a power of two), each adding up one
//                     group or two, writing its modulations' gradients and weighting its sums for the parameters that all
//                     groups share; those of all teams are added in the end
//   more long groups  all workers' slots, weighted, for those parameters; further CTAs, one for each group, write its
//                     modulations' gradients (256 groups, 16384 rows of 2048 channels: 118 us with a row of CTAs per 16)
//   short groups      the weights' third slots of all workers; further CTAs, one each for the groups that workers share
constexpr int kStrip = 16, kSumsWarps = 16;

struct Quad {
    float4 v[4];  // A, S, P, Q of four channels
};

__device__ __forceinline__ void add(float4 &a, const float4 &b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }

// the sums of slots[w * stride] over w = w0, w0 + step ... w1
__device__ __forceinline__ void add_slots(const float *slots, int64_t stride, int C, int w0, int w1, int step, const Wants &want, Quad &q)
{
#pragma unroll 2
    for (int w = w0; w <= w1; w += step) {
        const float *p = slots + w * stride;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (want.has(k)) add(q.v[k], *reinterpret_cast<const float4 *>(p + k * C));
    }
}

// over the eight slots of a warp, in every lane
__device__ __forceinline__ void join_lanes(Quad &q)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            q.v[k].x += __shfl_xor_sync(0xffffffffu, q.v[k].x, o);
            q.v[k].y += __shfl_xor_sync(0xffffffffu, q.v[k].y, o);
            q.v[k].z += __shfl_xor_sync(0xffffffffu, q.v[k].z, o);
            q.v[k].w += __shfl_xor_sync(0xffffffffu, q.v[k].w, o);
        }
    }
}

// the gradients of a group that several workers share (short groups), or any number
__device__ __forceinline__ void write_cut_group(const NormArgs &a, const Ranges &rg, const Wants &want, int group, int w0, int w1)
{
    const int C = a.d.C;
    const int64_t stride = gated_norm_worker_floats(C);
    for (int c = 4 * threadIdx.x; c < C; c += 4 * blockDim.x) {
        f2 s[4][2] = {};
#pragma unroll 2
        for (int w = w0; w <= w1; ++w) {
            // it is the first in the ranges of its workers but, perhaps, that of the first of them
            const float *p = a.partial + w * stride + (w == w0 && rg.first(w) / rg.per_group != group ? 4 * C : 0) + c;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (!want.has(k)) continue;
                f2 q[2];
                Unit<float, 2>::get(p + k * C, q);
                s[k][0] = add2(s[k][0], q[0]);
                s[k][1] = add2(s[k][1], q[1]);
            }
        }
        write_group<2>(a, group, c, s[0], s[1], s[2], s[3]);
    }
}

template <int PER_SM>
__global__ void __launch_bounds__(32 * kSumsWarps, PER_SM)
    gated_norm_sums_kernel(const __grid_constant__ NormArgs a, Ranges rg, int64_t n_groups)
{
    __shared__ float4 part[kSumsWarps][4][4];  // [warp][sum][quad]
    const bsa_gated_norm_desc &d = a.d;
    const int C = d.C, strips = (C + kStrip - 1) / kStrip;
    const int64_t stride = gated_norm_worker_floats(C);
    const Wants want(a);
    grid_dependency_wait();
    if (static_cast<int>(blockIdx.x) >= strips) {
        // the group itself where there are at most as many groups as workers; else the one that the range begins inside
        const int i = blockIdx.x - strips;
        const int64_t group = n_groups <= rg.workers ? i : rg.first(i) / rg.per_group;
        const int w0 = rg.worker_of(group * rg.per_group), w1 = rg.worker_of((group + 1) * rg.per_group - 1);
        // written by its worker, or by another CTA
        if (!rg.long_groups && (w0 == w1 || (n_groups > rg.workers && i != w0 + 1))) return;
        write_cut_group(a, rg, want, static_cast<int>(group), w0, w1);
        return;
    }
    // the groups that this CTA looks at one by one; with none of them it adds up the weights' gradients alone
    const int groups = rg.long_groups && n_groups <= kSumsWarps ? static_cast<int>(n_groups) : 0;
    if (groups == 0 && !want.weights) return;

    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, quad = lane % 4, c = blockIdx.x * kStrip + 4 * quad;
    const int at = c < C ? c : 0;
    const float *const slots = a.partial + at;
    int teams = 1;
    while (2 * teams <= groups) teams *= 2;
    const int size = kSumsWarps / teams, team = warp / size, in = warp % size;  // warps of a team
    const int slice = in * 8 + lane / 4, slices = 8 * size;
    const bool writes = in == 0 && lane < 4 && c < C;
    Quad all = {};  // for the weights
    auto weighted = [&](int group, const Quad &q) {
        f2 s[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k][0] = pair(q.v[k].x, q.v[k].y), s[k][1] = pair(q.v[k].z, q.v[k].w);
        weight<2>(d, group, at, s[0], s[1], s[2], s[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float4 x;
            split(s[k][0], x.x, x.y);
            split(s[k][1], x.z, x.w);
            add(all.v[k], x);
        }
    };
    // a team's sums, in its first lanes
    auto join = [&](Quad &q) {
        join_lanes(q);
        if (size == 1) return;
        if (lane < 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) part[warp][k][quad] = q.v[k];
        }
        __syncthreads();
        if (writes) {
            for (int i = 1; i < size; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) add(q.v[k], part[warp + i][k][quad]);
            }
        }
        __syncthreads();
    };
    if (groups == 0) {
        if (!rg.long_groups) {
            add_slots(slots + 8 * C, stride, C, slice, rg.workers - 1, slices, want, all);
        } else {
            for (int w = slice; w < rg.workers; w += slices) {
                const int group = rg.first(w) / rg.per_group;
                Quad q = {};
                add_slots(slots, stride, C, w, w, 1, want, q);
                weighted(group, q);
                if ((rg.first(w + 1) - 1) / rg.per_group != group) {
                    q = Quad{};
                    add_slots(slots + 4 * C, stride, C, w, w, 1, want, q);
                    weighted(group + 1, q);
                }
            }
        }
        join(all);
    }
    for (int g0 = 0; g0 < groups; g0 += teams) {
        const int group = g0 + team;
        const bool some = group < groups;
        Quad q = {};
        if (some) {
            // a group is the first in the ranges of its workers but, perhaps, that of the first of them
            int w0 = rg.worker_of(group * rg.per_group);
            const int w1 = rg.worker_of((group + 1) * rg.per_group - 1);
            if (rg.first(w0) / rg.per_group != group) {
                if (in == 0 && lane < 4) add_slots(slots + 4 * C, stride, C, w0, w0, 1, want, q);
                ++w0;
            }
            add_slots(slots, stride, C, w0 + slice, w1, slices, want, q);
        }
        join(q);
        if (!writes || !some) continue;
        f2 s[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k][0] = pair(q.v[k].x, q.v[k].y), s[k][1] = pair(q.v[k].z, q.v[k].w);
        write_group<2>(a, group, c, s[0], s[1], s[2], s[3]);
        if (want.weights) weighted(group, q);
    }
    if (!want.weights) return;
    if (teams > 1) {
        if (in == 0 && lane < 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) part[team][k][quad] = all.v[k];
        }
        __syncthreads();
        if (warp > 0) return;
        for (int i = 1; i < teams; ++i) {
#pragma unroll
            for (int k = 0; k < 4; ++k) add(all.v[k], part[i][k][quad]);
        }
    }
    if (warp > 0 || !writes) return;
    if (a.dpre_b) *reinterpret_cast<float4 *>(a.dpre_b + c) = all.v[0];
    if (a.dpre_w) *reinterpret_cast<float4 *>(a.dpre_w + c) = all.v[1];
    if (a.dpost_b) *reinterpret_cast<float4 *>(a.dpost_b + c) = all.v[2];
    if (a.dpost_w) *reinterpret_cast<float4 *>(a.dpost_w + c) = all.v[3];
}

template <typename TS, typename TB, int REGS, bool MULTI, bool POST, bool LN>
bsa_status backward(const NormArgs &a, int sms, cudaStream_t st)
{
    auto kern = gated_norm_backward_kernel<TS, TB, REGS, MULTI, POST, LN>;
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> regs{0};
    constexpr int MOST = most_threads(REGS, MULTI, sizeof(TB)), BYTES = 16 * V * (sizeof(TS) + sizeof(TB)), KEPT = 64 * V,
                  STAGES = stages_for(MOST, BYTES, KEPT);
    const bsa_status ok = ready(kern, MOST * (STAGES * BYTES + KEPT + (MULTI ? 32 * V : 0)), done, regs);
    if (ok != BSA_OK) return ok;
    const int pre = a.d.pre.kind != BSA_NORM_NONE;
    const Shape s = shape_of(a.d, regs.load(std::memory_order_relaxed), sms, STAGES,
                             8 * V * static_cast<int>(sizeof(TS) * (pre + (a.dh.p ? 1 : 0)) + sizeof(TB) * (pre + (a.y.p ? 1 : 0))), KEPT, true);
    kern<<<s.rg.workers, s.threads, s.smem, st>>>(a, s.rg, s.tpr);
    if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
    if (a.partial == nullptr) return BSA_OK;
    const int64_t n_groups = static_cast<int64_t>(a.d.B) * a.d.F;
    const unsigned strips = (a.d.C + kStrip - 1) / kStrip;
    const unsigned cut = s.rg.long_groups && n_groups <= kSumsWarps ? 0 : static_cast<unsigned>(n_groups < s.rg.workers ? n_groups : s.rg.workers);
    const unsigned ctas = strips + cut;
    // one CTA per SM, which spills no registers, unless there are more of them than SMs (us with one and with two: 16384 rows
    // of 2048 channels, 128 CTAs, 88.4 and 90.4; 8192 rows of 4096 channels, 256 CTAs, 122.3 and 119.2)
    auto sums = ctas <= static_cast<unsigned>(sms) ? gated_norm_sums_kernel<1> : gated_norm_sums_kernel<2>;
    return pdl_launch(sums, dim3(ctas), 32 * kSumsWarps, 0, st, a, s.rg, n_groups) ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace

int64_t gated_norm_max_workers(int64_t rows, int C)
{
    const int tpr = row_threads(C / 8, V);
    const int64_t w = kNormMaxThreads / (tpr < 128 ? 128 / tpr * tpr : tpr);
    return rows < w ? rows : w;
}

bsa_status launch_gated_norm_backward(const NormArgs &a, cudaStream_t st)
{
    int sms = 0;
    const bsa_status s = current_sm_count(&sms);
    if (s != BSA_OK) return s;
    return by_kernel<64, true>(a.d, [&](auto ts, auto tb, auto regs, auto multi, auto post, auto ln) {
        return backward<decltype(ts), decltype(tb), decltype(regs)::value, decltype(multi)::value, decltype(post)::value,
                        decltype(ln)::value>(a, sms, st);
    });
}

}  // namespace bsa
