// block_api.cu -- host side of the C ABI in bsa_block.h: argument checks, the rotary plan, workspace
// sizes and dispatch. Every check runs before any launch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "block_internal.h"
#include "footprint.h"

namespace {

constexpr uint32_t kPlanMagic = 0x52625341u;

bool valid_dt(int dt) { return dt == BSA_BF16 || dt == BSA_FP32; }

int size_of(int dt) { return dt == BSA_BF16 ? 2 : 4; }

bsa_status check_rotary(const bsa_rotary_plan *plan, int dt, int B, int N, const int32_t *positions, int64_t pos_batch,
                        bool turns, int norm, float eps)
{
    if (!plan || plan->magic != kPlanMagic) return BSA_ERR_INVALID_ARG;
    if (B < 1 || N < 1 || static_cast<int64_t>(B) * N > INT32_MAX) return BSA_ERR_SHAPE;
    if (!valid_dt(dt)) return BSA_ERR_DTYPE;
    // the kernels index by these: a plan changed by hand is caught here
    if ((plan->d != 64 && plan->d != 128) || plan->rot < 2 || plan->rot > plan->d || plan->rot % 2 != 0 || plan->n_axes < 1 ||
        plan->n_axes > BSA_ROTARY_MAX_AXES ||
        (plan->pairing != BSA_ROTARY_INTERLEAVED && plan->pairing != BSA_ROTARY_HALVES) ||
        (plan->pairing == BSA_ROTARY_HALVES && plan->rot % 16 != 0))
        return BSA_ERR_INVALID_ARG;
    for (int p = 0; p < plan->rot / 2; ++p)
        if (plan->axis[p] >= plan->n_axes) return BSA_ERR_INVALID_ARG;
    if (turns && (!positions || !aligned(positions, 4) || pos_batch < 0 || pos_batch > (INT64_MAX >> 32) ||
                  4.0 * (B - 1) * static_cast<double>(pos_batch) > 4.0e18))
        return BSA_ERR_INVALID_ARG;
    if (norm && !(std::isfinite(eps) && eps >= 0.0f)) return BSA_ERR_INVALID_ARG;
    return BSA_OK;
}

// scale * theta^(-2 j / dim) as f + rest. The exponent is a double and what it lacks, e + e_rest, of which the second
// comes in by theta^e_rest = 1 + e_rest log(theta); the product's rounding is kept too. What remains is the rounding of
// pow, one unit in the last place at most: 2^-52 of the value.
void frequency(double scale, double theta, int j, int dim, double *f, double *rest)
{
    const double e = -2.0 * j / dim, e_rest = std::fma(-e, static_cast<double>(dim), -2.0 * j) / dim;
    const double power = std::pow(theta, e);
    *f = scale * power;
    *rest = std::fma(scale, power, -*f) + scale * (power * (e_rest * std::log(theta)));
}

// x, at most 0.5 in magnitude, as 2^64 x modulo 2^64
uint64_t fixed(double x) { return x >= 0.5 ? uint64_t(1) << 63 : static_cast<uint64_t>(static_cast<int64_t>(std::rint(std::ldexp(x, 64)))); }

// (f + rest) / 2 pi turns in 2^-64 turns, modulo one turn: positions are whole numbers, so whole turns drop out. 1 / 2 pi
// and the product are kept in two doubles each; the remainder of a double is exact, and so is its product with 2^64.
uint64_t turns_of(double f, double rest)
{
    constexpr double kInvTwoPi = 0.15915494309189533577, kInvTwoPiRest = -9.839338337591243e-18;
    const double turns = f * kInvTwoPi, more = std::fma(f, kInvTwoPi, -turns) + f * kInvTwoPiRest + rest * kInvTwoPi;
    const double whole = std::remainder(turns, 1.0), below = std::ldexp(whole, 64) - std::rint(std::ldexp(whole, 64));
    return fixed(whole) + fixed(std::remainder(more + std::ldexp(below, -64), 1.0));
}

bsa_status check_heads(int heads) { return heads >= 1 && heads <= 65535 ? BSA_OK : BSA_ERR_SHAPE; }

bool valid_norm(const bsa_norm &n)
{
    if (n.kind == BSA_NORM_NONE) return true;
    if (n.kind != BSA_NORM_RMS && n.kind != BSA_NORM_LAYER) return false;
    if (!(std::isfinite(n.eps) && n.eps >= 0.0f)) return false;
    return (!n.weight || aligned(n.weight, 16)) && (!n.bias || aligned(n.bias, 16));
}

bool modulation_of(const bsa_modulation &m, const bsa_gated_norm_desc &d, Footprint *f)
{
    return make_footprint(m.ptr, d.B, m.batch, d.F, m.frame, 1, 0, d.C, size_of(d.mod_dt), f);
}

bool valid_modulation(const bsa_modulation &m, const bsa_gated_norm_desc &d)
{
    Footprint f;
    return !m.ptr || modulation_of(m, d, &f);
}

bool broadcast(const bsa_modulation &m, const bsa_gated_norm_desc &d)
{
    return (d.B > 1 && m.batch == 0) || (d.F > 1 && m.frame == 0);
}

bsa_status check_desc(const bsa_gated_norm_desc *d)
{
    if (!d) return BSA_ERR_INVALID_ARG;
    if (d->B < 1 || d->N < 1 || static_cast<int64_t>(d->B) * d->N > INT32_MAX) return BSA_ERR_SHAPE;
    if (d->C < 8 || d->C > 8192 || d->C % 8 != 0 || d->F < 1 || d->N % d->F != 0) return BSA_ERR_SHAPE;
    if (!valid_dt(d->stream_dt) || !valid_dt(d->branch_dt) || !valid_dt(d->mod_dt)) return BSA_ERR_DTYPE;
    if (d->stream_dt == BSA_BF16 && d->branch_dt == BSA_FP32) return BSA_ERR_DTYPE;
    if (!std::isfinite(d->alpha) || !valid_norm(d->post) || !valid_norm(d->pre)) return BSA_ERR_INVALID_ARG;
    if (!valid_modulation(d->gate, *d) || !valid_modulation(d->scale, *d) || !valid_modulation(d->shift, *d))
        return BSA_ERR_INVALID_ARG;
    if (d->pre.kind == BSA_NORM_NONE && (d->scale.ptr || d->shift.ptr)) return BSA_ERR_INVALID_ARG;
    return BSA_OK;
}

// the [B][N][C] tensor r as a footprint and a view; false if it is unusable
bool rows_of(const bsa_rows &r, const bsa_gated_norm_desc &d, int dt, Footprint *f, bsa::RowsView *v)
{
    if (!make_footprint(r.ptr, d.B, r.batch, d.N, r.token, 1, 0, d.C, size_of(dt), f)) return false;
    v->p = static_cast<char *>(r.ptr);
    v->b = d.B > 1 ? r.batch : 0;
    v->n = d.N > 1 ? r.token : 0;
    return true;
}

// a desc whose unused parts cannot mislead a kernel: norms that are off carry no weights, dimensions of
// length one no strides
bsa_gated_norm_desc tidy(const bsa_gated_norm_desc &in)
{
    bsa_gated_norm_desc d = in;
    for (bsa_norm *n : {&d.post, &d.pre})
        if (n->kind == BSA_NORM_NONE) n->weight = n->bias = nullptr;
    for (bsa_modulation *m : {&d.gate, &d.scale, &d.shift}) {
        if (d.B == 1) m->batch = 0;
        if (d.F == 1) m->frame = 0;
    }
    return d;
}

// the weights and modulations that a (tidy) desc names
void reads_parameters(const bsa_gated_norm_desc &d, Tensors *all)
{
    for (const bsa_norm *n : {&d.post, &d.pre}) {
        all->reads(n->weight, int64_t(4) * d.C);
        all->reads(n->bias, int64_t(4) * d.C);
    }
    for (const bsa_modulation *m : {&d.gate, &d.scale, &d.shift})
        if (m->ptr) modulation_of(*m, d, &all->in[all->n_in++]);
}

}  // namespace

extern "C" {

bsa_status bsa_rotary_plan_init(const bsa_rotary_spec *spec, int d, bsa_rotary_plan *plan)
{
    if (!spec || !plan) return BSA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return BSA_ERR_SHAPE;
    if (spec->n_axes < 1 || spec->n_axes > BSA_ROTARY_MAX_AXES) return BSA_ERR_INVALID_ARG;
    if (spec->pairing != BSA_ROTARY_INTERLEAVED && spec->pairing != BSA_ROTARY_HALVES) return BSA_ERR_INVALID_ARG;
    int rot = 0;
    for (int a = 0; a < spec->n_axes; ++a) {
        const int dim = spec->axis_dim[a];
        if (dim < 2 || dim % 2 != 0 || dim > d - rot) return BSA_ERR_INVALID_ARG;
        rot += dim;
        if (!spec->inv_freq &&
            !(std::isfinite(spec->theta[a]) && spec->theta[a] > 0.0 && std::isfinite(spec->scale[a])))
            return BSA_ERR_INVALID_ARG;
    }
    if (spec->pairing == BSA_ROTARY_HALVES && rot % 16 != 0) return BSA_ERR_INVALID_ARG;
    bsa_rotary_plan out;
    std::memset(&out, 0, sizeof(out));
    out.magic = kPlanMagic;
    out.d = d;
    out.rot = rot;
    out.n_axes = spec->n_axes;
    out.pairing = spec->pairing;
    int p = 0;
    for (int a = 0; a < spec->n_axes; ++a) {
        for (int j = 0; j < spec->axis_dim[a] / 2; ++j, ++p) {
            double f = 0.0, rest = 0.0;  // their sum
            if (spec->inv_freq)
                f = spec->inv_freq[p];
            else
                frequency(spec->scale[a], spec->theta[a], j, spec->axis_dim[a], &f, &rest);
            if (!std::isfinite(f)) return BSA_ERR_INVALID_ARG;
            out.turns[p] = turns_of(f, rest);
            out.axis[p] = static_cast<uint8_t>(a);
        }
    }
    *plan = out;
    return BSA_OK;
}

bsa_status bsa_rotary(const bsa_rotary_plan *plan, const bsa_heads *q, const bsa_heads *k, const bsa_heads *v, int dt,
                      int B, int N, const int32_t *positions, int64_t pos_batch, int norm, float eps, void *stream)
{
    bsa_status s = check_rotary(plan, dt, B, N, positions, pos_batch, q || k, norm, eps);
    if (s != BSA_OK) return s;
    if (!q && !k && !v) return BSA_ERR_INVALID_ARG;
    const bsa_heads *t[3] = {q, k, v};
    bsa::RotaryArgs a{};
    Tensors all;
    const int e = size_of(dt), d = plan->d;
    for (int i = 0; i < 3; ++i) {
        if (!t[i]) continue;
        s = check_heads(t[i]->heads);
        if (s != BSA_OK) return s;
        bsa::HeadsView &h = a.t[i];
        const int heads = t[i]->heads;
        Footprint &in = all.in[all.n_in], &out = all.out[all.n_out];
        if (!make_footprint(t[i]->src, B, t[i]->src_batch, N, t[i]->src_token, heads, t[i]->src_head, d, e, &in) ||
            !make_footprint(t[i]->dst, B, t[i]->dst_batch, N, t[i]->dst_token, heads, t[i]->dst_head, d, e, &out))
            return BSA_ERR_INVALID_ARG;
        all.may_be[all.n_out++] = 1u << all.n_in++;
        h.src = static_cast<const char *>(t[i]->src);
        h.src_b = in.stride[0] / e, h.src_n = in.stride[1] / e, h.src_h = in.stride[2] / e;
        h.dst = static_cast<char *>(t[i]->dst);
        h.dst_b = out.stride[0] / e, h.dst_n = out.stride[1] / e, h.dst_h = out.stride[2] / e;
        if (norm && i < 2) {
            if (t[i]->weight && !aligned(t[i]->weight, 16)) return BSA_ERR_INVALID_ARG;
            h.weight = t[i]->weight;
            all.reads(h.weight, int64_t(4) * d);
        }
        h.heads = heads;
    }
    if (q || k) all.in[all.n_in++] = block_of(positions, int64_t(4) * N * plan->n_axes, B, 4 * pos_batch);
    if (!all.check()) return BSA_ERR_INVALID_ARG;
    a.positions = positions;
    a.pos_batch = B > 1 ? pos_batch : 0;
    a.dt = dt;
    a.B = B;
    a.N = N;
    a.norm = norm != 0;
    a.eps = eps;
    a.plan = *plan;
    return bsa::launch_rotary(a, static_cast<cudaStream_t>(stream));
}

bsa_status bsa_rotary_backward(const bsa_rotary_plan *plan, const bsa_heads_grad *q, const bsa_heads_grad *k,
                               const bsa_heads_grad *v, int dt, int B, int N, const int32_t *positions,
                               int64_t pos_batch, int norm, float eps, void *workspace, size_t workspace_bytes,
                               void *stream)
{
    bsa_status s = check_rotary(plan, dt, B, N, positions, pos_batch, q || k, norm, eps);
    if (s != BSA_OK) return s;
    if (!q && !k && !v) return BSA_ERR_INVALID_ARG;
    const bsa_heads_grad *t[3] = {q, k, v};
    bsa::RotaryArgs a{};
    Tensors all;
    bool sums = false;
    const int e = size_of(dt), d = plan->d;
    for (int i = 0; i < 3; ++i) {
        if (!t[i]) continue;
        s = check_heads(t[i]->heads);
        if (s != BSA_OK) return s;
        bsa::HeadsView &h = a.t[i];
        const int heads = t[i]->heads;
        Footprint &in = all.in[all.n_in], &out = all.out[all.n_out];
        if (!make_footprint(t[i]->dy, B, t[i]->dy_batch, N, t[i]->dy_token, heads, t[i]->dy_head, d, e, &in) ||
            !make_footprint(t[i]->dx, B, t[i]->dx_batch, N, t[i]->dx_token, heads, t[i]->dx_head, d, e, &out))
            return BSA_ERR_INVALID_ARG;
        ++all.n_in;
        unsigned may_be = 0;
        h.src = static_cast<const char *>(t[i]->dy);
        h.src_b = in.stride[0] / e, h.src_n = in.stride[1] / e, h.src_h = in.stride[2] / e;
        h.dst = static_cast<char *>(t[i]->dx);
        h.dst_b = out.stride[0] / e, h.dst_n = out.stride[1] / e, h.dst_h = out.stride[2] / e;
        if (norm && i < 2) {
            Footprint &x = all.in[all.n_in];
            if (!make_footprint(t[i]->x, B, t[i]->x_batch, N, t[i]->x_token, heads, t[i]->x_head, d, e, &x))
                return BSA_ERR_INVALID_ARG;
            may_be = 1u << all.n_in++;
            h.x = static_cast<const char *>(t[i]->x);
            h.x_b = x.stride[0] / e, h.x_n = x.stride[1] / e, h.x_h = x.stride[2] / e;
            if ((t[i]->weight && !aligned(t[i]->weight, 16)) || (t[i]->dweight && !aligned(t[i]->dweight, 4)))
                return BSA_ERR_INVALID_ARG;
            h.weight = t[i]->weight;
            h.dweight = t[i]->dweight;
            all.reads(h.weight, int64_t(4) * d);
            sums = sums || h.dweight;
        } else if (t[i]->dweight) {
            return BSA_ERR_INVALID_ARG;  // no norm, no weight
        }
        all.may_be[all.n_out++] = may_be;
        all.writes(h.dweight, int64_t(4) * d);
        h.heads = heads;
    }
    if (q || k) all.in[all.n_in++] = block_of(positions, int64_t(4) * N * plan->n_axes, B, 4 * pos_batch);
    if (sums) {
        size_t need = 0;
        s = bsa_rotary_workspace_size(B, N, d, &need);
        if (s != BSA_OK) return s;
        if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return BSA_ERR_WORKSPACE;
        a.partial = static_cast<float *>(workspace);
        all.writes(workspace, static_cast<int64_t>(need));
    }
    if (!all.check()) return BSA_ERR_INVALID_ARG;
    a.positions = positions;
    a.pos_batch = B > 1 ? pos_batch : 0;
    a.dt = dt;
    a.B = B;
    a.N = N;
    a.norm = norm != 0;
    a.eps = eps;
    a.plan = *plan;
    return bsa::launch_rotary_backward(a, static_cast<cudaStream_t>(stream));
}

bsa_status bsa_rotary_workspace_size(int B, int N, int d, size_t *bytes)
{
    if (!bytes) return BSA_ERR_INVALID_ARG;
    if (B < 1 || N < 1 || static_cast<int64_t>(B) * N > INT32_MAX || (d != 64 && d != 128)) return BSA_ERR_SHAPE;
    *bytes = sizeof(float) * bsa::kRotaryMaxCtas * 2 * static_cast<size_t>(d);
    return BSA_OK;
}

bsa_status bsa_gated_norm(const bsa_gated_norm_desc *desc, const bsa_rows *x, const bsa_rows *y, const bsa_rows *h,
                          const bsa_rows *z, void *stream)
{
    const bsa_status s = check_desc(desc);
    if (s != BSA_OK) return s;
    const bsa_gated_norm_desc &d = *desc;
    const bool branch = y && y->ptr, pre = d.pre.kind != BSA_NORM_NONE;
    if (!x || (!branch && !pre)) return BSA_ERR_INVALID_ARG;
    if (branch != (h && h->ptr) || pre != (z && z->ptr)) return BSA_ERR_INVALID_ARG;
    if (!branch && (d.gate.ptr || d.post.kind != BSA_NORM_NONE)) return BSA_ERR_INVALID_ARG;
    bsa::NormArgs a{};
    a.d = tidy(d);
    Tensors all;
    if (!rows_of(*x, d, d.stream_dt, &all.in[0], &a.x)) return BSA_ERR_INVALID_ARG;
    all.n_in = 1;
    if (branch) {
        if (!rows_of(*y, d, d.branch_dt, &all.in[1], &a.y)) return BSA_ERR_INVALID_ARG;
        all.n_in = 2;
        if (!rows_of(*h, d, d.stream_dt, &all.out[all.n_out], &a.h)) return BSA_ERR_INVALID_ARG;
        all.may_be[all.n_out++] = 1u;
    }
    if (pre) {
        if (!rows_of(*z, d, d.branch_dt, &all.out[all.n_out], &a.z)) return BSA_ERR_INVALID_ARG;
        all.may_be[all.n_out++] = 2u;
    }
    reads_parameters(a.d, &all);
    if (!all.check()) return BSA_ERR_INVALID_ARG;
    return bsa::launch_gated_norm(a, static_cast<cudaStream_t>(stream));
}

bsa_status bsa_gated_norm_backward(const bsa_gated_norm_desc *desc, const bsa_gated_norm_grads *grads, void *workspace,
                                   size_t workspace_bytes, void *stream)
{
    bsa_status s = check_desc(desc);
    if (s != BSA_OK) return s;
    if (!grads) return BSA_ERR_INVALID_ARG;
    const bsa_gated_norm_desc &d = *desc;
    const bsa_gated_norm_grads &g = *grads;
    const bool pre = d.pre.kind != BSA_NORM_NONE, post_sums = g.dgate || g.dpost_weight || g.dpost_bias,
               pre_sums = g.dscale || g.dshift || g.dpre_weight || g.dpre_bias;
    if (pre != (g.dz.ptr != nullptr) || (pre && !g.h.ptr) || (!pre && !g.dh.ptr)) return BSA_ERR_INVALID_ARG;
    if (!g.dx.ptr && !g.dy.ptr && !post_sums && !pre_sums) return BSA_ERR_INVALID_ARG;
    if ((g.dy.ptr || post_sums) && !g.y.ptr) return BSA_ERR_INVALID_ARG;
    if (pre_sums && !pre) return BSA_ERR_INVALID_ARG;
    if ((g.dpost_weight || g.dpost_bias) && d.post.kind == BSA_NORM_NONE) return BSA_ERR_INVALID_ARG;
    if ((g.dgate && (!d.gate.ptr || broadcast(d.gate, d))) || (g.dscale && (!d.scale.ptr || broadcast(d.scale, d))) ||
        (g.dshift && (!d.shift.ptr || broadcast(d.shift, d))))
        return BSA_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(g.dgate), static_cast<const void *>(g.dscale),
                          static_cast<const void *>(g.dshift), static_cast<const void *>(g.dpost_weight),
                          static_cast<const void *>(g.dpost_bias), static_cast<const void *>(g.dpre_weight),
                          static_cast<const void *>(g.dpre_bias)})
        if (p && !aligned(p, 16)) return BSA_ERR_INVALID_ARG;

    bsa::NormArgs a{};
    a.d = tidy(d);
    Tensors all;
    unsigned dh_bit = 0, dz_bit = 0, h_bit = 0, y_bit = 0;
    auto input = [&](const bsa_rows &r, int dt, bsa::RowsView *v, unsigned *bit) {
        if (!rows_of(r, d, dt, &all.in[all.n_in], v)) return false;
        *bit = 1u << all.n_in++;
        return true;
    };
    if (g.dh.ptr && !input(g.dh, d.stream_dt, &a.dh, &dh_bit)) return BSA_ERR_INVALID_ARG;
    if (pre && (!input(g.dz, d.branch_dt, &a.dz, &dz_bit) || !input(g.h, d.stream_dt, &a.h, &h_bit)))
        return BSA_ERR_INVALID_ARG;
    if ((g.dy.ptr || post_sums) && !input(g.y, d.branch_dt, &a.y, &y_bit)) return BSA_ERR_INVALID_ARG;
    if (g.dx.ptr) {
        if (!rows_of(g.dx, d, d.stream_dt, &all.out[all.n_out], &a.dx)) return BSA_ERR_INVALID_ARG;
        all.may_be[all.n_out++] = dh_bit | h_bit;
    }
    if (g.dy.ptr) {
        if (!rows_of(g.dy, d, d.branch_dt, &all.out[all.n_out], &a.dy)) return BSA_ERR_INVALID_ARG;
        all.may_be[all.n_out++] = y_bit | dz_bit;
    }
    if (!a.y.p) a.d.post = bsa_norm{};  // nothing is asked for behind the post norm
    reads_parameters(a.d, &all);
    for (const void *p : {g.dgate, g.dscale, g.dshift}) all.writes(p, int64_t(d.B) * d.F * d.C * size_of(d.mod_dt));
    for (const float *p : {g.dpost_weight, g.dpost_bias, g.dpre_weight, g.dpre_bias}) all.writes(p, int64_t(4) * d.C);
    a.dgate = static_cast<char *>(g.dgate);
    a.dscale = static_cast<char *>(g.dscale);
    a.dshift = static_cast<char *>(g.dshift);
    a.dpost_w = g.dpost_weight;
    a.dpost_b = g.dpost_bias;
    a.dpre_w = g.dpre_weight;
    a.dpre_b = g.dpre_bias;
    if (pre_sums || post_sums) {
        size_t need = 0;
        s = bsa_gated_norm_workspace_size(d.B, d.N, d.C, &need);
        if (s != BSA_OK) return s;
        if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return BSA_ERR_WORKSPACE;
        a.partial = static_cast<float *>(workspace);
        all.writes(workspace, static_cast<int64_t>(need));
    }
    if (!all.check()) return BSA_ERR_INVALID_ARG;
    return bsa::launch_gated_norm_backward(a, static_cast<cudaStream_t>(stream));
}

bsa_status bsa_gated_norm_workspace_size(int B, int N, int C, size_t *bytes)
{
    if (!bytes) return BSA_ERR_INVALID_ARG;
    if (B < 1 || N < 1 || static_cast<int64_t>(B) * N > INT32_MAX || C < 8 || C > 8192 || C % 8 != 0) return BSA_ERR_SHAPE;
    const int64_t rows = static_cast<int64_t>(B) * N;
    *bytes = sizeof(float) * static_cast<size_t>(bsa::gated_norm_max_workers(rows, C)) *
             static_cast<size_t>(bsa::gated_norm_worker_floats(C));
    return BSA_OK;
}

}  // extern "C"
