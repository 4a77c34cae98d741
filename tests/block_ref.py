"""Plain 64-bit forms of the operators around the attention, each with a bound on what a correct fp32
evaluation may be off by.

U = 2^-24 is the fp32 rounding unit (half a step). A bound adds, to first order, one U per rounding of a
value times that value's magnitude; sums of many terms count the longest chain of additions, CHAIN below:
a thread adds at most 16 terms of a row, a warp five levels, a CTA at most 32 warps, and rsqrtf, the division
by C and the products after it are within 8 more. Column sums count COLUMN: the rows that one thread adds
(the tests' shapes keep them below 128), five levels, 32 slices of at most 32 partial sums, and 8 warps.
The result's own rounding to its dtype (half a step: bf16 2^-8, fp32 2^-24) is added by `within`.
"""
import torch

U = 2.0 ** -24
CHAIN = 64
COLUMN = 256
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def within(got, ref, bound, what):
    """every element of got within its rounding plus the bound of ref (equal where ref is not finite)"""
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} against {tuple(ref.shape)}"
    half = HALF_STEP[got.dtype]
    got = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{what}: infinities differ"
    allowed = half * ref.abs() + (1 + half) * bound + 1e-37
    over = ((got - ref).abs() / allowed)[fine]
    assert over.numel() == 0 or over.max() <= 1.0, f"{what}: {over.max().item():.3g} times the bound"


# ------------------------------------------------------------------ rotary


def angles(pos, axis_dims, theta, scale=1.0):
    """[.., N, rot / 2] angles in 64 bits"""
    cols = []
    for a, dim in enumerate(axis_dims):
        j = torch.arange(dim // 2, dtype=torch.float64, device=pos.device)
        cols.append(pos[..., a:a + 1].double() * (scale * theta ** (-2.0 * j / dim)))
    return torch.cat(cols, dim=-1)


def split_pairs(x, p, interleaved):
    return (x[..., 0:2 * p:2], x[..., 1:2 * p:2]) if interleaved else (x[..., :p], x[..., p:2 * p])


def join_pairs(a, b, rest, interleaved):
    head = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((head, rest), -1)


def turned(u, du, ang, interleaved):
    """u [B, N, H, d] turned by ang [.., N, P], and the bound: per pair, products and sum (4 roundings), sincospif
    (4) and the fp32 half turns (pi of them), all on |u_a| + |u_b|."""
    ang = ang[:, :, None] if ang.dim() == 3 else ang[None, :, None]
    p = ang.shape[-1]
    c, s = ang.cos(), ang.sin()
    a, b = split_pairs(u, p, interleaved)
    da, db = split_pairs(du, p, interleaved)
    y = join_pairs(a * c - b * s, b * c + a * s, u[..., 2 * p:], interleaved)
    bound = da + db + 12 * U * (a.abs() + b.abs())
    return y, join_pairs(bound, bound, du[..., 2 * p:], interleaved)


def head_norm(x, w, eps):
    x = x.double()
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    n = x * r
    u = n * w.double() if w is not None else n
    return n, r, u


def rotary(x, ang, interleaved, norm_eps=None, w=None):
    """x [B, N, H, d] -> ([B, H, N, d], bound)"""
    u = x.double()
    du = torch.zeros_like(u)
    if norm_eps is not None:
        _, _, u = head_norm(x, w, norm_eps)
        du = CHAIN * U * u.abs()
    y, dy = turned(u, du, ang, interleaved)
    return y.transpose(1, 2), dy.transpose(1, 2)


def rotary_backward(dy, ang, interleaved, x=None, norm_eps=None, w=None):
    """dy [B, H, N, d] -> (dx, bound, dw, bound) with dx [B, N, H, d]"""
    g = dy.double().transpose(1, 2)
    g, dg = turned(g, torch.zeros_like(g), -ang, interleaved)
    if norm_eps is None:
        return g, dg, None, None
    n, r, _ = head_norm(x, w, norm_eps)
    dw = (g * n).sum((0, 1, 2))
    dw_bound = (COLUMN * U * (g * n).abs() + dg * n.abs()).sum((0, 1, 2))
    wd = w.double() if w is not None else torch.ones(x.shape[-1], dtype=torch.float64, device=x.device)
    v, dv = g * wd, dg * wd.abs()
    m, mabs = (v * n).mean(-1, keepdim=True), (v * n).abs().mean(-1, keepdim=True)
    dx = r * (v - n * m)
    bound = r * (dv + n.abs() * (dv * n.abs()).mean(-1, keepdim=True) + 2 * CHAIN * U * (v.abs() + n.abs() * mabs))
    return dx, bound, dw, dw_bound


# ------------------------------------------------------------------ gated norm


def norm(t, dt, kind, eps):
    """(n, r, bound of n, relative bound of r) of the rows of t, known to dt"""
    mean = t.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(t[..., :1])
    c = t - mean
    r = (c.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    n = c * r
    dc = dt.clone()
    if kind == "layer":
        dc = dc + dt.mean(-1, keepdim=True) + CHAIN * U * t.abs().mean(-1, keepdim=True) + U * c.abs()
    dr = r * r * (c.abs() * dc).mean(-1, keepdim=True) + CHAIN * U
    return n, r, r * dc + n.abs() * dr, dr


def affine(n, dn, w, b):
    if w is not None:
        n, dn = n * w.double(), dn * w.double().abs() + U * (n * w.double()).abs()
    if b is not None:
        n, dn = n + b.double(), dn + U * (n.abs() + 2 * b.double().abs())
    return n, dn


def by_token(m, N):
    """[B, C] or [B, F, C] as [B, N, C] in 64 bits"""
    m = m.double()
    m = m[:, None] if m.dim() == 2 else m
    return m.repeat_interleave(N // m.shape[1], dim=1)


def gated_norm(x, y=None, gate=None, alpha=1.0, post=None, pre=None, scale=None, shift=None):
    """((h, bound), (z, bound)); post and pre: (kind, weight, bias, eps) or None"""
    N = x.shape[1]
    h = x.double()
    dh = torch.zeros_like(h)
    if y is not None:
        u, du = y.double(), torch.zeros_like(h)
        if post is not None:
            u, _, du, _ = norm(u, du, post[0], post[3])
            u, du = affine(u, du, post[1], post[2])
        if gate is not None:
            g = by_token(gate, N)
            u, du = u * g, du * g.abs() + U * (u * g).abs()
        h = h + alpha * u
        dh = abs(alpha) * du + 2 * U * (h.abs() + abs(alpha) * u.abs())
    z = dz = None
    if pre is not None:
        z, _, dz, _ = norm(h, dh, pre[0], pre[3])
        z, dz = affine(z, dz, pre[1], pre[2])
        if scale is not None:
            s = 1.0 + by_token(scale, N)
            z, dz = z * s, dz * s.abs() + 2 * U * (z * s).abs()
        if shift is not None:
            t = by_token(shift, N)
            z, dz = z + t, dz + U * (z.abs() + 2 * t.abs())
    return (h, dh), (z, dz)


def _sum_frames(t, F):
    B, N, C = t.shape
    return t.reshape(B, F, N // F, C).sum(2)


def _through(g, dg, n, r, dn, dr, kind):
    """gradient through a normalisation, g (known to dg) arriving at n"""
    along, aabs = (g * n).mean(-1, keepdim=True), (g * n).abs().mean(-1, keepdim=True)
    mean = g.mean(-1, keepdim=True) if kind == "layer" else 0.0 * along
    gabs = g.abs().mean(-1, keepdim=True) if kind == "layer" else 0.0 * along
    out = r * (g - mean - n * along)
    size = g.abs() + gabs + n.abs() * aabs
    bound = r * (dg + dg.mean(-1, keepdim=True) + n.abs() * (dg * n.abs() + g.abs() * dn).mean(-1, keepdim=True)
                 + dn * aabs + (2 * CHAIN * U + dr) * size)
    return out, bound


def gated_norm_backward(dh, dz, h, y=None, gate=None, alpha=1.0, post=None, pre=None, scale=None, shift=None):
    """{name: (gradient, bound)} at (h, y) as given"""
    some = dh if dh is not None else dz
    N = some.shape[1]
    out = {}
    g = dh.double() if dh is not None else torch.zeros(some.shape, dtype=torch.float64, device=some.device)
    dg = torch.zeros_like(g)

    def column(name, t, dt, F):
        total = t.sum((0, 1)) if F is None else _sum_frames(t, F)
        off = COLUMN * U * t.abs() + dt
        out[name] = (total, off.sum((0, 1)) if F is None else _sum_frames(off, F))

    def frames(m):
        return 1 if m.dim() == 2 else m.shape[1]

    if pre is not None:
        kind, w, b, eps = pre
        n, r, dn, dr = norm(h.double(), torch.zeros_like(g), kind, eps)
        a = dz.double()
        da = torch.zeros_like(a)
        if shift is not None:
            column("dshift", a, da, frames(shift))
        if scale is not None:
            m, dm = affine(n, dn, w, b)
            column("dscale", a * m, a.abs() * dm + COLUMN * U * (a * n).abs() * (w.double().abs() if w is not None else 1.0)
                   + (COLUMN * U * (a * b.double()).abs() if b is not None else 0.0), frames(scale))
            s = 1.0 + by_token(scale, N)
            a, da = a * s, 2 * U * (a * s).abs()
        if w is not None:
            column("dpre_weight", a * n, da * n.abs() + a.abs() * dn, None)
        if b is not None:
            column("dpre_bias", a, da, None)
        if w is not None:
            a, da = a * w.double(), da * w.double().abs() + U * (a * w.double()).abs()
        t, dt = _through(a, da, n, r, dn, dr, kind)
        g, dg = g + t, dt + U * (g.abs() + 2 * t.abs())
        out["dx"] = (g, dg)
    if y is not None:
        m = y.double()
        r = dr = None
        dm = torch.zeros_like(m)
        if post is not None:
            m, r, dm, dr = norm(m, dm, post[0], post[3])
        e, de = alpha * g, abs(alpha) * (dg + U * g.abs())
        if gate is not None:
            u, du = affine(m, dm, post[1], post[2]) if post is not None else (m, dm)
            w2 = post[1].double().abs() if post is not None and post[1] is not None else 1.0
            b2 = post[2].double().abs() if post is not None and post[2] is not None else 0.0
            column("dgate", e * u, e.abs() * du + de * u.abs() + COLUMN * U * e.abs() * (m.abs() * w2 + b2), frames(gate))
            t = by_token(gate, N)
            e, de = e * t, de * t.abs() + U * (e * t).abs()
        if post is not None:
            kind, w, b, eps = post
            if w is not None:
                column("dpost_weight", e * m, de * m.abs() + e.abs() * dm, None)
            if b is not None:
                column("dpost_bias", e, de, None)
            if w is not None:
                e, de = e * w.double(), de * w.double().abs() + U * (e * w.double()).abs()
            e, de = _through(e, de, m, r, dm, dr, kind)
        out["dy"] = (e, de)
    return out
