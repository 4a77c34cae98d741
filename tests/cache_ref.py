"""Plain 64-bit forms of attention over packed sequences and paged caches, each with a bound on what a correct
evaluation may be off by.

U = 2^-24. Scores: q k are products of bf16 numbers, exact in fp32, summed in fp32 in any order and with at most a
whole unit in the last place a sum (the tensor cores need not round to nearest): 2 U (d + 4) sum |q||k| scale, where
the 4 covers the scaling, the change to base 2 and the subtraction of the maximum (whose result is at most the largest
magnitude among the row's scores, counted once more by `shift`). A weight 2^x is within 2^-21 of its value. Sums of n positive terms in chains of at most
n / 4 + 64 are within that many U. Weights rounded to t bits are off by half a step each, 2^-8 for bf16 (numerator
and normaliser both), 2^-11 for fp16 (numerator only) and 2^-25 of the largest weight where fp16 has no more bits.
"""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def e4m3_rows(x):
    """(values held, exponent bytes) of rows x [..., d], by exact steps in 64 bits"""
    x = x.double()
    a = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1, keepdim=True)
    e = torch.full(a.shape, -100, dtype=torch.int64, device=x.device)
    for i in range(-100, 119):
        e += a > 448.0 * 2.0 ** i
    unit = ((e + 1023) << 52).view(torch.float64)
    y = x / unit
    step = ((torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].long() - 4 + 1023) << 52).view(torch.float64)
    y = (torch.round(y / step) * step).clamp(-448.0, 448.0)
    y = torch.where(x.isfinite(), y, float("nan"))
    return y * unit, (e[..., 0] + 127).to(torch.uint8)


def visible(n_q, n_k, causal, device):
    """bool [n_q, n_k]"""
    i, j = torch.arange(n_q, device=device)[:, None], torch.arange(n_k, device=device)
    return (j <= i + n_k - n_q) if causal else (j < n_k).expand(n_q, n_k)


def attention(q, k, v, see, scale, half_weights=False):
    """q [n_q, d], k, v [n_k, d] (values), see bool [n_q, n_k]: (O, bound of O before its rounding, LSE, bound)"""
    q, k, v = q.double(), k.double(), v.double()
    d, n = q.shape[1], k.shape[0]
    if n == 0 or q.shape[0] == 0:
        o = torch.zeros_like(q)
        return o, o, torch.full_like(o[:, 0], float("-inf")), torch.zeros_like(o[:, 0])
    s = (q @ k.T) * scale
    ds = 2 * U * (d + 4) * (q.abs() @ k.abs().T) * scale
    if half_weights:  # q in fp16, relative to its row's largest: below 2^-14 of it in steps of 2^-24
        ds = ds + 2.0 ** -24 * q.abs().amax(-1, keepdim=True) * k.abs().sum(-1) * scale
    s = torch.where(see, s, float("-inf"))
    ds = torch.where(see, ds, 0.0)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    shift = 4 * U * torch.where(see, s.abs(), 0.0).amax(-1, keepdim=True)
    p = torch.where(see, torch.exp(s - m), 0.0)
    total = p.sum(-1, keepdim=True)
    w = p / torch.where(total > 0, total, 1.0)
    vz = torch.where(v.isfinite(), v, 0.0)
    o = w @ vz
    bad = ~v.isfinite()
    if bad.any():  # what is not finite reaches exactly the rows that see it
        for j in bad.any(-1).nonzero()[:, 0].tolist():
            rows = see[:, j]
            o[rows] = torch.where(bad[j], o[rows] + v[j], o[rows])
    chain = (n / 4 + 64) * U
    off = (ds.amax(-1, keepdim=True) + shift) + 2.0 ** -21 + chain
    half = 2.0 ** -11 if half_weights else 2.0 ** -8
    size = w @ vz.abs()
    bound = (2 * off + (1 if half_weights else 2) * half * (1 + 2.0 ** -7)) * size
    if half_weights:
        # fp16 of a weight times its value's unit, relative to the largest such product: steps of 2^-24, the maximum
        # within 2^8 of the largest (the running one) and the data at most 448
        unit = vz.abs().amax(-1)
        bound = bound + 2.0 ** -24 * 2 * n * (w * unit).amax(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    return o, bound, lse, (off + 4 * U * lse.abs().clamp(max=1e30)[:, None]).squeeze(-1)


def within(got, ref, bound, what):
    """every element of got within its rounding plus the bound of ref (equal where ref is not finite)"""
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} against {tuple(ref.shape)}"
    half = HALF_STEP[got.dtype]
    got = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{what}: infinities differ"
    over = ((got - ref).abs() / (half * ref.abs() + (1 + half) * bound + 1e-37))[fine]
    assert over.numel() == 0 or over.max() <= 1.0, f"{what}: {over.max().item():.3g} times the bound"
