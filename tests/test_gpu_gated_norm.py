"""bsa_gated_norm and bsa_gated_norm_backward against their 64-bit forms."""
import pytest
import torch

import block_sparse_attention_mean_gb300 as pkg
from block_sparse_attention_mean_gb300 import binding as bb
from block_sparse_attention_mean_gb300 import block_binding as ob
from block_sparse_attention_mean_gb300 import build as bbuild
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP32 = torch.bfloat16, torch.float32
NAMES = ("dx", "dy", "dgate", "dscale", "dshift", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bbuild.build()
    ob.load()


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def draw(g, *shape, dt=FP32, scale=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale + mean).to(dt)


def make(seed, B, N, C, F=1, types=(BF16, BF16, BF16), post=None, pre=("layer", ""), gate=True, modulate=True,
         branch=True, alpha=1.0):
    """operands of a forward call: x, y, and the keyword arguments of both sides. post, pre: (kind, "wb" subset)"""
    g = gen(seed)
    stream, bdt, mdt = types

    def spec(n):
        if n is None:
            return None, None
        w = draw(g, C, scale=0.3, mean=1.0) if "w" in n[1] else None
        b = draw(g, C, scale=0.3) if "b" in n[1] else None
        return pkg.NormSpec(n[0], w, b, 1e-5), (n[0], w, b, 1e-5)

    post_spec, post_ref = spec(post)
    pre_spec, pre_ref = spec(pre)
    rows = draw(g, B, F, 3, C, dt=mdt, scale=0.5)  # strided views, as of one projection
    mods = [rows[:, :, i] if F > 1 else rows[:, 0, i] for i in range(3)]
    kw = dict(gate=mods[0] if gate and branch else None, alpha=alpha,
              scale=mods[1] if modulate and pre else None, shift=mods[2] if modulate and pre else None)
    x = draw(g, B, N, C, scale=2.0, mean=0.5)
    x[..., ::37] *= 10.0
    y = draw(g, B, N, C, dt=bdt) if branch else None
    return x.to(stream), y, dict(kw, post=post_spec, pre=pre_spec), dict(kw, post=post_ref, pre=pre_ref)


def check_forward(x, y, kw, rkw):
    h, z = pkg.gated_norm(x, y, **kw)
    (rh, dh), (rz, dz) = ref.gated_norm(x, y, **rkw)
    if y is not None:
        ref.within(h, rh, dh, "h")
    else:
        assert h is None
    if kw["pre"] is not None:
        ref.within(z, rz, dz, "z")
    else:
        assert z is None
    return h, z


def check_backward(h, y, kw, rkw, dh, dz):
    got = pkg.gated_norm_backward(dh, dz, h, y, **kw)
    want = ref.gated_norm_backward(dh, dz, h, y, **rkw)
    if kw["pre"] is None:
        assert got.dx is dh
    for name in NAMES:
        value = getattr(got, name)
        if name in want:
            ref.within(value.view(want[name][0].shape) if name in NAMES[2:5] else value, *want[name], name)
        else:
            assert value is None or name == "dx", name
    return got


def assert_same(got, expected):
    for a, b in zip(got, expected):
        assert (a is None) == (b is None)
        assert a is None or torch.equal(a, b)


def both(seed, B, N, C, types=(BF16, BF16, BF16), arriving=True, **more):
    x, y, kw, rkw = make(seed, B, N, C, types=types, **more)
    h, z = check_forward(x, y, kw, rkw)
    g = gen(seed + 1)
    dz = draw(g, B, N, C, dt=types[1]) if kw["pre"] is not None else None
    dh = draw(g, B, N, C, dt=types[0]) if arriving or dz is None else None
    check_backward(h if y is not None else x, y, kw, rkw, dh, dz)


TYPES = [(BF16, BF16, BF16), (FP32, BF16, FP32), (FP32, FP32, BF16), (BF16, BF16, FP32)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [8, 24, 64, 72, 256, 264, 504, 520, 1000, 1032, 2048, 3080, 4096, 4104, 6152, 8192])
def test_widths_and_types(C, types):
    both(C, 2, 37, C, types=types, post=("rms", "w"), pre=("layer", "wb"))


@pytest.mark.parametrize("post", [None, ("rms", ""), ("rms", "wb"), ("layer", "w"), ("layer", "wb")])
@pytest.mark.parametrize("pre", [None, ("rms", "w"), ("layer", ""), ("layer", "wb")])
@pytest.mark.parametrize("gate,modulate", [(True, True), (False, True), (True, False), (False, False)])
def test_kinds(post, pre, gate, modulate):
    both(11, 2, 19, 136, post=post, pre=pre, gate=gate, modulate=modulate, alpha=0.7)


@pytest.mark.parametrize("pre", [("rms", "w"), ("layer", ""), ("layer", "b")])
@pytest.mark.parametrize("types", TYPES[:3])
def test_first_norm_without_a_branch(pre, types):
    both(13, 3, 21, 520, types=types, pre=pre, branch=False)
    both(14, 1, 5, 520, types=types, pre=pre, branch=False, arriving=False, modulate=False)


@pytest.mark.parametrize("B,N,F", [(1, 1, 1), (5, 1, 1), (1, 2, 2), (2, 6, 3), (3, 64, 64), (1, 1000, 1), (2, 700, 7),
                                   (1, 999, 333), (4, 500, 2)])
@pytest.mark.parametrize("C", [16, 48, 400, 800, 1160])
def test_groups(B, N, F, C):
    """groups shorter than, as long as and longer than a worker's rows, one row each among them"""
    both(B + N + F, B, N, C, F=F, types=(FP32, FP32, FP32), post=("layer", "wb"), pre=("rms", "wb"))


@pytest.mark.parametrize("N,F,C", [(9000, 1, 1024), (9000, 9000, 1024), (9000, 18, 1024), (6000, 2000, 2048),
                                   (20000, 10, 64), (20000, 20000, 16), (30011, 1, 136), (7000, 1000, 264),
                                   (9001, 1, 920), (6006, 858, 700 * 8), (40000, 20000, 40)])
def test_many_rows(N, F, C):
    """several rows per worker: groups that lie within, cross and span the workers' ranges"""
    both(N + F, 1, N, C, F=F, post=("rms", "w"), pre=("layer", "wb"))


def test_long_column_sums():
    # of the training shapes: the longest chain of a column sum is a worker's rows, below 128
    both(5, 1, 16384, 2048, F=16, post=("rms", "w"), pre=("rms", "w"))


def test_in_place():
    for types in ((BF16, BF16, BF16), (FP32, BF16, FP32)):
        x, y, kw, _ = make(21, 2, 77, 1032, types=types, post=("layer", "wb"), pre=("rms", "w"))
        h, z = pkg.gated_norm(x, y, **kw)
        x2, y2 = x.clone(), y.clone()
        pkg.gated_norm(x2, y2, **kw, out=(x2, y2))
        assert torch.equal(x2, h) and torch.equal(y2, z)
        g = gen(22)
        dh, dz = draw(g, 2, 77, 1032, dt=types[0]), draw(g, 2, 77, 1032, dt=types[1])
        plain = pkg.gated_norm_backward(dh, dz, h, y, **kw)
        for dx_over, dy_over in (("dh", "dz"), ("h", "y")):
            t = dict(dh=dh.clone(), dz=dz.clone(), h=h.clone(), y=y.clone())
            got = pkg.gated_norm_backward(t["dh"], t["dz"], t["h"], t["y"], **kw, out=(t[dx_over], t[dy_over]))
            assert_same(got, plain)


def test_slices_of_larger_buffers():
    """text and image tokens of a joint sequence, channels of a wider buffer: the rest stays as it was"""
    B, N, C = 2, 23, 264
    x, y, kw, rkw = make(31, B, N, C, post=("rms", "w"), pre=("layer", ""))
    h, z = pkg.gated_norm(x, y, **kw)
    room = torch.full((4, B, N + 9, C + 16), 3.0, dtype=BF16, device=DEV)
    xs, ys, hs, zs = (r[:, 4:4 + N, 8:8 + C] for r in room)
    xs.copy_(x)
    ys.copy_(y)
    pkg.gated_norm(xs, ys, **kw, out=(hs, zs))
    assert torch.equal(hs, h) and torch.equal(zs, z)
    dh, dz = draw(gen(32), B, N, C, dt=BF16), draw(gen(33), B, N, C, dt=BF16)
    plain = pkg.gated_norm_backward(dh, dz, h, y, **kw)
    got = pkg.gated_norm_backward(dh, dz, hs, ys, **kw, out=(xs, zs))
    assert_same(got, plain)
    for t in (xs, ys, hs, zs):
        t.fill_(3.0)
    assert room.eq(3.0).all()
    # two halves of one buffer, the second the first's output
    pair = torch.stack((x, x), 2)
    pkg.gated_norm(pair[:, :, 0], y, **kw, out=(pair[:, :, 1], None))
    assert torch.equal(pair[:, :, 1], h) and torch.equal(pair[:, :, 0], x)


@pytest.mark.parametrize("C", [8, 24, 72, 136, 264, 520, 1032, 2056, 4104, 5600, 8184])
def test_nothing_past_the_channels_is_read(C):
    """rows, modulations and weights with NaN right behind their channels: none of it reaches a result"""
    B, N, F = 2, 45, 3

    def fenced(t):
        room = torch.full((*t.shape[:-1], C + 512), float("nan"), dtype=t.dtype, device=DEV)
        room[..., :C] = t
        return room[..., :C]

    for types in TYPES[:3]:
        x, y, kw, rkw = make(C, B, N, C, F=F, types=types, post=("layer", "wb"), pre=("layer", "wb"))
        for n in ("gate", "scale", "shift"):
            kw[n] = rkw[n] = fenced(kw[n])
        for n in ("post", "pre"):
            kind, w, b, eps = rkw[n]
            w, b = fenced(w), fenced(b)
            kw[n], rkw[n] = pkg.NormSpec(kind, w, b, eps), (kind, w, b, eps)
        x, y = fenced(x), fenced(y)
        h, _ = check_forward(x, y, kw, rkw)
        dh, dz = fenced(draw(gen(1), B, N, C, dt=types[0])), fenced(draw(gen(2), B, N, C, dt=types[1]))
        check_backward(fenced(h), y, kw, rkw, dh, dz)


def test_broadcast_inputs():
    x, y, kw, rkw = make(41, 3, 10, 96, F=2)
    one = dict(kw, gate=kw["gate"][:1].expand(3, 2, 96), scale=kw["scale"][:, :1].expand(3, 2, 96))
    check_forward(x[:1].expand(3, 10, 96), y, one, dict(rkw, gate=one["gate"], scale=one["scale"]))
    for name in ("gate", "scale"):  # their gradients would have to be summed: the caller's to do
        with pytest.raises(bb.BsaError) as e:
            pkg.gated_norm_backward(x, y, x, y, **dict(kw, **{name: one[name]}))
        assert e.value.code == bb.ERR_INVALID_ARG


def test_rows_far_from_zero_and_constant():
    C = 768
    x, y, kw, rkw = make(51, 1, 12, C, types=(FP32, FP32, FP32), branch=False)
    x[0, 0] = 1000.0 + draw(gen(54), C)                  # mean 1000 times the spread
    x[0, 1] = 5.0                                        # no spread: z is the shift
    x[0, 2] = 0.0
    x[0, 3] = 1e-20
    check_forward(x, None, kw, rkw)
    check_backward(x, None, kw, rkw, draw(gen(52), 1, 12, C), draw(gen(53), 1, 12, C))
    _, z = pkg.gated_norm(x, None, pre=pkg.NormSpec("layer", eps=0.0))  # 0 / 0 where there is no spread
    assert not torch.isfinite(z[0, 2]).any() and torch.isfinite(z[0, 4:]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_finite_stay_alone(bad):
    for C in (16, 1024):
        x, y, kw, rkw = make(61, 1, 9, C, post=("rms", ""), pre=("layer", ""))
        h, z = pkg.gated_norm(x, y, **kw)
        x2 = x.clone()
        x2[0, 4, 3] = bad
        h2, z2 = pkg.gated_norm(x2, y, **kw)
        keep = [0, 1, 2, 3, 5, 6, 7, 8]
        assert torch.equal(h2[0, keep], h[0, keep]) and torch.equal(z2[0, keep], z[0, keep])
        assert not torch.isfinite(z2[0, 4]).any()
        assert torch.isfinite(h2[0, 4]).sum() == C - 1
        dh, dz = draw(gen(62), 1, 9, C, dt=BF16), draw(gen(63), 1, 9, C, dt=BF16)
        a = pkg.gated_norm_backward(dh, dz, h, y, **kw)
        h3 = h.clone()
        h3[0, 4, 3] = bad
        b = pkg.gated_norm_backward(dh, dz, h3, y, **kw)
        assert torch.equal(a.dx[0, keep], b.dx[0, keep]) and torch.equal(a.dy[0, keep], b.dy[0, keep])


def test_offsets_past_32_bits():
    stride, C = (1 << 31) + 64, 64
    big = torch.empty(2 * stride + 1024, dtype=BF16, device=DEV)
    far = big.as_strided((1, 3, C), (0, stride, 1))
    x, y, kw, _ = make(71, 1, 3, C)
    h, z = pkg.gated_norm(x, y, **kw)
    far.copy_(x)
    _, z2 = pkg.gated_norm(far, y, **kw, out=(far, None))
    assert torch.equal(far, h) and torch.equal(z2, z)
    dh, dz = draw(gen(72), 1, 3, C, dt=BF16), draw(gen(73), 1, 3, C, dt=BF16)
    a = pkg.gated_norm_backward(dh, dz, h, y, **kw)
    assert_same(pkg.gated_norm_backward(dh, dz, far, y, **kw, out=(far, None)), a)


def test_same_bits_again_and_on_another_stream():
    x, y, kw, _ = make(81, 2, 3000, 512, F=5, post=("rms", "w"), pre=("layer", "wb"))
    dh, dz = draw(gen(82), 2, 3000, 512, dt=BF16), draw(gen(83), 2, 3000, 512, dt=BF16)
    h, z = pkg.gated_norm(x, y, **kw)
    first = pkg.gated_norm_backward(dh, dz, h, y, **kw)
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        ws = pkg.gated_norm_workspace(2, 3000, 512).fill_(255)  # what the workspace held does not matter
        out = torch.zeros_like(h), torch.zeros_like(z), torch.zeros_like(h), torch.zeros_like(y)
        torch.cuda.synchronize()
        pkg.gated_norm(x, y, **kw, out=out[:2], stream=stream)
        got = pkg.gated_norm_backward(dh, dz, h, y, **kw, out=out[2:], ws=ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out[0], h) and torch.equal(out[1], z)
        assert_same(got, first)


def test_captured_and_replayed():
    x, y, kw, _ = make(91, 1, 600, 1024, F=3, post=("rms", "w"), pre=("rms", "w"))
    dh, dz = draw(gen(92), 1, 600, 1024, dt=BF16), draw(gen(93), 1, 600, 1024, dt=BF16)
    h, z = pkg.gated_norm(x, y, **kw)
    ws = pkg.gated_norm_workspace(1, 600, 1024)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.gated_norm(x, y, **kw, out=(h, z))
        got = pkg.gated_norm_backward(dh, dz, h, y, **kw, ws=ws)
    for seed in (1, 2):
        for t in (x, y, dh, dz):
            t.copy_(draw(gen(seed), *t.shape, dt=BF16))
        graph.replay()
        torch.cuda.synchronize()
        h2, z2 = pkg.gated_norm(x, y, **kw)
        assert torch.equal(h, h2) and torch.equal(z, z2)
        assert_same(got, pkg.gated_norm_backward(dh, dz, h2, y, **kw))


def test_gradients_against_differences():
    x, y, kw, rkw = make(101, 1, 4, 40, F=2, types=(FP32, FP32, FP32), post=("layer", "wb"), pre=("rms", "wb"), alpha=0.6)
    dh, dz = draw(gen(102), 1, 4, 40), draw(gen(103), 1, 4, 40)
    h = pkg.gated_norm(x, y, **kw)[0]
    got = pkg.gated_norm_backward(dh, dz, h, y, **kw)

    def loss(**changed):
        """<dh, h> + <dz, z> in 64 bits, one operand changed"""
        r = dict(rkw)
        for n in ("post", "pre"):
            spec = list(r[n])
            spec[1] = changed.get(n + "_w", spec[1].double())
            spec[2] = changed.get(n + "_b", spec[2].double())
            r[n] = tuple(spec)
        for n in ("gate", "scale", "shift"):
            r[n] = changed.get(n, r[n])
        (rh, _), (rz, _) = ref.gated_norm(changed.get("x", x), changed.get("y", y), **r)
        return (rh * dh.double()).sum() + (rz * dz.double()).sum()

    step = 1e-4
    for name, t, grad, at in (("x", x, got.dx, (0, 1, 7)), ("y", y, got.dy, (0, 3, 39)),
                              ("gate", kw["gate"], got.dgate, (0, 1, 5)), ("scale", kw["scale"], got.dscale, (0, 0, 9)),
                              ("shift", kw["shift"], got.dshift, (0, 1, 0)),
                              ("post_w", rkw["post"][1], got.dpost_weight, (3,)),
                              ("post_b", rkw["post"][2], got.dpost_bias, (4,)),
                              ("pre_w", rkw["pre"][1], got.dpre_weight, (5,)),
                              ("pre_b", rkw["pre"][2], got.dpre_bias, (6,))):
        e = torch.zeros(t.shape, dtype=torch.float64, device=DEV)
        e[at] = step
        d = (loss(**{name: t.double() + e}) - loss(**{name: t.double() - e})) / (2 * step)
        # h in the backward pass is fp32; the differences' own error is step^2 times third derivatives
        assert abs(d - grad[at].double()) <= 1e-5 * (1 + abs(d)), name


def test_some_gradients_alone():
    """through the C entry: any one of the gradients, the others' tensors not needed"""
    B, N, C = 2, 33, 128
    x, y, kw, rkw = make(111, B, N, C, post=("rms", "w"), pre=("rms", "w"))
    dh, dz = draw(gen(112), B, N, C, dt=BF16), draw(gen(113), B, N, C, dt=BF16)
    h = pkg.gated_norm(x, y, **kw)[0]
    full = pkg.gated_norm_backward(dh, dz, h, y, **kw)
    mod = lambda m: ob.Modulation(m.data_ptr(), m.stride(0), 0)  # noqa: E731
    norm = lambda n: ob.Norm(ob.NORM_RMS, n.eps, n.weight.data_ptr(), None)  # noqa: E731
    rows = lambda t: ob.Rows(t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731
    desc = ob.GatedNormDesc(B, N, C, 1, bb.BF16, bb.BF16, bb.BF16, 1.0, norm(kw["post"]), norm(kw["pre"]), mod(kw["gate"]),
                            mod(kw["scale"]), mod(kw["shift"]))
    ws = pkg.gated_norm_workspace(B, N, C)
    for name in NAMES:
        out = torch.zeros_like(getattr(full, name)) if getattr(full, name) is not None else None
        if out is None:
            continue
        g = ob.GatedNormGradArgs()
        g.dh, g.dz, g.h, g.y = (rows(t) for t in (dh, dz, h, y))
        setattr(g, name, rows(out) if name in ("dx", "dy") else out.data_ptr())
        ob.bsa_gated_norm_backward(desc, g, ws, ws.numel())
        torch.cuda.synchronize()
        assert torch.equal(out, getattr(full, name)), name


@pytest.mark.parametrize("B,F,per_group,C", [(1, 2, 900, 520), (3, 1, 900, 264), (1, 5, 900, 1032), (2, 8, 900, 40),
                                             (1, 17, 640, 264), (3, 7, 640, 1544), (1, 200, 64, 136), (8, 40, 32, 24)])
def test_groups_of_many_rows(B, F, per_group, C):
    both(131, B, F * per_group, C, F=F, post=("layer", "wb"), pre=("rms", "wb"))


@pytest.mark.parametrize("F,N", [(1, 130), (4, 2400), (20, 4000), (1000, 2000)])
def test_gradients_alone_with_biases(F, N):
    """each gradient alone is the one that comes with the others: the sums that only others need may be missing"""
    B, C = 1, 264
    x, y, kw, rkw = make(121, B, N, C, F=F, post=("layer", "wb"), pre=("rms", "wb"))
    dh, dz = draw(gen(122), B, N, C, dt=BF16), draw(gen(123), B, N, C, dt=BF16)
    h = pkg.gated_norm(x, y, **kw)[0]
    full = pkg.gated_norm_backward(dh, dz, h, y, **kw)
    mod = lambda m: ob.Modulation(m.data_ptr(), m.stride(0), m.stride(1) if F > 1 else 0)  # noqa: E731
    norm = lambda kind, n: ob.Norm(kind, n.eps, n.weight.data_ptr(), n.bias.data_ptr())  # noqa: E731
    rows = lambda t: ob.Rows(t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731
    desc = ob.GatedNormDesc(B, N, C, F, bb.BF16, bb.BF16, bb.BF16, 1.0, norm(ob.NORM_LAYER, kw["post"]),
                            norm(ob.NORM_RMS, kw["pre"]), mod(kw["gate"]), mod(kw["scale"]), mod(kw["shift"]))
    ws = pkg.gated_norm_workspace(B, N, C)
    for name in NAMES:
        out = torch.zeros_like(getattr(full, name))
        ws.fill_(0xff)  # NaN, whichever sums are not written
        g = ob.GatedNormGradArgs()
        g.dh, g.dz, g.h, g.y = (rows(t) for t in (dh, dz, h, y))
        setattr(g, name, rows(out) if name in ("dx", "dy") else out.data_ptr())
        ob.bsa_gated_norm_backward(desc, g, ws, ws.numel())
        torch.cuda.synchronize()
        assert torch.equal(out, getattr(full, name)), name


def test_helper_refusals():
    x, y, kw, _ = make(121, 2, 8, 64)

    def bad(code, fn, *args, **more):
        with pytest.raises(bb.BsaError) as e:
            fn(*args, **more)
        assert e.value.code == code

    pre = dict(pre=kw["pre"])
    bad(bb.ERR_SHAPE, pkg.gated_norm, x[0], **pre)
    bad(bb.ERR_SHAPE, pkg.gated_norm, x, y[:1], **pre)
    bad(bb.ERR_DTYPE, pkg.gated_norm, x, y.float(), **pre)     # an fp32 branch on a bf16 stream
    bad(bb.ERR_DTYPE, pkg.gated_norm, x.half(), **pre)
    bad(bb.ERR_INVALID_ARG, pkg.gated_norm, x, y.cpu(), **pre)
    bad(bb.ERR_INVALID_ARG, pkg.gated_norm, x.transpose(1, 2).contiguous().transpose(1, 2), **pre)
    bad(bb.ERR_SHAPE, pkg.gated_norm, x, y, gate=kw["gate"][:1], **pre)
    bad(bb.ERR_SHAPE, pkg.gated_norm, x, y, gate=torch.zeros(2, 3, 64, device=DEV), **pre)   # 3 frames of 8 tokens
    bad(bb.ERR_SHAPE, pkg.gated_norm, x, y, gate=torch.zeros(2, 2, 64, device=DEV), scale=torch.zeros(2, 64, device=DEV),
        **pre)
    bad(bb.ERR_DTYPE, pkg.gated_norm, x, y, gate=kw["gate"], scale=kw["scale"].float(), **pre)
    bad(bb.ERR_DTYPE, pkg.gated_norm, x, y, gate=kw["gate"].half(), **pre)
    bad(bb.ERR_SHAPE, pkg.gated_norm, x, y, pre=pkg.NormSpec("rms", torch.ones(8, device=DEV)))
    bad(bb.ERR_DTYPE, pkg.gated_norm, x, y, pre=pkg.NormSpec("rms", torch.ones(64, device=DEV, dtype=BF16)))
    bad(bb.ERR_SHAPE, pkg.gated_norm, x, y, **pre, out=(x[:1], None))
    bad(bb.ERR_INVALID_ARG, pkg.gated_norm, x)                 # nothing to do
    bad(bb.ERR_INVALID_ARG, pkg.gated_norm, x, gate=kw["gate"], **pre)
    bad(bb.ERR_INVALID_ARG, pkg.gated_norm_backward, x, None, x, y, **pre)
    bad(bb.ERR_INVALID_ARG, pkg.gated_norm_backward, x, y, None, y, **pre)
    bad(bb.ERR_SHAPE, pkg.gated_norm_backward, x, y, x[:1], y, **pre)
    small = torch.empty(256, device=DEV, dtype=torch.uint8)
    bad(bb.ERR_WORKSPACE, pkg.gated_norm_backward, x, y, x, y, **kw, ws=small)
    bad(bb.ERR_INVALID_ARG, pkg.gated_norm_backward, x, y, x, y, **kw, ws=small.cpu())


# the kernels differ by types, by width (several rows in a CTA, one row, one row of few registers), by whether there is a
# post norm and whether a layer norm is among the norms: every one of them, forward and backward
FORMS = [(None, ("layer", "")), (None, ("rms", "w")), (("rms", "w"), ("rms", "w")), (("layer", "wb"), ("rms", "")),
         (("rms", ""), None), (("layer", "w"), None), (None, None)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [136, 520, 1536, 4096, 6144])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_forms_over_widths(form, C, types):
    post, pre = FORMS[form]
    both(C + form, 2, 19, C, types=types, post=post, pre=pre, alpha=0.7)


@pytest.mark.parametrize("types", TYPES[:3])
@pytest.mark.parametrize("C", [264, 1536, 6144])
@pytest.mark.parametrize("post", [None, ("rms", "")])
def test_forms_with_many_rows(post, C, types):
    """several rows per worker, two groups, of a branch, a gate and a layer norm"""
    both(C, 1, 1402, C, F=2, types=types, post=post, pre=("layer", ""))
    both(C + 1, 1, 1402, C, F=2, types=types, post=post, pre=("rms", ""), arriving=False)


@pytest.mark.parametrize("C", [136, 1536, 6144])
@pytest.mark.parametrize("pre", [("layer", "wb"), ("rms", "w")])
def test_first_norm_of_an_fp32_stream_for_a_bf16_branch(C, pre):
    """without a branch the result's dtype is asked for, or that of the tensor that is given"""
    x, _, kw, rkw = make(141, 2, 33, C, types=(FP32, BF16, FP32), pre=pre, branch=False)
    h, z = pkg.gated_norm(x, None, **kw, branch_dtype=BF16)
    assert h is None and z.dtype == BF16
    (_, _), (rz, dz) = ref.gated_norm(x, None, **rkw)
    ref.within(z, rz, dz, "z")
    given = torch.empty_like(z)
    assert pkg.gated_norm(x, None, **kw, out=(None, given))[1] is given and torch.equal(given, z)
    plain = pkg.gated_norm(x, None, **kw)[1]
    assert plain.dtype == FP32
    ref.within(plain, rz, dz, "z")
