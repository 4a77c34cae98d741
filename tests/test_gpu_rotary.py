"""bsa_rotary and bsa_rotary_backward against their 64-bit forms."""
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


def fused(g, B, N, H, Hk, d, dt):
    return draw(g, B, N, H + 2 * Hk, d, dt=dt).split([H, Hk, Hk], dim=2)


def check_forward(q, k, v, out, ang, interleaved, eps, wq, wk):
    for x, o, w, name in ((q, out[0], wq, "q"), (k, out[1], wk, "k")):
        if x is not None:
            ref.within(o, *ref.rotary(x, ang, interleaved, eps, w), name)
    if v is not None:
        assert torch.equal(out[2], v.transpose(1, 2))


def check_backward(grads, q, k, got, ang, interleaved, eps, wq, wk):
    for dy, x, dx, w, dw, name in ((grads[0], q, got[0], wq, got[3], "q"), (grads[1], k, got[1], wk, got[4], "k")):
        if dy is None:
            continue
        rdx, bound, rdw, dw_bound = ref.rotary_backward(dy, ang, interleaved, x, eps, w)
        ref.within(dx, rdx, bound, "d" + name)
        if w is not None:
            ref.within(dw, rdw, dw_bound, name + " weight")
        else:
            assert dw is None
    if grads[2] is not None:
        assert torch.equal(got[2], grads[2].transpose(1, 2))


CASES = [
    # dt, B, N, H, Hk, d, axes, interleaved, eps, weights
    (FP32, 1, 1, 1, 1, 64, (64,), True, None, False),
    (BF16, 1, 1, 3, 1, 128, (16, 56, 56), False, 1e-6, True),
    (BF16, 2, 33, 5, 5, 64, (32, 32), True, 1e-6, True),
    (FP32, 3, 31, 4, 2, 128, (44, 42, 42), True, 1e-5, True),
    (FP32, 2, 65, 7, 7, 64, (10, 20, 18), False, 1e-6, False),
    (BF16, 1, 257, 24, 24, 128, (44, 42, 42), True, 1e-6, True),
    (BF16, 2, 100, 8, 2, 128, (6, 4), True, 1e-6, True),          # most channels do not turn
    (FP32, 1, 129, 9, 3, 128, (2, 2, 2, 10), False, None, False),
    (BF16, 1, 64, 2, 2, 64, (62,), True, None, False),            # the last pair does not turn
    (BF16, 1, 300, 17, 17, 64, (16, 24, 24), False, 0.0, True),
    (BF16, 1, 12, 64, 8, 128, (128,), False, 1e-6, True),
    (FP32, 2, 70, 48, 24, 64, (16, 16), False, 1e-6, True),       # halves, half of the channels turn, heads by fours
    (FP32, 1, 41, 32, 8, 128, (32, 16, 48), False, 1e-6, True),
    (BF16, 2, 39, 26, 26, 64, (20, 6, 4), True, 1e-6, True),      # heads by twos
    (FP32, 1, 1000, 24, 24, 128, (44, 42, 42), True, 1e-6, True),  # many tiles per CTA
    (BF16, 3, 2000, 1, 1, 64, (16, 24, 24), True, 1e-6, True),
]


@pytest.mark.parametrize("dt,B,N,H,Hk,d,axes,interleaved,eps,weights", CASES)
def test_rotary_and_backward(dt, B, N, H, Hk, d, axes, interleaved, eps, weights):
    g = gen(N * 7 + H)
    q, k, v = fused(g, B, N, H, Hk, d, dt)
    pos = torch.randint(-50, 4000, (N, len(axes)), generator=g, device=DEV, dtype=torch.int32)
    wq, wk = (draw(g, d, scale=0.3, mean=1.0), draw(g, d, scale=0.3, mean=1.0)) if weights else (None, None)
    plan = pkg.rotary_plan(d, axes, interleaved=interleaved)
    ang = ref.angles(pos, axes, 10000.0)
    out = pkg.rotary(plan, q, k, v, positions=pos, norm_eps=eps, q_weight=wq, k_weight=wk)
    assert all(o.is_contiguous() and o.shape[1] == h for o, h in zip(out, (H, Hk, Hk)))
    check_forward(q, k, v, out, ang, interleaved, eps, wq, wk)
    grads = [draw(g, *o.shape, dt=dt) for o in out]
    got = pkg.rotary_backward(plan, *grads, positions=pos, q=q, k=k, norm_eps=eps, q_weight=wq, k_weight=wk)
    check_backward(grads, q, k, got, ang, interleaved, eps, wq if eps is not None else None,
                   wk if eps is not None else None)


def test_weights_of_one_side_and_parts_alone():
    g = gen(3)
    q, k, v = fused(g, 2, 50, 4, 4, 64, BF16)
    pos = pkg.grid_positions((2, 5, 5))
    plan = pkg.rotary_plan(64, (16, 24, 24))
    ang = ref.angles(pos, (16, 24, 24), 10000.0)
    w = draw(g, 64, mean=1.0)
    for args in ((q, None, None), (None, k, None), (None, None, v), (q, None, v), (q, k, None)):
        out = pkg.rotary(plan, *args, positions=pos, norm_eps=1e-6, k_weight=w)
        assert [o is None for o in out] == [x is None for x in args]
        check_forward(*args, out, ang, True, 1e-6, None, w)
        grads = [None if o is None else draw(g, *o.shape, dt=BF16) for o in out]
        got = pkg.rotary_backward(plan, *grads, positions=pos, q=q, k=k, norm_eps=1e-6, k_weight=w)
        check_backward(grads, q, k, got, ang, True, 1e-6, None, w)
    out = pkg.rotary(plan, None, None, v)  # V alone: a change of layout, no positions
    assert torch.equal(out[2], v.transpose(1, 2))


def test_positions_per_batch_and_far():
    g = gen(4)
    B, N = 3, 40
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, N, 2), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    # frequencies of 2^-k: pos * f is exact in 64 bits, so the reference is too
    freq = [2.0 ** -(3 + j % 20) for j in range(32)]
    plan = pkg.rotary_plan(64, (24, 40), inv_freq=freq)
    axis = torch.tensor([0] * 12 + [1] * 20, device=DEV)
    ang = pos.double()[..., axis] * torch.tensor(freq, dtype=torch.float64, device=DEV)
    x = draw(g, B, N, 2, 64)
    out = pkg.rotary(plan, x, positions=pos)
    y, bound = ref.rotary(x, ang, True)
    # the frequency itself is within 2^-51 of its value: up to 2^31 * 2^-3 * 2^-51 radians, below U
    ref.within(out[0], y, bound, "far positions")
    padded = torch.zeros(B, N + 5, 2, dtype=torch.int32, device=DEV)  # a batch stride of its own
    padded[:, :N] = pos
    assert torch.equal(pkg.rotary(plan, x, positions=padded[:, :N])[0], out[0])


def test_scales_and_bases_per_axis():
    g = gen(5)
    pos = pkg.grid_positions((3, 4, 5), n_text=7)
    theta, scale, axes = (100.0, 10000.0, 1e6), (2.0, 0.5, 1.0), (32, 48, 48)
    plan = pkg.rotary_plan(128, axes, theta=theta, scale=scale, interleaved=False)
    ang = torch.cat([ref.angles(pos[:, a:a + 1], (axes[a],), theta[a], scale[a]) for a in range(3)], -1)
    x = draw(g, 2, 67, 3, 128, dt=BF16)
    ref.within(pkg.rotary(plan, x, positions=pos)[0], *ref.rotary(x, ang, False), "scaled")


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("eps", [None, 1e-6])
def test_in_place(interleaved, eps):
    g = gen(6)
    B, N, H = 2, 45, 3
    qkv = draw(g, B, N, 3 * H, 128, dt=BF16)
    q, k, v = qkv.clone().split(H, dim=2)
    pos = torch.arange(N, device=DEV, dtype=torch.int32)[:, None]
    plan = pkg.rotary_plan(128, (96,), interleaved=interleaved)
    expected = pkg.rotary(plan, *qkv.split(H, dim=2), positions=pos, norm_eps=eps)
    out = [t.transpose(1, 2) for t in (q, k, v)]
    pkg.rotary(plan, q, k, v, positions=pos, norm_eps=eps, out=out)
    for o, e in zip(out, expected):
        assert torch.equal(o, e)
    # backward: the gradient of the projection over the projection
    grads = [draw(g, B, H, N, 128, dt=BF16) for _ in range(3)]
    plain = pkg.rotary_backward(plan, *grads, positions=pos, q=qkv[:, :, :H], k=qkv[:, :, H:2 * H], norm_eps=eps)
    if eps is not None:
        again = qkv.clone().split(H, dim=2)
        pkg.rotary_backward(plan, *grads, positions=pos, q=again[0], k=again[1], norm_eps=eps, out=again)
        for o, e in zip(again, plain):
            assert torch.equal(o, e)


def test_strided_outputs_leave_the_rest():
    g = gen(7)
    B, N, H, d = 2, 37, 3, 64
    x = draw(g, B, N, H, d)
    plan = pkg.rotary_plan(d, (64,))
    pos = torch.arange(N, device=DEV, dtype=torch.int32)[:, None]
    expected = pkg.rotary(plan, x, positions=pos)[0]
    room = torch.full((B, H + 1, N + 11, d + 4), 7.0, device=DEV)
    o = room[:, :H, 5:5 + N, :d]
    pkg.rotary(plan, x, positions=pos, out=(o, None, None))
    assert torch.equal(o, expected)
    room[:, :H, 5:5 + N, :d] = 7.0
    assert room.eq(7.0).all()
    # a broadcast input: one batch for both
    both = pkg.rotary(plan, x[:1].expand(B, N, H, d), positions=pos)[0]
    assert torch.equal(both[0], expected[0]) and torch.equal(both[1], expected[0])


def test_offsets_past_32_bits():
    g = gen(8)
    stride = (1 << 31) + 64
    big = torch.empty(2 * stride + 1024, dtype=BF16, device=DEV)
    x = big.as_strided((1, 3, 2, 64), (0, stride, 64, 1))
    x.copy_(draw(g, 1, 3, 2, 64, dt=BF16))
    plan = pkg.rotary_plan(64, (64,))
    pos = torch.tensor([[3], [5], [9]], device=DEV, dtype=torch.int32)
    out = pkg.rotary(plan, x, positions=pos, norm_eps=1e-6)[0]
    assert torch.equal(out, pkg.rotary(plan, x.contiguous(), positions=pos, norm_eps=1e-6)[0])
    dy = draw(g, 1, 2, 3, 64, dt=BF16)
    got = pkg.rotary_backward(plan, dy, positions=pos, q=x.contiguous(), norm_eps=1e-6)[0]
    pkg.rotary_backward(plan, dy, positions=pos, q=x, norm_eps=1e-6, out=(x, None, None))
    assert torch.equal(x, got)


def test_values_that_are_not_finite():
    g = gen(9)
    x = draw(g, 1, 8, 2, 64, dt=BF16)
    x[0, 2, 0, 40] = float("inf")   # past the turned channels: passes through
    x[0, 3, 1, 41] = float("nan")
    x[0, 5, 0, 3] = float("nan")    # a turned pair: both its channels, no others
    plan = pkg.rotary_plan(64, (32,))
    pos = torch.arange(8, device=DEV, dtype=torch.int32)[:, None]
    out = pkg.rotary(plan, x, positions=pos)[0]
    y, bound = ref.rotary(x, ref.angles(pos, (32,), 10000.0), True)
    ref.within(out, y, torch.nan_to_num(bound), "not finite")
    zero = torch.zeros_like(x)      # a head of zeros under the norm stays zero
    assert pkg.rotary(plan, zero, positions=pos, norm_eps=1e-6)[0].eq(0).all()


def test_same_bits_again_and_on_another_stream():
    g = gen(10)
    q, k, v = fused(g, 1, 1000, 6, 6, 128, BF16)
    grads = [draw(g, 1, 6, 1000, 128, dt=BF16) for _ in range(3)]
    w = draw(g, 128, mean=1.0)
    pos = torch.arange(1000, device=DEV, dtype=torch.int32)[:, None]
    plan = pkg.rotary_plan(128, (128,))
    kw = dict(positions=pos, norm_eps=1e-6, q_weight=w, k_weight=w)
    first = pkg.rotary(plan, q, k, v, **kw), pkg.rotary_backward(plan, *grads, q=q, k=k, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        ws = pkg.rotary_workspace(1, 1000, 128).fill_(255)  # what the workspace held does not matter
        out = [torch.zeros_like(o) for o in first[0]]
        dx = [torch.zeros_like(o) for o in first[1][:3]]
        torch.cuda.synchronize()
        pkg.rotary(plan, q, k, v, **kw, out=out, stream=stream)
        got = pkg.rotary_backward(plan, *grads, q=q, k=k, **kw, out=dx, ws=ws, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip((*out, *got), (*first[0], *first[1])):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    g = gen(11)
    q, k, v = fused(g, 1, 130, 4, 2, 64, BF16)
    w = draw(g, 64, mean=1.0)
    pos = torch.arange(130, device=DEV, dtype=torch.int32)[:, None]
    plan = pkg.rotary_plan(64, (64,))
    kw = dict(positions=pos, norm_eps=1e-6, q_weight=w, k_weight=w)
    out = pkg.rotary(plan, q, k, v, **kw)
    grads = [torch.empty_like(o) for o in out]
    ws = pkg.rotary_workspace(1, 130, 64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.rotary(plan, q, k, v, **kw, out=out)
        got = pkg.rotary_backward(plan, *grads, q=q, k=k, **kw, ws=ws)
    del plan  # the captured launches hold the frequencies themselves
    plan = pkg.rotary_plan(64, (64,))
    for seed in (1, 2):
        for t in (q, k, v, *grads):
            t.copy_(draw(gen(seed), *t.shape, dt=BF16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*out, *got), (*pkg.rotary(plan, q, k, v, **kw),
                                       *pkg.rotary_backward(plan, *grads, q=q, k=k, **kw))):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    g = gen(12)
    B, N, H, d = 1, 3, 2, 64
    x = draw(g, B, N, H, d)
    w = draw(g, d, scale=0.3, mean=1.0)
    pos = torch.tensor([[1, 7], [0, 3], [12, 5]], device=DEV, dtype=torch.int32)
    plan = pkg.rotary_plan(d, (24, 40), interleaved=False)
    dy = draw(g, B, H, N, d)
    got = pkg.rotary_backward(plan, dy, positions=pos, q=x, norm_eps=1e-3, q_weight=w)
    ang = ref.angles(pos, (24, 40), 10000.0)

    def loss(x, w):
        return (ref.rotary(x, ang, False, 1e-3, w)[0] * dy.double()).sum()

    # central differences in 64 bits: step h leaves h^2 of third derivatives and 2^-52 / h of rounding
    h = 1e-4
    for t, grad, at in ((x, got[0], (0, 1, 1, 5)), (x, got[0], (0, 2, 0, 63)), (w, got[3], (17,))):
        e = torch.zeros_like(t, dtype=torch.float64)
        e[at] = h
        args = [(x.double(), w.double())] * 2
        args = [(a + s * e, b) if t is x else (a, b + s * e) for (a, b), s in zip(args, (1, -1))]
        d_num = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        assert abs(d_num - grad[at].double()) <= 1e-5 * (1 + abs(d_num))


def test_helper_refusals():
    g = gen(13)
    q, k, v = fused(g, 2, 16, 4, 2, 64, BF16)
    plan = pkg.rotary_plan(64, (32, 32))
    pos = pkg.grid_positions((4, 4))

    def bad(code, fn, *args, **kw):
        with pytest.raises(bb.BsaError) as e:
            fn(*args, **kw)
        assert e.value.code == code

    bad(bb.ERR_INVALID_ARG, pkg.rotary, plan, q)
    bad(bb.ERR_SHAPE, pkg.rotary, plan, q, positions=pos[:15])
    bad(bb.ERR_SHAPE, pkg.rotary, plan, q, positions=pos[:, :1].contiguous())
    bad(bb.ERR_DTYPE, pkg.rotary, plan, q, positions=pos.long())
    bad(bb.ERR_INVALID_ARG, pkg.rotary, plan, q, positions=pos.t().contiguous().t())
    bad(bb.ERR_INVALID_ARG, pkg.rotary, plan, q, positions=pos.cpu())
    bad(bb.ERR_DTYPE, pkg.rotary, plan, q.half(), positions=pos)
    bad(bb.ERR_DTYPE, pkg.rotary, plan, q, k.float(), positions=pos)
    bad(bb.ERR_SHAPE, pkg.rotary, plan, q, k[:, :8], positions=pos)
    bad(bb.ERR_SHAPE, pkg.rotary, pkg.rotary_plan(128, (32, 32)), q, positions=pos)
    bad(bb.ERR_INVALID_ARG, pkg.rotary, plan, q.transpose(1, 3).contiguous().transpose(1, 3), positions=pos)
    bad(bb.ERR_SHAPE, pkg.rotary, plan, q, positions=pos, out=(torch.empty_like(q), None, None))
    bad(bb.ERR_SHAPE, pkg.rotary, plan, q, positions=pos, norm_eps=1e-6, q_weight=torch.ones(128, device=DEV))
    bad(bb.ERR_DTYPE, pkg.rotary, plan, q, positions=pos, norm_eps=1e-6, q_weight=torch.ones(64, device=DEV, dtype=BF16))
    o = torch.empty(2, 4, 1, 64, device=DEV, dtype=BF16).expand(2, 4, 16, 64)  # every token in one place
    bad(bb.ERR_INVALID_ARG, pkg.rotary, plan, q, positions=pos, out=(o, None, None))
    dq = torch.empty(2, 4, 16, 64, device=DEV, dtype=BF16)
    bad(bb.ERR_INVALID_ARG, pkg.rotary_backward, plan, dq, positions=pos, norm_eps=1e-6)
    bad(bb.ERR_SHAPE, pkg.rotary_backward, plan, dq, positions=pos, norm_eps=1e-6, q=k)
    small = torch.empty(256, device=DEV, dtype=torch.uint8)
    bad(bb.ERR_WORKSPACE, pkg.rotary_backward, plan, dq, positions=pos, norm_eps=1e-6, q=q,
        q_weight=torch.ones(64, device=DEV), ws=small)


def test_weight_without_the_norm_is_refused():
    """it would change nothing, and its gradient would be missing"""
    g = gen(14)
    q, k, _ = fused(g, 1, 8, 2, 2, 64, BF16)
    plan, pos, w = pkg.rotary_plan(64, (64,)), pkg.grid_positions((8,)), torch.ones(64, device=DEV)
    dq, dk = (t.transpose(1, 2).contiguous() for t in (q, k))
    for fn, args, more in ((pkg.rotary, (q, k), {}), (pkg.rotary_backward, (dq, dk), dict(q=q, k=k))):
        for weights in (dict(q_weight=w), dict(k_weight=w), dict(q_weight=w, k_weight=w)):
            with pytest.raises(bb.BsaError) as e:
                fn(plan, *args, positions=pos, **more, **weights)
            assert e.value.code == bb.ERR_INVALID_ARG
        fn(plan, *args, positions=pos, **more)


@pytest.mark.parametrize("d,axes,interleaved", [(64, (24, 40), True), (128, (16, 56, 56), False), (128, (44, 42, 42), True)])
def test_cosine_and_sine_of_every_position(d, axes, interleaved):
    """Pairs of (1, 0) come out as (cos t, sin t), and as (cos t, -sin t) on the way back, with t as the plan has it
    in whole numbers. In units of 2^-24 the larger error, the cosine's, is at most 1.39: t's conversion 0.31 (2^-27 and
    2^-31 half turns, pi each, a slope of sin(pi / 4)), r^2 0.15 (half of 2^-28, times pi^2 / 2), the coefficient and the
    rounding beside it 0.15 and 0.25 (of 4.93, times 1 / 16), the further terms 0.03, the result 0.5. The sine's terms
    beside pi r are below 0.08: 0.31, 0.32 and 0.5."""
    g = gen(15)
    n_axes, rot = len(axes), sum(axes)
    some = torch.tensor([0, 1, -1, 2, 3, 4095, -4096, 2 ** 31 - 1, -2 ** 31, 2 ** 30], device=DEV, dtype=torch.int64)
    pos = torch.cat([some[:, None].expand(-1, n_axes),
                     torch.randint(-2 ** 31, 2 ** 31 - 1, (1000, n_axes), generator=g, device=DEV, dtype=torch.int64),
                     torch.randint(-4000, 4000, (1000, n_axes), generator=g, device=DEV, dtype=torch.int64)])
    N = pos.shape[0]
    plan = pkg.rotary_plan(d, axes, interleaved=interleaved)
    at = pos.tolist()
    t = torch.tensor([[(plan.turns[p] * at[n][plan.axis[p]]) % 2 ** 64 / 2.0 ** 64 for p in range(rot // 2)] for n in range(N)],
                     dtype=torch.float64, device=DEV) * (2.0 * torch.pi)
    x = torch.zeros(1, N, 1, d, device=DEV)
    a, _ = ref.split_pairs(x, rot // 2, interleaved)
    a.fill_(1.0)
    pos = pos.to(torch.int32)
    bound = 1.4 * 2.0 ** -24 + 2.0 ** -50  # and the 64-bit reference's own
    out = pkg.rotary(plan, x, positions=pos)[0].transpose(1, 2)
    back = pkg.rotary_backward(plan, x.transpose(1, 2).contiguous(), positions=pos)[0]
    for got, sign in ((out, 1.0), (back, -1.0)):
        c, s = (v[0, :, 0].double() for v in ref.split_pairs(got, rot // 2, interleaved))
        assert (c - t.cos()).abs().max() <= bound
        assert (s - sign * t.sin()).abs().max() <= bound
