"""The attention step of a block as a model runs it: fused projection -> rotary -> mask -> sparse forward ->
gated norm, and the operators' backward passes around it, each stage against its own reference."""
import concurrent.futures
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_sparse_attention_mean_gb300 as pkg
import oracle
from block_sparse_attention_mean_gb300 import binding as bb
from block_sparse_attention_mean_gb300 import block_binding as ob
from block_sparse_attention_mean_gb300 import build as bbuild
from tests import block_ref as ref
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bbuild.build()
    oracle.build()
    ob.load()


@pytest.mark.parametrize("static,d,grid,n_text", [(True, 64, (8, 8, 8), 128), (False, 128, (4, 8, 9), 40)])
def test_attention_step(static, d, grid, n_text):
    B, H = 2, 4
    N, C = n_text + grid[0] * grid[1] * grid[2], H * d
    g = torch.Generator(DEV).manual_seed(1)

    def draw(*shape, dt=torch.bfloat16, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale + mean).to(dt)

    qkv, x = draw(B, N, 3 * H, d), draw(B, N, C)
    src = qkv.split(H, dim=2)
    weights = [draw(d, dt=torch.float32, scale=0.2, mean=1.0) for _ in range(2)]
    axes = (16, 24, 24) if d == 64 else (44, 42, 42)
    plan = pkg.rotary_plan(d, axes)
    pos = pkg.grid_positions(grid, n_text, cuboid=(4, 4, 4) if static else None)
    spec = bb.cuboid_spec(n_text // 64, tuple(s // 4 for s in grid)) if static else None
    post, pre = pkg.NormSpec("rms", draw(C, dt=torch.float32, mean=1.0)), pkg.NormSpec("layer")
    rows = draw(B, 3, C, scale=0.3)
    mods = dict(gate=rows[:, 0], scale=rows[:, 1], shift=rows[:, 2])
    proj = draw(C, C, scale=C ** -0.5)

    # the step, without a wait between its calls
    q, k, v = pkg.rotary(plan, *src, positions=pos, norm_eps=1e-6, q_weight=weights[0], k_weight=weights[1])
    idx = bb.build_mask(None if static else q, None if static else k, 64, density=0.25, spec=spec, shape=(B, H, N, d),
                        check=False)
    o, lse = bb.forward(q, k, v, idx, check=False)
    y = o.transpose(1, 2).reshape(B, N, C) @ proj
    h, z = pkg.gated_norm(x, y, post=post, pre=pre, **mods)
    torch.cuda.synchronize()

    ang = ref.angles(pos, axes, 10000.0)
    for got, t, w, name in ((q, src[0], weights[0], "q"), (k, src[1], weights[1], "k")):
        ref.within(got, *ref.rotary(t, ang, True, 1e-6, w), name)
    assert torch.equal(v, src[2].transpose(1, 2))

    host = [t.float().cpu().numpy() for t in (q, k, v)]
    nB = -(-N // 64)
    if static:
        mask = np.broadcast_to(oracle.cuboid_mask(n_text // 64, tuple(s // 4 for s in grid)), (B, H, nB, nB)).copy()
    else:
        mask = oracle.select_mask(host[0], host[1], 64, 0.25)
    gu.assert_index_equal(idx, mask)
    o_ref, l_ref = oracle.attention(*host, mask, 64)
    err = np.abs(o.float().cpu().numpy().reshape(-1, d) - o_ref)
    assert err.max() <= gu.O_MAX_ABS and err.mean() <= gu.O_MEAN_ABS
    assert np.abs(lse.cpu().numpy().reshape(-1) - l_ref).max() <= gu.LSE_MAX_ABS

    kw = dict(mods, post=("rms", post.weight, None, 1e-6), pre=("layer", None, None, 1e-6))
    (rh, dh), (rz, dz) = ref.gated_norm(x, y, **kw)
    ref.within(h, rh, dh, "h")
    ref.within(z, rz, dz, "z")

    # the way back through the two operators, the arriving gradients in the layouts the attention has
    gh, gz = draw(B, N, C), draw(B, N, C)
    back = pkg.gated_norm_backward(gh, gz, h, y, post=post, pre=pre, **mods)
    want = ref.gated_norm_backward(gh, gz, h, y, **kw)
    for name in ("dx", "dy", "dpost_weight"):
        ref.within(getattr(back, name), *want[name], name)
    dqkv = torch.empty_like(qkv)
    do = [draw(B, H, N, d) for _ in range(3)]
    dw = pkg.rotary_backward(plan, *do, positions=pos, q=src[0], k=src[1], norm_eps=1e-6, q_weight=weights[0],
                             k_weight=weights[1], out=dqkv.split(H, dim=2))[3:]
    for i, w in enumerate(weights):
        dx, bound, rdw, dw_bound = ref.rotary_backward(do[i], ang, True, src[i], 1e-6, w)
        ref.within(dqkv[:, :, i * H:(i + 1) * H], dx, bound, f"d{'qk'[i]}")
        ref.within(dw[i], rdw, dw_bound, "weight")
    assert torch.equal(dqkv[:, :, 2 * H:], do[2].transpose(1, 2))


def test_two_steps_on_two_streams():
    """the operators on two streams at once, each with its own buffers, as two halves of a batch would run"""
    g = torch.Generator(DEV).manual_seed(2)
    B, N, H, d = 1, 2000, 8, 128
    plan = pkg.rotary_plan(d, (44, 42, 42))
    pos = pkg.grid_positions((8, 10, 25))
    w = torch.ones(d, device=DEV)
    post = pkg.NormSpec("rms", torch.ones(H * d, device=DEV))
    pre = pkg.NormSpec("layer")
    inputs = [[torch.randn(*s, generator=g, device=DEV).bfloat16() for s in ((B, N, 3 * H, d), (B, N, H * d), (B, N, H * d))]
              for _ in range(2)]

    def half(qkv, x, y):
        out = pkg.rotary(plan, *qkv.split(H, dim=2), positions=pos, norm_eps=1e-6, q_weight=w, k_weight=w)
        back = pkg.rotary_backward(plan, *out, positions=pos, q=qkv[:, :, :H], k=qkv[:, :, H:2 * H], norm_eps=1e-6,
                                   q_weight=w, k_weight=w)
        h, z = pkg.gated_norm(x, y, post=post, pre=pre)
        return (*out, *back, h, z, *(t for t in pkg.gated_norm_backward(h, z, h, y, post=post, pre=pre) if t is not None))

    alone = [half(*i) for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, i in zip(streams, inputs):
            with torch.cuda.stream(s):
                got.append(half(*i))
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def side_stream_case():
    """(plan, call): call(stream) runs the two operators and their backward passes, all results and workspaces
    left to the helpers"""
    g = torch.Generator(DEV).manual_seed(3)
    B, N, H, d = 1, 1500, 4, 128
    C = H * d
    pos = pkg.grid_positions((6, 10, 25))
    plan = pkg.rotary_plan(d, (44, 42, 42))
    w = torch.randn(d, generator=g, device=DEV)
    qkv = torch.randn(B, N, 3, H, d, generator=g, device=DEV).bfloat16().unbind(2)
    x, y, dh, dz = (torch.randn(B, N, C, generator=g, device=DEV).bfloat16() for _ in range(4))
    kw = dict(gate=torch.randn(B, C, generator=g, device=DEV),
              post=pkg.NormSpec("rms", torch.randn(C, generator=g, device=DEV)), pre=pkg.NormSpec("layer"))
    grads = [torch.randn(B, H, N, d, generator=g, device=DEV).bfloat16() for _ in range(3)]
    turn = dict(positions=pos, norm_eps=1e-6, q_weight=w, k_weight=w)

    def call(stream):
        out = [*pkg.rotary(plan, *qkv, **turn, stream=stream)]
        out += pkg.rotary_backward(plan, *grads, q=qkv[0], k=qkv[1], **turn, stream=stream)
        out += pkg.gated_norm(x, y, **kw, stream=stream)
        out += pkg.gated_norm_backward(dh, dz, x, y, **kw, stream=stream)
        return [t for t in out if t is not None]

    sizes = sorted({t.numel() * t.element_size() for t in call(None)} |
                   {pkg.rotary_workspace(B, N, d).numel(), pkg.gated_norm_workspace(B, N, C).numel()})
    return call, sizes


@pytest.mark.parametrize("given", ["stream", "handle"])
@pytest.mark.parametrize("late", ["side", "current"])
def test_what_a_call_allocates_belongs_to_its_stream(given, late):
    """Around a call on a side stream the current stream frees, allocates and fills tensors of the sizes of its
    workspaces and results. Whichever of the two streams runs late, neither may touch the other's tensors: a workspace
    that goes back to the current stream's pool would be written behind the fill of the tensor that took its place,
    and a result from that pool would be written before the fill of the tensor that had its place."""
    call, sizes = side_stream_case()
    expected = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        if late == "current":
            torch.cuda._sleep(20_000_000)
        else:
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0x55)
        got = call(side if given == "stream" else side.cuda_stream)
        mine = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xAA) for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        assert len(got) == len(expected)
        for a, b in zip(got, expected):
            assert torch.equal(a, b)
        for t in mine:
            assert t.eq(0xAA).all()


def test_the_default_stream_from_another():
    """handles 0 and 1 both name the default stream, and a stream object of it does"""
    call, _ = side_stream_case()
    expected = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (0, 1, torch.cuda.default_stream()):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            got = call(stream)
            assert torch.cuda.current_stream() == side
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, expected))


def test_inside_an_autograd_function():
    """as a training step uses the two pairs: parameters that require gradients, which arrive from the backward
    helpers"""
    g = torch.Generator(DEV).manual_seed(4)
    B, N, H, d = 2, 70, 4, 64
    C = H * d
    plan, pos = pkg.rotary_plan(d, (16, 24, 24)), pkg.grid_positions((2, 5, 7))

    def draw(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, w):
            ctx.save_for_backward(q, w)
            return pkg.rotary(plan, q, positions=pos, norm_eps=1e-6, q_weight=w)[0]

        @staticmethod
        def backward(ctx, dy):
            q, w = ctx.saved_tensors
            got = pkg.rotary_backward(plan, dy.contiguous(), positions=pos, q=q, norm_eps=1e-6, q_weight=w)
            return got[0], got[3]

    class Step(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, y, gate, w):
            h, z = pkg.gated_norm(x, y, gate=gate, pre=pkg.NormSpec("rms", w))
            ctx.save_for_backward(h, y, gate, w)
            return h, z

        @staticmethod
        def backward(ctx, dh, dz):
            h, y, gate, w = ctx.saved_tensors
            got = pkg.gated_norm_backward(dh.contiguous(), dz.contiguous(), h, y, gate=gate, pre=pkg.NormSpec("rms", w))
            return got.dx, got.dy, got.dgate, got.dpre_weight

    q, wq, x, gate, w = draw(B, N, H, d), draw(d), draw(B, N, C), draw(B, C), draw(C)
    leaves = [t.requires_grad_() for t in (q, wq, x, gate, w)]
    o = Turn.apply(q, wq)
    h, z = Step.apply(x, o.transpose(1, 2).reshape(B, N, C), gate, w)
    ch, cz = draw(B, N, C), draw(B, N, C)
    got = torch.autograd.grad((h * ch + z * cz).sum(), leaves)

    # the calls one by one (each is compared with its 64-bit form elsewhere): the same bits
    with torch.no_grad():
        y = pkg.rotary(plan, q, positions=pos, norm_eps=1e-6, q_weight=wq)[0].transpose(1, 2).reshape(B, N, C)
        pre = pkg.NormSpec("rms", w)
        h2, z2 = pkg.gated_norm(x, y, gate=gate, pre=pre)
        back = pkg.gated_norm_backward(ch, cz, h2, y, gate=gate, pre=pre)
        dy = back.dy.view(B, N, H, d).transpose(1, 2).contiguous()
        turned = pkg.rotary_backward(plan, dy, positions=pos, q=q, norm_eps=1e-6, q_weight=wq)
    assert torch.equal(h, h2) and torch.equal(z, z2)
    for a, b, name in zip(got, (turned[0], turned[3], back.dx, back.dgate, back.dpre_weight), ("q", "wq", "x", "gate", "w")):
        assert torch.equal(a, b), name


def test_two_graphs_with_one_workspace():
    """captured one after the other with the same workspaces and replayed in turn on one stream: neither needs what
    the other left there"""
    g = torch.Generator(DEV).manual_seed(5)
    N, H, d = 700, 4, 64
    C = H * d
    plan, pos, w = pkg.rotary_plan(d, (64,)), torch.arange(N, device=DEV, dtype=torch.int32)[:, None], torch.ones(d, device=DEV)
    ws = pkg.rotary_workspace(1, N, d), pkg.gated_norm_workspace(1, N, C)
    post = pkg.NormSpec("rms", torch.ones(C, device=DEV))

    def draw(*s):
        return torch.randn(*s, generator=g, device=DEV).bfloat16()

    def back(q, dy, x, y, ws):
        got = pkg.rotary_backward(plan, dy, positions=pos, q=q, norm_eps=1e-6, q_weight=w, ws=ws[0])
        more = pkg.gated_norm_backward(x, y, x, y, post=post, pre=pkg.NormSpec("layer"), ws=ws[1])
        return [t for t in (*got, *more) if t is not None]

    inputs = [(draw(1, N, H, d), draw(1, H, N, d), draw(1, N, C), draw(1, N, C)) for _ in range(2)]
    expected = [back(*i, (None, None)) for i in inputs]
    torch.cuda.synchronize()
    graphs, got = [], []
    for i in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(back(*i, ws))
        graphs.append(graph)
    for k in (0, 1, 1, 0, 1):
        for t in got[k]:
            t.zero_()
        graphs[k].replay()
        graphs[1 - k].replay()
        torch.cuda.synchronize()
        for a, b in zip(got, expected):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_threads_at_once():
    """two host threads, a stream each: every call has the bits that it has alone"""
    g = torch.Generator(DEV).manual_seed(6)
    N, d = 300, 128
    plan, pos, w = pkg.rotary_plan(d, (44, 42, 42)), pkg.grid_positions((3, 10, 10)), torch.ones(d, device=DEV)

    def draw(*s):
        return torch.randn(*s, generator=g, device=DEV).bfloat16()

    def step(q, x, y):
        turned = pkg.rotary(plan, q, positions=pos, norm_eps=1e-6, q_weight=w)[0]
        back = pkg.rotary_backward(plan, turned, positions=pos, q=q, norm_eps=1e-6, q_weight=w)
        h, z = pkg.gated_norm(x, y, pre=pkg.NormSpec("layer"))
        more = pkg.gated_norm_backward(h, z, h, y, post=pkg.NormSpec("rms", eps=1e-3), pre=pkg.NormSpec("layer"))
        return [t for t in (turned, *back, h, z, *more) if t is not None]

    inputs = [(draw(1, N, 4, d), draw(1, N, 512 + 520 * i), draw(1, N, 512 + 520 * i)) for i in range(2)]
    expected = [step(*i) for i in inputs]
    torch.cuda.synchronize()

    def work(i):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            runs = [step(*inputs[i]) for _ in range(20)]
        side.synchronize()
        return all(torch.equal(a, b) for run in runs for a, b in zip(run, expected[i]))

    with concurrent.futures.ThreadPoolExecutor(2) as pool:
        assert all(pool.map(work, range(2)))


FIRST_CALL = """
import torch
import block_sparse_attention_mean_gb300 as pkg
g = torch.Generator("cuda").manual_seed(1)
def draw(*s): return torch.randn(*s, generator=g, device="cuda").bfloat16()
q, x, y = draw(1, 40, 2, 64), draw(1, 40, 1032), draw(1, 40, 1032)
pos, w = torch.arange(40, device="cuda", dtype=torch.int32)[:, None], torch.ones(64, device="cuda")
plan, post, pre = pkg.rotary_plan(64, (64,)), pkg.NormSpec("rms", torch.ones(1032, device="cuda")), pkg.NormSpec("layer")
def step():
    a = pkg.rotary(plan, q, positions=pos, norm_eps=1e-6, q_weight=w)[0]
    b = pkg.rotary_backward(plan, a, positions=pos, q=q, norm_eps=1e-6, q_weight=w)
    h, z = pkg.gated_norm(x, y, post=post, pre=pre)
    return [t for t in (a, *b, h, z, *pkg.gated_norm_backward(h, z, h, y, post=post, pre=pre)) if t is not None]
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("same")
"""


def test_first_call_of_a_process_inside_a_capture():
    """what the library looks up once per kernel it may look up while a graph is captured"""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.split() == ["same"], r.stdout + r.stderr
