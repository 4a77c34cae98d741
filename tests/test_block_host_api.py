"""Checks of the operators around the attention that need no GPU: the header and the binding agree,
the rotary plan's frequencies, and the refusals, which all happen before any launch."""
import contextlib
import ctypes
import decimal
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

import block_sparse_attention_mean_gb300 as pkg
from block_sparse_attention_mean_gb300 import binding as bb
from block_sparse_attention_mean_gb300 import block_binding as ob
from block_sparse_attention_mean_gb300 import build as bbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bsa_block.h")
FAKE = 1 << 40  # an aligned non-null address that is never dereferenced on these paths
FAR = 1 << 36   # between two such tensors


@pytest.fixture(scope="module", autouse=True)
def lib():
    bbuild.build()
    return ob.load()


def refused(code, fn, *args, **kw):
    with pytest.raises(bb.BsaError) as e:
        fn(*args, **kw)
    assert e.value.code == code, str(e.value)


def test_header_symbols_exported(lib):
    names = sorted(re.findall(r"^bsa_status\s+(bsa_\w+)\s*\(", open(HEADER).read(), re.M))
    assert sorted(ob.EXPORTS) == names
    for n in names:
        assert getattr(lib, n) is not None


@pytest.mark.parametrize("cc,std,lang", [("gcc", "-std=c99", "c"), ("g++", "-std=c++17", "c++")])
def test_header_is_plain_c_and_cpp(cc, std, lang):
    if shutil.which(cc) is None:
        pytest.skip(f"{cc} not available")
    r = subprocess.run([cc, std, "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-x", lang, HEADER],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_struct_layouts_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    mirrors = {"bsa_rotary_spec": ob.RotarySpec, "bsa_rotary_plan": ob.RotaryPlan, "bsa_heads": ob.Heads,
               "bsa_heads_grad": ob.HeadsGrad, "bsa_norm": ob.Norm, "bsa_rows": ob.Rows,
               "bsa_modulation": ob.Modulation, "bsa_gated_norm_desc": ob.GatedNormDesc,
               "bsa_gated_norm_grads": ob.GatedNormGradArgs}
    lines, expected = [], []
    for c, m in mirrors.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        expected.append(ctypes.sizeof(m))
        for name, _ in m._fields_:
            lines.append(f'printf("%zu\\n", offsetof({c}, {name}));')
            expected.append(getattr(m, name).offset)
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stdio.h>\n#include "{HEADER}"\nint main(void) {{\n' + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == expected


def test_packed_descriptors_match_the_structures():
    """the helpers' byte layouts: every field of a mirror holds what was packed at its place"""
    for fmt, mirror in ((ob._HEADS, ob.Heads), (ob._HEADS_GRAD, ob.HeadsGrad), (ob._ROWS, ob.Rows),
                        (ob._DESC, ob.GatedNormDesc), (ob._GRADS, ob.GatedNormGradArgs)):
        assert fmt.size == ctypes.sizeof(mirror)
        n = len(fmt.unpack(bytes(fmt.size)))
        got = mirror.from_buffer_copy(fmt.pack(*range(1, n + 1)))

        def flat(v):
            return [x for f, _ in v._fields_ for x in flat(getattr(v, f))] if isinstance(v, ctypes.Structure) else [v]

        assert flat(got) == list(range(1, n + 1))


def test_package_offers_the_helpers():
    for name in ("rotary", "rotary_backward", "rotary_plan", "gated_norm", "gated_norm_backward", "NormSpec",
                 "grid_positions"):
        assert name in pkg.__all__ and getattr(pkg, name) is getattr(ob, name)


# ------------------------------------------------------------------ the rotary plan


def _angle(plan, p, pos):
    """the angle of pair p at a position, as the kernels form it: the product modulo 2^64, in turns"""
    ph = (plan.turns[p] * (pos % (1 << 64))) % (1 << 64)
    ph = ph - (1 << 64) if ph >= 1 << 63 else ph
    return ph / 2.0 ** 64 * 2.0 * math.pi


@pytest.mark.parametrize("dims,theta,scale", [((128,), 10000.0, 1.0), ((44, 42, 42), 256.0, 1.0),
                                              ((16, 56, 56), (100.0, 10000.0, 500000.0), (1.0, 0.5, 40.0)),
                                              ((2, 2, 2, 2), 10000.0, -1.0)])
@pytest.mark.parametrize("pos", [0, 1, -1, 17, 4095, -70001, 2 ** 31 - 1, -2 ** 31])
def test_plan_angles(dims, theta, scale, pos):
    plan = ob.rotary_plan(128, dims, theta=theta, scale=scale, interleaved=True)
    p = 0
    for a, dim in enumerate(dims):
        th = theta if isinstance(theta, float) else theta[a]
        sc = scale if isinstance(scale, float) else scale[a]
        for j in range(dim // 2):
            f = sc * th ** (-2.0 * j / dim)
            # f is within 2^-51 (the plan's, and this one's pow) and the fixed point within 2^-65 turns
            off = abs(pos) * (abs(f) * 2.0 ** -50 + 2.0 ** -64 * math.pi) + 1e-15
            d = math.remainder(_angle(plan, p, pos) - math.remainder(pos * f, 2.0 * math.pi), 2.0 * math.pi)
            assert abs(d) <= off + abs(pos * f) * 2.0 ** -51
            assert plan.axis[p] == a
            p += 1
    assert (plan.rot, plan.n_axes, plan.d) == (sum(dims), len(dims), 128)


# 2 pi to 60 places
TWO_PI = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def check_turns(plan, p, f):
    """turns[p] against the frequency f (60 digits): within 2^-51 of its value and half a unit, 2^-65 turns"""
    with decimal.localcontext(prec=60):
        turns = f / TWO_PI
        off = (decimal.Decimal(plan.turns[p]) / 2 ** 64 - turns) % 1
        off = min(abs(off), abs(off - 1), abs(off + 1))
        assert off <= abs(turns) / 2 ** 51 + decimal.Decimal(2) ** -65, (p, float(off / (abs(turns) + decimal.Decimal(10) ** -40)))


@pytest.mark.parametrize("theta", [10000.0, 500000.0, 256.0, 3.7, 1e8, 0.25, 1.0])
@pytest.mark.parametrize("dim", [2, 6, 16, 42, 44, 48, 56, 62, 112, 128])
def test_plan_frequencies(theta, dim):
    for scale in (1.0, -0.3, 40.0):
        plan = ob.rotary_plan(128, [dim], theta=theta, scale=scale)
        with decimal.localcontext(prec=60):
            for j in range(dim // 2):
                f = decimal.Decimal(scale) * decimal.Decimal(theta) ** (decimal.Decimal(-2 * j) / dim)
                check_turns(plan, j, f)


def test_plan_given_frequencies_are_exact():
    freq = [1.0, math.pi, -0.1, 3e-7, 1e-19, 12345.678, 2.0 ** 40 + 0.5, 0.0]
    plan = ob.rotary_plan(64, [16], inv_freq=freq)
    for p, f in enumerate(freq):
        check_turns(plan, p, decimal.Decimal(f))


def test_plan_given_frequencies():
    plan = ob.rotary_plan(64, [4, 2], inv_freq=[0.0, math.pi, -0.25])
    assert abs(_angle(plan, 0, 12345)) == 0.0
    assert abs(abs(_angle(plan, 1, 3)) - math.pi) < 1e-12
    assert abs(_angle(plan, 2, 2) + 0.5) < 1e-12


def test_plan_refusals():
    for dims in ([], [2] * 5, [3], [0], [-2], [64, 66], [130]):
        refused(bb.ERR_INVALID_ARG, ob.rotary_plan, 128, dims)
    refused(bb.ERR_INVALID_ARG, ob.rotary_plan, 64, [66])
    refused(bb.ERR_INVALID_ARG, ob.rotary_plan, 64, [6, 2], interleaved=False)  # rot not a multiple of 16
    for d in (0, 32, 96, 256):
        refused(bb.ERR_SHAPE, ob.rotary_plan, d, [16])
    for theta in (0.0, -1.0, math.inf, math.nan):
        refused(bb.ERR_INVALID_ARG, ob.rotary_plan, 64, [16], theta=theta)
    refused(bb.ERR_INVALID_ARG, ob.rotary_plan, 64, [16], scale=math.inf)
    refused(bb.ERR_INVALID_ARG, ob.rotary_plan, 64, [16, 16], theta=[1.0])
    refused(bb.ERR_INVALID_ARG, ob.rotary_plan, 64, [4], inv_freq=[1.0])
    refused(bb.ERR_INVALID_ARG, ob.rotary_plan, 64, [4], inv_freq=[1.0, math.nan])
    refused(bb.ERR_INVALID_ARG, ob.bsa_rotary_plan_init, None, 64, None)


def test_grid_positions():
    pos = ob.grid_positions((2, 4, 4), n_text=3, device="cpu")
    assert pos.dtype == torch.int32 and pos.shape == (35, 3)
    assert pos[:3].eq(0).all() and pos[3 + 1 * 16 + 2 * 4 + 3].tolist() == [1, 2, 3]
    cub = ob.grid_positions((4, 8, 8), cuboid=(2, 4, 4), device="cpu")
    assert cub.shape == (256, 3)
    # cuboid (1, 0, 1) is number 5 of 8; its token (1, 2, 3) is number 27 of 32
    assert cub[5 * 32 + 27].tolist() == [2 + 1, 0 + 2, 4 + 3]
    assert len({tuple(p) for p in cub.tolist()}) == 256
    refused(bb.ERR_SHAPE, ob.grid_positions, (4, 6), cuboid=(2, 4), device="cpu")


# ------------------------------------------------------------------ refusals, rotary


def _plan(**kw):
    return ob.rotary_plan(64, [32, 32], **kw)


def _heads(i, H=2, N=16, d=64, **kw):
    a = dict(src=FAKE + i * FAR, src_batch=N * H * d, src_token=H * d, src_head=d, dst=FAKE + (i + 8) * FAR,
             dst_batch=H * N * d, dst_token=d, dst_head=N * d, weight=None, heads=H)
    a.update(kw)
    return ob.Heads(*a.values())


def _rotary(code, plan=None, q=True, k=None, v=None, dt=bb.BF16, B=2, N=16, pos=FAKE, pos_batch=0, norm=1, eps=1e-6):
    refused(code, ob.bsa_rotary, _plan() if plan is None else plan, _heads(0) if q is True else q, k, v, dt, B, N, pos,
            pos_batch, norm, eps, 0)


def test_rotary_refusals():
    inv = bb.ERR_INVALID_ARG
    refused(inv, ob.bsa_rotary, None, _heads(0), None, None, bb.BF16, 2, 16, FAKE, 0, 1, 1e-6, 0)
    _rotary(inv, plan=ob.RotaryPlan())
    for field, value in (("d", 96), ("rot", 66), ("rot", 3), ("rot", 0), ("n_axes", 0), ("n_axes", 1), ("pairing", 2)):
        bad = _plan()
        setattr(bad, field, value)
        _rotary(inv, plan=bad)
    bad = _plan()
    bad.axis[3] = 2
    _rotary(inv, plan=bad)
    _rotary(inv, q=None)
    _rotary(bb.ERR_SHAPE, B=0)
    _rotary(bb.ERR_SHAPE, N=0)
    _rotary(bb.ERR_SHAPE, B=1 << 20, N=1 << 20)
    _rotary(bb.ERR_DTYPE, dt=2)
    _rotary(inv, pos=None)
    _rotary(inv, pos=FAKE + 2)
    _rotary(inv, pos_batch=-1)
    _rotary(inv, eps=-1.0)
    _rotary(inv, eps=math.nan)
    for bad in (dict(src=None), dict(dst=None), dict(src=FAKE + 8), dict(src_token=132), dict(dst_head=-1024),
                dict(src_head=4), dict(weight=FAKE + 4), dict(src_batch=1 << 60), dict(dst_token=0), dict(dst_head=64),
                dict(dst_batch=64)):
        _rotary(inv, q=_heads(0, **bad))
    _rotary(bb.ERR_SHAPE, q=_heads(0, heads=0))
    _rotary(bb.ERR_SHAPE, q=_heads(0, heads=65536))


def test_rotary_overlaps():
    inv = bb.ERR_INVALID_ARG
    same = dict(dst_batch=16 * 128, dst_token=128, dst_head=64)
    _rotary(inv, q=_heads(0, dst=FAKE))                                  # in place, with other strides
    _rotary(inv, q=_heads(0, dst=FAKE + 128, **same))                    # half a token further
    _rotary(inv, q=_heads(0, dst=FAKE + 2 * 16 * 128, **same))           # a batch further
    _rotary(inv, q=_heads(0), k=_heads(1, dst=FAKE + 8 * FAR))           # two outputs in one place
    _rotary(inv, q=_heads(0), k=_heads(1, src=FAKE + 8 * FAR))           # an output over another's input
    # q and k interleaved in one buffer with one head too many
    t = dict(dst_batch=16 * 384, dst_token=384, dst_head=64)
    _rotary(inv, q=_heads(0, dst=FAKE + 9 * FAR, **t), k=_heads(1, H=3, dst=FAKE + 9 * FAR + 128, **t), v=_heads(
        2, H=3, dst=FAKE + 9 * FAR + 128 * 3, **t))


def _grad(i, H=2, N=16, d=64, **kw):
    a = dict(dy=FAKE + i * FAR, dy_batch=H * N * d, dy_token=d, dy_head=N * d, x=FAKE + (i + 8) * FAR,
             x_batch=N * H * d, x_token=H * d, x_head=d, dx=FAKE + (i + 16) * FAR, dx_batch=N * H * d, dx_token=H * d,
             dx_head=d, weight=FAKE, dweight=FAKE, heads=H)
    a.update(kw)
    return ob.HeadsGrad(*a.values())


def test_rotary_backward_refusals():
    def call(code, q=True, k=None, v=None, dt=bb.BF16, B=2, N=16, pos=FAKE, norm=1, eps=1e-6, ws=FAKE, n=1 << 30):
        refused(code, ob.bsa_rotary_backward, _plan(), _grad(0) if q is True else q, k, v, dt, B, N, pos, 0, norm, eps,
                ws, n, 0)

    inv = bb.ERR_INVALID_ARG
    call(inv, q=None)
    call(bb.ERR_SHAPE, N=0)
    call(bb.ERR_DTYPE, dt=-1)
    call(inv, pos=None)
    call(inv, eps=math.inf)
    call(inv, q=_grad(0, x=None))
    call(inv, q=_grad(0, dy=None))
    call(inv, q=_grad(0, dx=None))
    call(inv, q=_grad(0, dweight=FAKE + 2))
    call(inv, norm=0)                                     # a weight's gradient without the norm
    call(inv, q=None, v=_grad(0))                         # V has no weight
    call(inv, q=_grad(0, dx=FAKE))                        # over dy, in another layout
    call(inv, q=_grad(0, dx_token=0))
    call(bb.ERR_SHAPE, q=_grad(0, heads=0))
    need = ob.bsa_rotary_workspace_size(2, 16, 64)
    call(bb.ERR_WORKSPACE, ws=None)
    call(bb.ERR_WORKSPACE, ws=FAKE + 128)
    call(bb.ERR_WORKSPACE, n=need - 1)
    refused(bb.ERR_SHAPE, ob.bsa_rotary_workspace_size, 1, 0, 64)
    refused(bb.ERR_SHAPE, ob.bsa_rotary_workspace_size, 1, 1, 80)


# ------------------------------------------------------------------ refusals, gated norm


def _rows(i, N=16, C=64, **kw):
    a = dict(ptr=FAKE + i * FAR, batch=N * C, token=C)
    a.update(kw)
    return ob.Rows(*a.values())


def _norm(kind=ob.NORM_LAYER, eps=1e-6, weight=None, bias=None):
    return ob.Norm(kind, eps, weight, bias)


def _mod(ptr=FAKE, batch=64, frame=64):
    return ob.Modulation(ptr, batch, frame)


def _desc(**kw):
    a = dict(B=2, N=16, C=64, F=1, stream_dt=bb.BF16, branch_dt=bb.BF16, mod_dt=bb.BF16, alpha=1.0,
             post=_norm(ob.NORM_NONE), pre=_norm(), gate=_mod(), scale=_mod(), shift=_mod())
    a.update(kw)
    return ob.GatedNormDesc(*a.values())


def _gated(code, x=True, y=True, h=True, z=True, **desc):
    pick = lambda t, i: _rows(i) if t is True else t  # noqa: E731
    refused(code, ob.bsa_gated_norm, _desc(**desc), pick(x, 0), pick(y, 1), pick(h, 2), pick(z, 3), 0)


BAD_DESC = [(bb.ERR_SHAPE, dict(B=0)), (bb.ERR_SHAPE, dict(N=0)), (bb.ERR_SHAPE, dict(B=1 << 20, N=1 << 20)),
            (bb.ERR_SHAPE, dict(C=0)), (bb.ERR_SHAPE, dict(C=60)), (bb.ERR_SHAPE, dict(C=8200)), (bb.ERR_SHAPE, dict(F=0)),
            (bb.ERR_SHAPE, dict(F=3)), (bb.ERR_DTYPE, dict(stream_dt=2)), (bb.ERR_DTYPE, dict(mod_dt=-1)),
            (bb.ERR_DTYPE, dict(branch_dt=bb.FP32)), (bb.ERR_INVALID_ARG, dict(alpha=math.nan)),
            (bb.ERR_INVALID_ARG, dict(pre=_norm(3))), (bb.ERR_INVALID_ARG, dict(pre=_norm(eps=-1.0))),
            (bb.ERR_INVALID_ARG, dict(pre=_norm(weight=FAKE + 4))),
            (bb.ERR_INVALID_ARG, dict(post=_norm(bias=FAKE + 8))),
            (bb.ERR_INVALID_ARG, dict(gate=_mod(FAKE + 2))), (bb.ERR_INVALID_ARG, dict(scale=_mod(batch=-64))),
            (bb.ERR_INVALID_ARG, dict(shift=_mod(batch=68))), (bb.ERR_INVALID_ARG, dict(F=2, shift=_mod(frame=3)))]


@pytest.mark.parametrize("code,bad", BAD_DESC)
def test_gated_norm_desc_refusals(code, bad):
    _gated(code, **bad)
    refused(code, ob.bsa_gated_norm_backward, _desc(**bad), _norm_grads(), FAKE, 1 << 40, 0)


def test_gated_norm_refusals():
    inv = bb.ERR_INVALID_ARG
    off = dict(pre=_norm(ob.NORM_NONE), scale=_mod(None), shift=_mod(None))
    refused(inv, ob.bsa_gated_norm, None, _rows(0), _rows(1), _rows(2), _rows(3), 0)
    _gated(inv, x=None)
    _gated(inv, h=None)
    _gated(inv, z=None)
    _gated(inv, y=None)                                     # an h without a branch
    _gated(inv, y=None, h=None)                             # a gate without one
    _gated(inv, y=None, h=None, gate=_mod(None), post=_norm())
    _gated(inv, y=None, h=None, z=None, gate=_mod(None), **off)  # nothing to do
    _gated(inv, **off)                                      # z without a pre norm
    _gated(inv, z=None, pre=_norm(ob.NORM_NONE))            # scale without one
    for bad in (dict(ptr=FAKE + 4), dict(token=60), dict(batch=-8), dict(token=1 << 60)):
        _gated(inv, x=_rows(0, **bad))
        _gated(inv, z=_rows(3, **bad))
    for bad in (dict(token=0), dict(token=32), dict(batch=0), dict(batch=64)):  # outputs over themselves
        _gated(inv, h=_rows(2, **bad))
    _gated(inv, h=_rows(3))                                 # both outputs in one place
    _gated(inv, h=_rows(1))                                 # h over y
    _gated(inv, z=_rows(0))                                 # z over x
    _gated(inv, h=_rows(0, token=128, batch=16 * 128), x=_rows(0))  # in place, with other strides
    _gated(inv, h=_rows(0, ptr=FAKE + 64), x=_rows(0))      # half a row further
    _gated(inv, h=_rows(0), x=_rows(0), stream_dt=bb.FP32, z=_rows(0))  # another dtype in the same place


def _norm_grads(**kw):
    p = {n: _rows(i) for i, n in enumerate(("dh", "dz", "h", "y", "dx", "dy"))}
    p.update({n: FAKE + (20 + i) * FAR for i, n in enumerate(("dgate", "dscale", "dshift"))})
    p.update({n: None for n in ("dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias")})
    p.update(kw)
    return ob.GatedNormGradArgs(*p.values())


def test_gated_norm_backward_refusals():
    inv, none = bb.ERR_INVALID_ARG, ob.Rows(None, 0, 0)

    def call(code, grads=None, ws=FAKE, n=1 << 40, **desc):
        refused(code, ob.bsa_gated_norm_backward, _desc(**desc), _norm_grads(**(grads or {})), ws, n, 0)

    refused(inv, ob.bsa_gated_norm_backward, _desc(), None, FAKE, 1 << 40, 0)
    for missing in ("dz", "h", "y"):
        call(inv, {missing: none})
    off = dict(pre=_norm(ob.NORM_NONE), scale=_mod(None), shift=_mod(None))
    call(inv, {"dscale": None, "dshift": None}, **off)                   # dz without a pre norm
    call(inv, {"dz": none, "dh": none, "dscale": None, "dshift": None}, **off)
    call(inv, {"dz": none, "dscale": None, "dshift": None, "dpre_weight": FAKE}, **off)
    call(inv, {"dpost_bias": FAKE})                                      # no post norm
    call(inv, gate=_mod(None))                                           # the gradient of a gate that is not there
    call(inv, scale=_mod(batch=0))                                       # ... of a broadcast scale
    call(inv, {n: none for n in ("dx", "dy")} | {"dgate": None, "dscale": None, "dshift": None})
    call(inv, {"dshift": FAKE + 2})
    call(inv, {"dx": _rows(5)})                                          # over dy
    call(inv, {"dx": _rows(3)})                                          # over y
    call(inv, {"dy": _rows(0)})                                          # over dh
    call(inv, {"dx": _rows(4, token=0)})
    need = ob.bsa_gated_norm_workspace_size(2, 16, 64)
    call(bb.ERR_WORKSPACE, ws=None)
    call(bb.ERR_WORKSPACE, ws=FAKE + 16)
    call(bb.ERR_WORKSPACE, n=need - 1)
    for bad in ((0, 1, 64), (1, 0, 64), (1, 1, 12), (1, 1, 0), (1, 1, 16384)):
        refused(bb.ERR_SHAPE, ob.bsa_gated_norm_workspace_size, *bad)


def test_helpers_refuse_host_tensors():
    plan = _plan()
    x = torch.zeros(1, 4, 2, 64)
    refused(bb.ERR_INVALID_ARG, pkg.rotary, plan, x)
    refused(bb.ERR_INVALID_ARG, pkg.rotary, plan, None)
    refused(bb.ERR_INVALID_ARG, pkg.rotary_backward, plan, x)
    refused(bb.ERR_INVALID_ARG, pkg.gated_norm, torch.zeros(1, 4, 64), pre=pkg.NormSpec("rms"))
    refused(bb.ERR_INVALID_ARG, pkg.gated_norm_backward, None, None, None)
    refused(bb.ERR_INVALID_ARG, pkg.NormSpec, "batch")


@pytest.mark.parametrize("call", ["rotary_backward", "gated_norm_backward"])
def test_workspace_is_allocated_on_the_calls_stream(monkeypatch, call):
    """with the CUDA calls faked: what a helper allocates for a call on another stream is allocated while that stream
    is current, and the launch goes to it"""
    now, allocated, launched, plan = [7], [], [], _plan()

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream, self.device = handle, device

    @contextlib.contextmanager
    def current(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    real = ob.load()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return getattr(real, name)
            return lambda *args: launched.append(args[-1]) or bb.OK

    monkeypatch.setattr(ob, "load", Lib)
    monkeypatch.setattr(ob, "_cuda_device", lambda t, what: t.device)
    monkeypatch.setattr(ob, "_current_stream", lambda index: now[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: Stream(0, device))
    monkeypatch.setattr(torch.cuda, "stream", current)
    for name in ("rotary_workspace", "gated_norm_workspace"):
        made = getattr(ob, name)
        monkeypatch.setattr(ob, name, lambda *args, made=made: allocated.append(now[-1]) or made(*args))

    def run(stream):
        if call == "rotary_backward":
            x = torch.zeros(1, 4, 2, 64)
            ob.rotary_backward(plan, x.transpose(1, 2).contiguous(), positions=torch.zeros(4, 2, dtype=torch.int32),
                               q=x, norm_eps=1e-6, q_weight=torch.ones(64), stream=stream)
        else:
            x = torch.zeros(1, 4, 64)
            ob.gated_norm_backward(x, x, x, x, gate=torch.zeros(1, 64), pre=ob.NormSpec("rms"), stream=stream)

    for stream, handle in ((None, 7), (7, 7), (40, 40), (Stream(48, torch.device("cpu")), 48), (0, 0), (1, 0)):
        run(stream)
        assert (allocated.pop(), launched.pop(), now) == (handle, handle, [7])
    refused(bb.ERR_INVALID_ARG, run, Stream(48, torch.device("meta")))


# ------------------------------------------------------------------ overlaps of every operand


def _passes(fn, *args):
    """not refused: without a device the call fails at its first CUDA call, behind all checks"""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    refused(bb.ERR_CUDA, fn, *args)


def test_rotary_outputs_over_weights_and_positions():
    inv, B, N, H, d = bb.ERR_INVALID_ARG, 2, 16, 2, 64
    dst, size = FAKE + 8 * FAR, B * N * H * d * 2

    def call(q=None, k=None, pos=FAKE + 30 * FAR, pos_batch=0):
        return _plan(), q or _heads(0, weight=FAKE + 31 * FAR), k, None, bb.BF16, B, N, pos, pos_batch, 1, 1e-6, 0

    _passes(ob.bsa_rotary, *call())
    for at in (dst - 4 * d + 16, dst, dst + size - 16):  # a weight whose end, whole or start lies in q's result
        refused(inv, ob.bsa_rotary, *call(_heads(0, weight=at)))
        refused(inv, ob.bsa_rotary, *call(k=_heads(1, weight=at)))
    for at in (dst - 4 * d, dst + size):
        _passes(ob.bsa_rotary, *call(_heads(0, weight=at)))
    for at in (dst - N * 2 * 4 + 4, dst + 64, dst + size - 4):
        refused(inv, ob.bsa_rotary, *call(pos=at))
    refused(inv, ob.bsa_rotary, *call(pos=dst - 4096, pos_batch=1024))  # the second batch's positions
    for at in (dst - N * 2 * 4, dst + size):
        _passes(ob.bsa_rotary, *call(pos=at))
    _passes(ob.bsa_rotary, *call(pos=dst - 4096, pos_batch=992))
    refused(inv, ob.bsa_rotary, *call(pos_batch=(1 << 31) + 1))
    # a weight and positions that the call does not read
    _passes(ob.bsa_rotary, _plan(), _heads(0, weight=dst), None, None, bb.BF16, B, N, FAKE + 30 * FAR, 0, 0, 0.0, 0)
    _passes(ob.bsa_rotary, _plan(), None, None, _heads(0, weight=dst), bb.BF16, B, N, dst, 0, 1, 1e-6, 0)


def test_rotary_backward_overlaps():
    inv, B, N, d = bb.ERR_INVALID_ARG, 2, 16, 64
    need = ob.bsa_rotary_workspace_size(B, N, d)
    pos, ws, dx = FAKE + 40 * FAR, FAKE + 41 * FAR, FAKE + 16 * FAR
    w = [FAKE + (42 + i) * FAR for i in range(4)]

    def call(ws=ws, k=None, **q):
        q = _grad(0, **{**dict(weight=w[0], dweight=w[1]), **q})
        k = _grad(1, **{**dict(weight=w[2], dweight=w[3]), **(k or {})})
        return _plan(), q, k, None, bb.BF16, B, N, pos, 0, 1, 1e-6, ws, need, 0

    _passes(ob.bsa_rotary_backward, *call())
    _passes(ob.bsa_rotary_backward, *call(weight=w[2]))                     # one weight for both
    _passes(ob.bsa_rotary_backward, *call(dx=FAKE + 8 * FAR))               # dx over x
    for bad in (w[0], w[2], w[3], dx, FAKE, FAKE + 8 * FAR, pos, ws, ws + need - 4):
        refused(inv, ob.bsa_rotary_backward, *call(dweight=bad))            # over a weight, the other's gradient, dx ...
    for bad in (w[1], dx, pos & ~255, FAKE, dx - need + 256):
        refused(inv, ob.bsa_rotary_backward, *call(ws=bad))
    refused(inv, ob.bsa_rotary_backward, *call(dx=w[2]))
    refused(inv, ob.bsa_rotary_backward, *call(k=dict(dweight=w[1])))
    _passes(ob.bsa_rotary_backward, *call(dweight=ws + need))               # behind what the workspace needs


def test_gated_norm_outputs_over_parameters():
    inv, B, N, C = bb.ERR_INVALID_ARG, 2, 16, 64
    p = [FAKE + (20 + i) * FAR for i in range(8)]
    h, z, size = FAKE + 2 * FAR, FAKE + 3 * FAR, B * N * C * 2

    def call(**kw):
        d = dict(post=_norm(ob.NORM_RMS, weight=p[0], bias=p[1]), pre=_norm(weight=p[2], bias=p[3]), gate=_mod(p[4]),
                 scale=_mod(p[5]), shift=_mod(p[6]))
        return _desc(**{**d, **kw}), _rows(0), _rows(1), _rows(2), _rows(3), 0

    _passes(ob.bsa_gated_norm, *call())
    for out in (h, z):
        for at in (out - 16, out, out + size - 16):
            for name in ("gate", "scale", "shift"):
                refused(inv, ob.bsa_gated_norm, *call(**{name: _mod(at)}))
            refused(inv, ob.bsa_gated_norm, *call(post=_norm(ob.NORM_RMS, weight=at)))
            refused(inv, ob.bsa_gated_norm, *call(post=_norm(ob.NORM_RMS, bias=at)))
            refused(inv, ob.bsa_gated_norm, *call(pre=_norm(weight=at)))
            refused(inv, ob.bsa_gated_norm, *call(pre=_norm(bias=at)))
        refused(inv, ob.bsa_gated_norm, *call(gate=_mod(out - 4096, batch=2048)))  # its second batch
        _passes(ob.bsa_gated_norm, *call(gate=_mod(out - 4096, batch=0)))
        _passes(ob.bsa_gated_norm, *call(gate=_mod(out + size)))
    # modulations between the rows of an output: one buffer [B][N][C + 3 * C]
    wide = dict(token=4 * C, batch=N * 4 * C)
    args = list(call(gate=_mod(h + 2 * C, batch=N * 4 * C)))
    args[3] = _rows(2, **wide)
    _passes(ob.bsa_gated_norm, *args)


def test_gated_norm_backward_overlaps():
    inv, none = bb.ERR_INVALID_ARG, ob.Rows(None, 0, 0)
    need = ob.bsa_gated_norm_workspace_size(2, 16, 64)
    p = [FAKE + (30 + i) * FAR for i in range(7)]
    ws = FAKE + 40 * FAR
    grads = {n: FAKE + (50 + i) * FAR for i, n in enumerate(("dgate", "dscale", "dshift", "dpost_weight", "dpost_bias",
                                                             "dpre_weight", "dpre_bias"))}
    desc = _desc(post=_norm(ob.NORM_RMS, weight=p[0], bias=p[1]), pre=_norm(weight=p[2], bias=p[3]), gate=_mod(p[4]),
                 scale=_mod(p[5]), shift=_mod(p[6]))

    def call(ws=ws, **kw):
        return desc, _norm_grads(**{**grads, **kw}), ws, need, 0

    _passes(ob.bsa_gated_norm_backward, *call())
    _passes(ob.bsa_gated_norm_backward, *call(dx=_rows(0), dy=_rows(1)))
    rows = [FAKE + i * FAR for i in range(6)]
    for name, own in grads.items():
        others = [g for n, g in grads.items() if n != name]
        for at in p + rows + others + [ws, ws + need - 16]:
            refused(inv, ob.bsa_gated_norm_backward, *call(**{name: at}))
        _passes(ob.bsa_gated_norm_backward, *call(**{name: ws + need}))
    for at in p + rows + list(grads.values()):
        refused(inv, ob.bsa_gated_norm_backward, *call(ws=at))
    for at in p:
        refused(inv, ob.bsa_gated_norm_backward, *call(dx=_rows(0, ptr=at)))
        refused(inv, ob.bsa_gated_norm_backward, *call(dy=_rows(0, ptr=at)))
    # without a gradient that needs it the workspace is not looked at
    alone = {n: None for n in grads}
    _passes(ob.bsa_gated_norm_backward, *call(ws=rows[4], **alone))
    _passes(ob.bsa_gated_norm_backward, *call(ws=rows[4], dx=none, **alone))


def test_weight_without_the_norm_is_refused(monkeypatch):
    monkeypatch.setattr(ob, "_cuda_device", lambda t, what: t.device)
    x, pos, w = torch.zeros(1, 4, 2, 64), torch.zeros(4, 2, dtype=torch.int32), torch.ones(64)
    for fn, t in ((pkg.rotary, x), (pkg.rotary_backward, x.transpose(1, 2))):
        for weights in (dict(q_weight=w), dict(k_weight=w)):
            with pytest.raises(bb.BsaError, match="norm_eps") as e:
                fn(_plan(), t, positions=pos, **weights)
            assert e.value.code == bb.ERR_INVALID_ARG


def test_gradients_that_would_vanish_are_refused(monkeypatch):
    """a tensor that requires a gradient, each operand in turn, while gradients are recorded"""
    monkeypatch.setattr(ob, "_cuda_device", lambda t, what: t.device)
    heads, rows, plan = torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 64), _plan()

    def back(**t):
        return pkg.rotary_backward(plan, t.pop("dq"), t.pop("dk"), t.pop("dv"), **t)

    def norms(t):
        w = {n: t.pop(n) for n in ("post_w", "post_b", "pre_w", "pre_b")}
        return dict(post=ob.NormSpec("rms", w["post_w"], w["post_b"]), pre=ob.NormSpec("layer", w["pre_w"], w["pre_b"]))

    pos, w64 = torch.zeros(4, 2, dtype=torch.int32), torch.ones(64)
    turn = dict(positions=pos, q_weight=w64, k_weight=w64)
    dy = heads.transpose(1, 2).contiguous()
    mods = {n: torch.zeros(1, 64) for n in ("gate", "scale", "shift")}
    params = {n: w64 for n in ("post_w", "post_b", "pre_w", "pre_b")}
    calls = [(lambda **t: pkg.rotary(plan, t.pop("q"), t.pop("k"), t.pop("v"), norm_eps=1e-6, **t),
              dict(q=heads, k=heads, v=heads, **turn)),
             (lambda **t: back(norm_eps=1e-6, **t), dict(dq=dy, dk=dy, dv=dy, q=heads, k=heads, **turn)),
             (lambda **t: pkg.gated_norm(t.pop("x"), t.pop("y"), **norms(t), **t), dict(x=rows, y=rows, **mods, **params)),
             (lambda **t: pkg.gated_norm_backward(t.pop("dh"), t.pop("dz"), t.pop("h"), t.pop("y"), **norms(t), **t),
              dict(dh=rows, dz=rows, h=rows, y=rows, **mods, **params))]

    class Reached(Exception):
        pass

    def launch(*args):
        raise Reached

    monkeypatch.setattr(ob, "_run", launch)
    for fn, tensors in calls:
        with pytest.raises(Reached):
            fn(**tensors)
        for name, t in tensors.items():
            if name == "positions":
                continue
            wanted = dict(tensors, **{name: t.clone().requires_grad_()})
            with pytest.raises(bb.BsaError, match="gradient") as e:
                fn(**wanted)
            assert e.value.code == bb.ERR_INVALID_ARG, name
            with torch.no_grad(), pytest.raises(Reached):
                fn(**wanted)
