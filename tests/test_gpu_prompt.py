"""bsa_prompt_attention against its 64-bit form, and the four calls together."""
import pytest
import torch

import block_sparse_attention_mean_gb300 as pkg
from block_sparse_attention_mean_gb300 import binding as bb
from block_sparse_attention_mean_gb300 import build as bbuild
from block_sparse_attention_mean_gb300 import cache_binding as cb
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bbuild.build()
    cb.load()


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return at


def draw(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(BF16)


def expected(q, k, v, cu_q, cu_k, causal, scale):
    T, H, d = q.shape
    g = H // k.shape[1]
    o, bo = (torch.zeros(T, H, d, dtype=torch.float64, device=DEV) for _ in range(2))
    lse, bl = (torch.zeros(H, T, dtype=torch.float64, device=DEV) for _ in range(2))
    for b in range(len(cu_q) - 1):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        see = ref.visible(cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b], causal, DEV)
        for h in range(H):
            o[rows, h], bo[rows, h], lse[h, rows], bl[h, rows] = ref.attention(q[rows, h], k[keys, h // g], v[keys, h // g], see, scale)
    return o, bo, lse, bl


def check(q, k, v, cu_q, cu_k, causal, scale=None, **kw):
    out, lse = pkg.prompt_attention(q, k, v, ints(cu_q), None if cu_k is cu_q else ints(cu_k), causal=causal,
                                    scale=0.0 if scale is None else scale, **kw)
    o, bo, l, bl = expected(q, k, v, cu_q, cu_k, causal, q.shape[2] ** -0.5 if scale is None else scale)
    rows = slice(cu_q[0], cu_q[-1])
    ref.within(out[rows], o[rows], bo[rows], "O")
    ref.within(lse[:, rows], l[:, rows], bl[:, rows], "LSE")
    return out, lse


CASES = [
    # H, Hk, d, query lengths, earlier keys (None: none)
    (1, 1, 64, [1], None),
    (1, 1, 128, [1], None),
    (2, 2, 128, [127, 128, 129], None),
    (2, 2, 64, [255, 256, 257, 1, 0, 64], None),
    (3, 1, 128, [1, 42, 43, 200], None),          # 42 tokens a tile, two rows of it unused
    (5, 1, 64, [7, 300], None),
    (8, 2, 128, [33, 0, 500], [1, 20, 3]),
    (16, 1, 64, [9, 100], [300, 0]),
    (128, 1, 64, [3], [130]),                     # one token a tile
    (65, 1, 128, [2, 5], None),
    (7, 7, 64, [1, 1, 1, 2], [0, 127, 128, 255]),
    (4, 4, 128, [700], [13]),
    (2, 1, 64, [1], [5000]),                      # few rows over many keys: parts, joined
    (4, 1, 128, [40], [9000]),
    (2, 2, 128, [300, 17], [2000, 4100]),
    (1, 1, 64, [1500], None),
    (24, 8, 128, [130, 77, 260], None),
    (2, 2, 64, [20] * 50, [i * 7 % 40 for i in range(50)]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hk,d,new,past", CASES)
def test_prompt_attention(H, Hk, d, new, past, causal):
    g = gen(1)
    cu_q = starts(new)
    cu_k = cu_q if past is None else starts([a + b for a, b in zip(new, past)])
    q, k, v = draw(g, cu_q[-1], H, d), draw(g, cu_k[-1], Hk, d), draw(g, cu_k[-1], Hk, d)
    check(q, k, v, cu_q, cu_k, causal)


@pytest.mark.parametrize("causal", [True, False])
def test_more_queries_than_keys(causal):
    g = gen(2)
    cu_q, cu_k = starts([200, 5, 130, 40]), starts([70, 0, 129, 1])
    q, k, v = draw(g, cu_q[-1], 4, 64), draw(g, cu_k[-1], 2, 64), draw(g, cu_k[-1], 2, 64)
    out, lse = check(q, k, v, cu_q, cu_k, causal)
    if causal:
        assert (out[:130] == 0).all() and (lse[:, :130] == -INF).all()
    assert (out[200:205] == 0).all() and (lse[:, 200:205] == -INF).all()


def test_no_keys_and_no_queries():
    g = gen(3)
    q, none = draw(g, 5, 2, 64), draw(g, 0, 2, 64)
    out, lse = pkg.prompt_attention(q, none, none, ints([0, 5]), ints([0, 0]))
    assert (out == 0).all() and (lse == -INF).all()
    out, lse = pkg.prompt_attention(none, q, q, ints([0, 0]), ints([0, 5]))
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_views_scale_and_spread_scores(d):
    """views of a fused projection, heads first, and scores of some tens (the maximum is raised in many steps)"""
    g = gen(4)
    cu = starts([600, 90])
    x = draw(g, cu[-1], 8, d)
    q, k, v = x.split([4, 2, 2], dim=1)
    check(q, k, v, cu, cu, True, scale=0.9 * 8 / d ** 0.5, out=torch.empty(cu[-1], 9, d, dtype=BF16, device=DEV)[:, 3:7])
    q, k, v = (draw(g, h, cu[-1], d).transpose(0, 1) for h in (4, 2, 2))
    check(q * 3, k * 2, v, cu, cu, True, out=torch.empty(4, cu[-1], d, dtype=BF16, device=DEV).transpose(0, 1))
    ramp = torch.linspace(-30, 30, cu[-1], device=DEV)[:, None, None]
    check(q, (k + ramp).to(BF16).contiguous(), v, cu, cu, True)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_of_no_sequence_are_neither_read_nor_written(causal):
    g = gen(5)
    cu_q, cu_k = starts([100, 30], 7), starts([150, 70], 3)
    q, k, v = draw(g, 160, 4, 128), draw(g, 300, 2, 128), draw(g, 300, 2, 128)
    for x, cu in ((q, cu_q), (k, cu_k), (v, cu_k)):
        x[:cu[0]] = float("nan")
        x[cu[-1]:] = INF
    out = torch.full((160, 4, 128), 5.0, dtype=BF16, device=DEV)
    lse = torch.full((4, 160), 5.0, device=DEV)
    check(q, k, v, cu_q, cu_k, causal, out=out, lse=lse)
    for rows in (slice(0, 7), slice(137, 160)):
        assert (out[rows] == 5).all() and (lse[:, rows] == 5).all()


@pytest.mark.parametrize("past", [0, 1000])
def test_what_is_not_seen_does_not_reach(past):
    """NaN and infinities in a key or a value reach the queries that see it, and no others, within a tile too"""
    g = gen(6)
    cu_q, cu_k = starts([300, 40]), starts([300 + past, 40])
    q, k, v = draw(g, 340, 2, 64), draw(g, 340 + past, 2, 64), draw(g, 340 + past, 2, 64)
    clean = pkg.prompt_attention(q, k, v, ints(cu_q), ints(cu_k))
    v[past + 290, 0, 5] = INF
    v[past + 295, 0, 5] = -INF
    v[past + 200, 0, 9] = float("nan")
    v[past + 260, 1] = INF
    k[past + 299, 0, 3] = float("nan")
    out, lse = pkg.prompt_attention(q, k, v, ints(cu_q), ints(cu_k))
    o, bo, l, bl = expected(q, k, v, cu_q, cu_k, True, 0.125)
    ref.within(out[:299], o[:299], bo[:299], "O")
    assert torch.equal(out[:200], clean[0][:200]) and torch.equal(out[300:], clean[0][300:])
    assert out[299, 0].isnan().all() and lse[0, 299].isnan() and torch.equal(lse[:, :299], clean[1][:, :299])
    assert torch.equal(lse[:, 300:], clean[1][:, 300:])


def test_the_same_call_gives_the_same_bits():
    g = gen(7)
    cu_q, cu_k = starts([300, 1, 64]), starts([3000, 5000, 64])
    q, k, v = draw(g, cu_q[-1], 4, 128), draw(g, cu_k[-1], 2, 128), draw(g, cu_k[-1], 2, 128)
    ws = pkg.cache_workspace(cu_q[-1], 3, 4, 2, 128, DEV)
    a = pkg.prompt_attention(q, k, v, ints(cu_q), ints(cu_k), ws=ws)
    for _ in range(5):
        b = pkg.prompt_attention(q, k, v, ints(cu_q), ints(cu_k), ws=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_malformed_sequences_are_reported():
    g = gen(8)
    q, k, v = draw(g, 100, 2, 64), draw(g, 100, 2, 64), draw(g, 100, 2, 64)
    ws = pkg.cache_workspace(100, 6, 2, 2, 64, DEV)
    for cu_q, cu_k in (([0, 101], [0, 100]), ([0, 50, 40], [0, 50, 100]), ([-1, 50], [0, 50]), ([0, 50], [0, 101]), ([0, 50], [10, 5])):
        with pytest.raises(bb.BsaError) as e:
            pkg.prompt_attention(q, k, v, ints(cu_q), ints(cu_k), ws=ws)
        assert e.value.code == bb.ERR_INVALID_ARG
        pkg.cache_check(ws)
    # one that is well formed beside one that is not gets its result, the other's rows stay
    out = torch.full((100, 2, 64), 5.0, dtype=BF16, device=DEV)
    out, lse = pkg.prompt_attention(q, k, v, ints([0, 40, 90]), ints([0, 40, 101]), ws=ws, check=False, out=out)
    o, bo, l, bl = expected(q, k, v, [0, 40], [0, 40], True, 0.125)
    ref.within(out[:40], o[:40], bo[:40], "O")
    assert (out[40:] == 5).all()
    with pytest.raises(bb.BsaError):
        pkg.cache_check(ws)
    # overlapping sequences of more tokens than there are
    ws = pkg.cache_workspace(100, 4001, 2, 2, 64, DEV)
    with pytest.raises(bb.BsaError):
        pkg.prompt_attention(q, k, v, ints([0, 100] * 2001), ints([0, 100] * 2001), ws=ws)


def test_a_wait_that_runs_out_is_reported():
    """nothing is loaded: the first waits give up after their limit, the call returns, and the next one is right"""
    g = gen(9)
    cu = starts([2000, 300])
    q, k, v = draw(g, cu[-1], 4, 128), draw(g, cu[-1], 4, 128), draw(g, cu[-1], 4, 128)
    ws = pkg.cache_workspace(cu[-1], 2, 4, 4, 128, DEV)
    a = pkg.prompt_attention(q, k, v, ints(cu), ws=ws)
    bb.bsa_debug_config(bb.DBG_STALL, 2_000_000)
    try:
        with pytest.raises(bb.BsaError) as e:
            pkg.prompt_attention(q, k, v, ints(cu), ws=ws)
        assert e.value.code == bb.ERR_TIMEOUT
    finally:
        bb.bsa_debug_config(0, 0)
    b = pkg.prompt_attention(q, k, v, ints(cu), ws=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
