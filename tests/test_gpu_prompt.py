"""bsa_prompt_attention against its 64-bit form, and the four calls together."""
import concurrent.futures
import os
import subprocess
import sys

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


def test_cut_sequences_of_equal_length_give_the_same_bits():
    """few items, cut evenly over the CTAs: where the cuts fall does not vary from call to call"""
    g = gen(10)
    cu_q, cu_k = starts([64] * 5), starts([4000] * 5)
    q, k, v = draw(g, cu_q[-1], 4, 64), draw(g, cu_k[-1], 2, 64), draw(g, cu_k[-1], 2, 64)
    a = check(q, k, v, cu_q, cu_k, False)
    for _ in range(10):
        b = pkg.prompt_attention(q, k, v, ints(cu_q), ints(cu_k), causal=False)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


LONG = [
    # many items, taken from the counter; more sequences than a plan holds in shared memory; mixed heads
    (4, 4, 128, [2500, 1, 900, 2500, 130], None, True),
    (2, 1, 64, [5 + i * 37 % 90 for i in range(300)], [i * 11 % 700 for i in range(300)], True),
    (6, 2, 128, [1200, 64], [300, 5000], True),
    (8, 8, 64, [1500, 1500], None, False),
]


@pytest.mark.parametrize("H,Hk,d,new,past,causal", LONG)
def test_longer_prompts(H, Hk, d, new, past, causal):
    g = gen(11)
    cu_q = starts(new)
    cu_k = cu_q if past is None else starts([a + b for a, b in zip(new, past)])
    q, k, v = draw(g, cu_q[-1], H, d), draw(g, cu_k[-1], Hk, d), draw(g, cu_k[-1], Hk, d)
    check(q, k, v, cu_q, cu_k, causal)


@pytest.mark.parametrize("seed", range(6))
def test_short_items_of_every_kind(seed):
    """hundreds of tiles of one to three steps, one after another in a CTA, empty ones among them"""
    g = gen(20 + seed)
    r = torch.Generator().manual_seed(seed)
    n = 60
    new = torch.randint(0, 300, (n,), generator=r).tolist()
    keys = [max(0, a + int(x)) for a, x in zip(new, torch.randint(-200, 200, (n,), generator=r))]
    cu_q, cu_k = starts(new), starts(keys)
    H, Hk, d = [(6, 2, 128), (4, 4, 64), (8, 1, 128), (3, 3, 128), (16, 8, 64), (5, 1, 64)][seed]
    q, k, v = draw(g, cu_q[-1], H, d), draw(g, cu_k[-1], Hk, d), draw(g, cu_k[-1], Hk, d)
    check(q, k, v, cu_q, cu_k, seed % 2 == 0)


# ------------------------------------------------------------------ the four calls together


def new_tokens(g, n, H, Hk, d):
    x = draw(g, n, H + 2 * Hk, d)
    return x.split([H, Hk, Hk], dim=1)


@pytest.mark.parametrize("kind,H,Hk,d,page", [("bf16", 6, 2, 128, 16), ("e4m3", 8, 8, 64, 64), ("e4m3", 12, 4, 128, 32)])
def test_prompts_then_a_later_chunk_then_tokens_one_by_one(kind, H, Hk, d, page):
    """as a model that answers uses them: prompts attend to themselves and go into the cache; a later chunk of each reads the
    cache back and attends to all of it; then tokens come one by one. Every result against the 64-bit form over what
    the cache holds."""
    g = gen(30)
    prompts, chunks, steps = [100, 1, 333], [20, 65, 7], 5
    B, most = 3, 512
    table = torch.randperm(B * (most // page), generator=g, device=DEV).to(torch.int32).view(B, most // page)
    cache = pkg.kv_cache(B * (most // page), page, Hk, d, kind, DEV)
    ws = pkg.cache_workspace(sum(prompts), B, H, Hk, d, DEV)
    held = [0] * B
    keys, values = ([torch.empty(0, Hk, d, dtype=BF16, device=DEV) for _ in range(B)] for _ in range(2))

    def append(new, k, v):
        at = 0
        for b, n in enumerate(new):
            for x, seen in ((k, keys), (v, values)):
                fresh = x[at:at + n]
                seen[b] = torch.cat((seen[b], fresh if kind == "bf16" else ref.e4m3_rows(fresh)[0].to(BF16)))
            at += n
            held[b] += n

    q, k, v = new_tokens(g, sum(prompts), H, Hk, d)
    check(q, k, v, starts(prompts), starts(prompts), True, ws=ws)
    append(prompts, k, v)
    pkg.cache_write(cache, k, v, table, ints(held), ints(starts(prompts)), ws=ws)

    q, k, v = new_tokens(g, sum(chunks), H, Hk, d)
    append(chunks, k, v)
    pkg.cache_write(cache, k, v, table, ints(held), ints(starts(chunks)), ws=ws)
    all_k, all_v = pkg.cache_read(cache, table, ints(starts(held)), sum(held), ws=ws)
    assert torch.equal(all_k, torch.cat(keys)) and torch.equal(all_v, torch.cat(values))
    check(q, all_k, all_v, starts(chunks), starts(held), True, ws=ws)

    for _ in range(steps):
        q, k, v = new_tokens(g, B, H, Hk, d)
        append([1] * B, k, v)
        pkg.cache_write(cache, k, v, table, ints(held), ws=ws)
        out, lse = pkg.cache_attention(q, cache, table, ints(held), ws=ws)
        for b in range(B):
            for h in range(H):
                kh = h // (H // Hk)
                see = torch.ones(1, held[b], dtype=torch.bool, device=DEV)
                o, bo, l, bl = ref.attention(q[b, h][None], keys[b][:, kh], values[b][:, kh], see, d ** -0.5, half_weights=kind == "e4m3")
                ref.within(out[b, h][None], o, bo, "O")
                ref.within(lse[b, h][None], l, bl, "LSE")


def test_rotary_outputs_are_inputs():
    """bsa_rotary's q, k, v [1, H, T, d] as packed views, and the block-sparse forward with every block over the same tokens"""
    g = gen(31)
    T, H, d = 512, 4, 128
    plan = pkg.rotary_plan(d, axis_dims=[d])
    pos = torch.arange(T, dtype=torch.int32, device=DEV)[:, None]
    q, k, v = pkg.rotary(plan, *(draw(g, 1, T, H, d) for _ in range(3)), positions=pos)
    pq, pk, pv = (x[0].transpose(0, 1) for x in (q, k, v))
    out, lse = check(pq, pk, pv, [0, T], [0, T], False)
    nb = T // 128
    ones = torch.full((nb,), -1, dtype=torch.int32, device=DEV)
    full = bb.build_mask(None, None, block=128, spec=bb.explicit_spec(ones, broadcast_bh=True), shape=q.shape)
    O, L = bb.forward(q, k, v, full)
    o, bo, l, bl = expected(pq, pk, pv, [0, T], [0, T], False, d ** -0.5)
    ref.within(O[0].transpose(0, 1), o, bo, "block-sparse O")
    ref.within(L[0], l, bl, "block-sparse LSE")


class Loop:
    """one sequence of tokens through the cache, with everything allocated: what a captured decoding step holds"""

    def __init__(self, g, kind="e4m3", B=4, H=8, Hk=2, d=128, page=32, most=256):
        self.q, self.k, self.v = new_tokens(g, B, H, Hk, d)
        self.table = torch.randperm(B * (most // page), generator=g, device=DEV).to(torch.int32).view(B, most // page)
        self.cache = pkg.kv_cache(B * (most // page), page, Hk, d, kind, DEV)
        self.held = ints([100, 1, 37, 200])
        past_k, past_v = draw(g, 338, Hk, d), draw(g, 338, Hk, d)
        pkg.cache_write(self.cache, past_k, past_v, self.table, self.held, ints(starts([100, 1, 37, 200])))
        self.out, self.lse = torch.empty(B, H, d, dtype=BF16, device=DEV), torch.empty(B, H, device=DEV)
        self.args = dict(H=H, Hk=Hk, d=d)

    def step(self, ws, stream=None):
        self.held += 1
        pkg.cache_write(self.cache, self.k, self.v, self.table, self.held, ws=ws, check=False)
        pkg.cache_attention(self.q, self.cache, self.table, self.held, out=self.out, lse=self.lse, ws=ws, check=False)

    def expected(self):
        fresh = pkg.cache_workspace(4, 4, self.args["H"], self.args["Hk"], self.args["d"], DEV)
        return pkg.cache_attention(self.q, self.cache, self.table, self.held, ws=fresh)


def test_a_captured_step_replayed_and_two_graphs_with_one_workspace():
    g = gen(32)
    a, b = Loop(g), Loop(g, kind="bf16")
    ws = pkg.cache_workspace(4, 4, 8, 2, 128, DEV)
    graphs = []
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for x in (a, b):
            x.step(ws)  # a first call outside
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                x.step(ws)
            graphs.append(graph)
        for _ in range(3):
            for graph in graphs:
                graph.replay()
        stream.synchronize()
    pkg.cache_check(ws)
    for x in (a, b):
        assert x.held.tolist() == [104, 5, 41, 204]
        o, l = x.expected()
        assert torch.equal(x.out, o) and torch.equal(x.lse, l)


def test_captured_prompts_replayed_with_other_lengths():
    """the lengths live on the device: a captured call follows them"""
    g = gen(33)
    T, H, Hk, d = 900, 4, 2, 64
    q, k, v = new_tokens(g, T, H, Hk, d)
    cu = ints([0, 300, 300, 900])
    out, lse = torch.empty(T, H, d, dtype=BF16, device=DEV), torch.empty(H, T, device=DEV)
    ws = pkg.cache_workspace(T, 3, H, Hk, d, DEV)
    pkg.prompt_attention(q, k, v, cu, out=out, lse=lse, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.prompt_attention(q, k, v, cu, out=out, lse=lse, ws=ws, check=False)
    for lens in ([0, 1, 450, 900], [0, 900, 900, 900], [0, 128, 640, 900]):
        cu.copy_(ints(lens))
        graph.replay()
        torch.cuda.synchronize()
        o, bo, l, bl = expected(q, k, v, lens, lens, True, d ** -0.5)
        ref.within(out, o, bo, "O")
        ref.within(lse, l, bl, "LSE")


def test_two_streams_with_a_workspace_each():
    g = gen(34)
    loops = [Loop(g), Loop(g, kind="bf16")]
    streams = [torch.cuda.Stream() for _ in loops]
    torch.cuda.synchronize()
    spaces = [pkg.cache_workspace(4, 4, 8, 2, 128, DEV) for _ in loops]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s, ws in zip(loops, streams, spaces):
            with torch.cuda.stream(s):
                x.step(ws)
    torch.cuda.synchronize()
    for x, ws in zip(loops, spaces):
        pkg.cache_check(ws)
        o, l = x.expected()
        assert torch.equal(x.out, o) and torch.equal(x.lse, l)


def test_the_stream_argument_orders_the_calls():
    g = gen(35)
    q, k, v = new_tokens(g, 500, 4, 2, 128)
    cu = ints([0, 500])
    want = pkg.prompt_attention(q, k, v, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pkg.prompt_attention(q, k, v, cu, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("H,Hk,d", [(4, 4, 64), (6, 2, 128), (5, 1, 128)])
@pytest.mark.parametrize("bad", [INF, float("nan"), 1e30])
def test_queries_of_others_in_the_same_tile_do_not_reach(H, Hk, d, bad):
    """a tile's rows behind its sequence hold the next one's queries, which may be anything; cut and whole tiles"""
    g = gen(12)
    cu_q, cu_k = starts([50, 60, 200]), starts([50, 5000, 200])
    q, k, v = draw(g, 310, H, d), draw(g, cu_k[-1], Hk, d), draw(g, cu_k[-1], Hk, d)
    clean = pkg.prompt_attention(q, k, v, ints(cu_q), ints(cu_k))
    q[110:] = bad
    out, lse = pkg.prompt_attention(q, k, v, ints(cu_q), ints(cu_k))
    assert torch.equal(out[:110], clean[0][:110]) and torch.equal(lse[:, :110], clean[1][:, :110])
    assert clean[0].isfinite().all()


@pytest.mark.parametrize("causal", [True, False])
def test_infinite_scores(causal):
    """a score of +inf is NaN in the results as in the formula, one of -inf is a weight of zero, in any step"""
    g = gen(13)
    cu = starts([600])
    q, k, v = (draw(g, 600, 2, 128).abs() for _ in range(3))
    k[400, 0, 7] = -INF
    k[500, 1, 7] = INF
    out, lse = pkg.prompt_attention(q, k, v, ints(cu), causal=causal)
    first = 500 if causal else 0
    assert out[first:, 1].isnan().all() and lse[1, first:].isnan().all()
    keep = torch.arange(600, device=DEV) != 400
    k2, v2 = k[keep][:, :1].contiguous(), v[keep][:, :1].contiguous()
    # without key 400: rows behind it see the same keys but that one
    if causal:
        o, bo, l, bl = expected(q[:400, :1].contiguous(), k[:400, :1].contiguous(), v[:400, :1].contiguous(), starts([400]), starts([400]), True, 128 ** -0.5)
        ref.within(out[:400, :1], o, bo, "O")
        o, bo, l, bl = expected(q[401:, :1].contiguous(), k2, v2, starts([199]), starts([599]), True, 128 ** -0.5)
        ref.within(out[401:, :1], o, bo, "O")
    else:
        o, bo, l, bl = expected(q[:, :1].contiguous(), k2, v2, starts([600]), starts([599]), False, 128 ** -0.5)
        ref.within(out[:, :1], o, bo, "O")


def test_one_workspace_for_calls_of_every_kind():
    """planned by a launch of its own or not, cut or not, and tokens between: each call leaves the workspace as the next needs it"""
    g = gen(36)
    calls = []
    for H, Hk, d, new, past in ((4, 2, 128, [40] * 40, [900] + [0] * 39), (4, 4, 64, [300, 20], None), (8, 2, 128, [16], [9000]),
                                (2, 1, 64, [5] * 50, None), (6, 2, 128, [700, 1, 64], [2000, 0, 5])):
        cu_q, cu_k = starts(new), starts([n + p for n, p in zip(new, past or [0] * len(new))])
        q, k, v = draw(g, cu_q[-1], H, d), draw(g, cu_k[-1], Hk, d), draw(g, cu_k[-1], Hk, d)
        calls.append((q, k, v, ints(cu_q), ints(cu_k)))
    loop = Loop(g)
    ws = pkg.cache_workspace(2000, 50, 8, 8, 128, DEV)
    want = [pkg.prompt_attention(*c) for c in calls]
    for order in (range(5), (3, 1, 4, 0, 2), (2, 2, 1, 3, 4)):
        for i in order:
            got = pkg.prompt_attention(*calls[i], ws=ws)
            assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])
            loop.step(ws)
            o, l = loop.expected()
            assert torch.equal(loop.out, o) and torch.equal(loop.lse, l)
    pkg.cache_check(ws)


def test_two_threads_at_once():
    g = gen(37)
    calls = []
    for H, Hk, d, new in ((4, 2, 128, [700, 60]), (4, 4, 64, [1500])):
        cu = starts(new)
        calls.append((draw(g, cu[-1], H, d), draw(g, cu[-1], Hk, d), draw(g, cu[-1], Hk, d), ints(cu)))
    want = [pkg.prompt_attention(*c) for c in calls]
    torch.cuda.synchronize()

    def work(i):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            runs = [pkg.prompt_attention(*calls[i]) for _ in range(20)]
        side.synchronize()
        return all(torch.equal(a, b) for run in runs for a, b in zip(run, want[i]))

    with concurrent.futures.ThreadPoolExecutor(2) as pool:
        assert all(pool.map(work, range(2)))


FIRST_CALL = """
import torch
import block_sparse_attention_mean_gb300 as pkg
g = torch.Generator("cuda").manual_seed(1)
def draw(*s): return torch.randn(*s, generator=g, device="cuda").bfloat16()
def ints(x): return torch.tensor(x, dtype=torch.int32, device="cuda")
q, k, v, cu, held, table = draw(300, 4, 64), draw(300, 2, 64), draw(300, 2, 64), ints([0, 100, 300]), ints([100, 200]), ints([list(range(4)), list(range(4, 8))])
ws, cache, q1 = pkg.cache_workspace(300, 2, 4, 2, 64), pkg.kv_cache(8, 64, 2, 64, "e4m3"), draw(2, 4, 64)
def step():
    pkg.cache_write(cache, k, v, table, held, cu, ws=ws, check=False)
    return (*pkg.prompt_attention(q, k, v, cu, ws=ws, check=False), *pkg.cache_attention(q1, cache, table, held, ws=ws, check=False),
            *pkg.cache_read(cache, table, cu, 300, ws=ws, check=False))
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
pkg.cache_check(ws)
print("same")
"""


def test_first_call_of_a_process_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.split() == ["same"], r.stdout + r.stderr


@pytest.mark.parametrize("H,Hk,d,B,most,past", [(2, 1, 64, 3000, 9, 0), (2, 2, 128, 1100, 3, 40), (3, 1, 64, 33, 200, 2000)])
def test_many_sequences(H, Hk, d, B, most, past):
    """more than a plan's threads, and a few more than a warp's lanes; some without queries, some without keys"""
    g = gen(38)
    new = torch.randint(0, most, (B,), generator=g, device=DEV).tolist()
    old = torch.randint(0, past + 1, (B,), generator=g, device=DEV).tolist()
    old[1::7] = [-n for n in new[1::7]]  # no keys
    cu_q, cu_k = starts(new), starts([n + p for n, p in zip(new, old)])
    q, k, v = draw(g, cu_q[-1], H, d), draw(g, cu_k[-1], Hk, d), draw(g, cu_k[-1], Hk, d)
    out, lse = pkg.prompt_attention(q, k, v, ints(cu_q), ints(cu_k))
    some = torch.randperm(B, generator=g, device=DEV)[:200].tolist() + [0, 1, B - 1]
    for b in some:
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        o, bo, l, bl = expected(q[rows], k[keys], v[keys], [0, new[b]], [0, new[b] + old[b]], True, d ** -0.5)
        ref.within(out[rows], o, bo, "O")
        ref.within(lse[:, rows], l, bl, "LSE")


@pytest.mark.parametrize("H,Hk,d,new", [(128, 1, 64, [3, 1, 260]), (64, 1, 128, [5, 130]), (100, 2, 64, [70])])
def test_many_heads_share_a_key_head(H, Hk, d, new):
    g = gen(39)
    cu = starts(new)
    check(draw(g, cu[-1], H, d), draw(g, cu[-1], Hk, d), draw(g, cu[-1], Hk, d), cu, cu, True)


@pytest.mark.parametrize("H,Hk,d,causal", [(48, 16, 128, True), (40, 40, 64, True), (64, 8, 64, False), (21, 7, 128, False)])
def test_short_items_of_few_sequences(H, Hk, d, causal):
    """as above where each CTA plans for itself: up to 32 sequences, ten tiles of one to four steps a CTA"""
    g = gen(40)
    new = torch.randint(0, 500, (32,), generator=g, device=DEV).tolist()
    keys = [max(0, a + x) for a, x in zip(new, torch.randint(-300, 100, (32,), generator=g, device=DEV).tolist())]
    cu_q, cu_k = starts(new), starts(keys)
    check(draw(g, cu_q[-1], H, d), draw(g, cu_k[-1], Hk, d), draw(g, cu_k[-1], Hk, d), cu_q, cu_k, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,first", [(64, 140), (128, 128), (128, 300), (64, 1)])
def test_low_scores_behind_infinite_ones(d, first, causal):
    """the first keys have scores of -inf, the others' lie far below zero: their weights count all the same"""
    g = gen(14)
    n = 600
    q, k, v = (draw(g, n, 2, d) for _ in range(3))
    q[..., 0], k[..., 0] = 16.0, -100.0     # scores of about -140 and -200
    k[:first, 0, 0] = -INF
    out, lse = pkg.prompt_attention(q, k, v, ints([0, n]), causal=causal)
    rest = n - first
    from_row = first if causal else 0
    o, bo, l, bl = expected(q[from_row:, :1], k[first:, :1], v[first:, :1], [0, n - from_row], [0, rest], causal, d ** -0.5)
    ref.within(out[from_row:, :1], o, bo, "O")
    ref.within(lse[:1, from_row:], l, bl, "LSE")
    o, bo, l, bl = expected(q[:, 1:], k[:, 1:], v[:, 1:], [0, n], [0, n], causal, d ** -0.5)
    ref.within(out[:, 1:], o, bo, "O")
    ref.within(lse[1:], l, bl, "LSE")
    if causal:  # they see nothing else
        assert (out[:first, 0] == 0).all() and (lse[0, :first] == -INF).all()
