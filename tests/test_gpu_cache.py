"""The cache's rows and attention over it (bsa_cache_write, bsa_cache_read, bsa_cache_attention) against their 64-bit forms."""
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


def starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return ints(at)


def paged(g, held, page, spare=3, width=None):
    """(table, pages in all): the sequences' pages in random order; entries behind a sequence's last page are not pages"""
    counts = [-(-n // page) for n in held]
    order = torch.randperm(sum(counts) + spare, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(held), width or max(1, max(counts))), -7, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(counts) + spare


def draw(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def rows(g, T, H, d):
    """keys and values [T, H, d] whose rows differ in size"""
    return tuple((draw(g, T, H, d) * torch.exp(draw(g, T, H, 1))).to(BF16) for _ in range(2))


def filled(g, n_pages, page, Hk, d, kind):
    """a cache of random contents, and its values [pages, Hk, page, d] in 64 bits"""
    k, v = rows(g, n_pages * Hk * page, 1, d)
    cache = pkg.kv_cache(n_pages, page, Hk, d, kind, DEV)
    values = []
    for x, data, exps in ((k, cache.k, cache.k_exp), (v, cache.v, cache.v_exp)):
        x = x.view(n_pages, Hk, page, d)
        if kind == "bf16":
            data.copy_(x)
            values.append(x.double())
        else:
            held, e = ref.e4m3_rows(x)
            unit = ((e.long() - 127 + 1023) << 52).view(torch.float64)[..., None]
            data.copy_((held / unit).float())
            exps.copy_(e)
            values.append(held)
    return cache, values


def sequence(values, table, b, n, page):
    """the first n tokens of sequence b: [n, Hk, d]"""
    ids = table[b, : -(-n // page)].long()
    return values[ids].transpose(1, 2).flatten(0, 1)[:n]


# ------------------------------------------------------------------ rows


ROWS = [
    # kind, page, Hk, d, tokens held before, new tokens
    ("bf16", 16, 1, 64, [0], [1]),
    ("e4m3", 16, 1, 128, [15], [1]),
    ("bf16", 64, 8, 128, [0, 63, 64, 130], [65, 1, 64, 3]),
    ("e4m3", 32, 5, 64, [0, 31, 7, 100], [33, 2, 0, 200]),
    ("e4m3", 128, 24, 128, [0, 500], [300, 129]),
    ("bf16", 256, 3, 64, [255, 0, 1], [2, 0, 511]),
    ("e4m3", 64, 2, 128, [10] * 70, [i % 4 for i in range(70)]),
]


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("kind,page,Hk,d,past,new", ROWS)
def test_write_then_read(kind, page, Hk, d, past, new, fused):
    g = gen(1)
    held = [a + b for a, b in zip(past, new)]
    table, n_pages = paged(g, held, page)
    cache, values = filled(g, n_pages, page, Hk, d, kind)
    T = sum(new)
    k, v = rows(g, T, Hk, d)
    k[T // 2, 0] = 0
    if fused:
        k, v = torch.cat((draw(g, T, 2, d).to(BF16), k, v), dim=1).split([2, Hk, Hk], dim=1)[1:]
    before = [None if x is None else x.clone() for x in cache]
    pkg.cache_write(cache, k, v, table, ints(held), starts(new))
    got_k, got_v = pkg.cache_read(cache, table, starts(held), sum(held))
    at_new = at = 0
    touched = torch.zeros(n_pages, page, dtype=torch.bool, device=DEV)
    for b, (p, n) in enumerate(zip(past, new)):
        for x, old, got in ((k, values[0], got_k), (v, values[1], got_v)):
            fresh = x[at_new:at_new + n]
            fresh = fresh.double() if kind == "bf16" else ref.e4m3_rows(fresh)[0]
            want = torch.cat((sequence(old, table, b, p, page), fresh))
            assert torch.equal(got[at:at + p + n].double(), want)
        for t in range(p, p + n):
            touched[table[b, t // page].long(), t % page] = True
        at_new, at = at_new + n, at + p + n
    # the other rows are as they were, exponents too
    for x, old in zip(cache, before):
        if x is not None:
            x, old = x.view(torch.uint8 if x.element_size() == 1 else torch.int16), old.view(torch.uint8 if x.element_size() == 1 else torch.int16)
            keep = ~touched[:, None, :].expand(n_pages, Hk, page)
            assert torch.equal(x[keep], old[keep])


def test_write_one_token_a_sequence_and_heads_first():
    g = gen(2)
    held = [1, 16, 17, 100]
    table, n_pages = paged(g, held, 16)
    cache, _ = filled(g, n_pages, 16, 3, 64, "bf16")
    k, v = (draw(g, 3, 4, 64).to(BF16).transpose(0, 1) for _ in range(2))  # [T, Hk, d] of [Hk, T, d]
    pkg.cache_write(cache, k, v, table, ints(held))
    for b, n in enumerate(held):
        for x, pool in ((k, cache.k), (v, cache.v)):
            assert torch.equal(pool[table[b, (n - 1) // 16].long(), :, (n - 1) % 16], x[b])
    out = tuple(torch.empty(3, 118 + 16, 64, dtype=BF16, device=DEV).transpose(0, 1) for _ in range(2))
    a = pkg.cache_read(cache, table, starts(held), out=out)
    b = pkg.cache_read(cache, table, starts(held), sum(held))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_quantised_rows_at_their_edges():
    g = gen(3)
    d, inf, nan = 64, float("inf"), float("nan")
    x = draw(g, 16, 1, d)
    x[0] = 0.0
    x[1] = 3.3e38
    x[2] = 0.0
    x[2, 0, 3] = 448.0
    x[3] = 0.0
    x[3, 0, 3] = 450.0          # one step of bf16 above 448
    x[4] *= 2.0 ** -120         # below the least exponent
    x[5, 0, 7] = inf
    x[6, 0, 9] = nan
    x[7] = -inf
    x[8, 0, 0], x[8, 0, 1] = 1.0e30, 1.0e-30
    x[9] = torch.arange(d, device=DEV) * 4.0 + 200.0   # ties between steps
    x[10] = 1.0e-38
    x = x.to(BF16)
    held, e = ref.e4m3_rows(x)
    cache = pkg.kv_cache(1, 16, 1, d, "e4m3", DEV)
    table = ints([[0]])
    pkg.cache_write(cache, x, x, table, ints([16]), ints([0, 16]))
    k, v = pkg.cache_read(cache, table, ints([0, 16]), 16)
    assert torch.equal(cache.k_exp[0, 0], e[:, 0]) and torch.equal(cache.v_exp[0, 0], e[:, 0])
    for got in (k, v):
        assert torch.equal(got.isnan(), held.isnan())
        assert torch.equal(torch.nan_to_num(got.double()), torch.nan_to_num(held))


def test_rows_of_no_sequence_stay():
    g = gen(4)
    cache, values = filled(g, 4, 16, 2, 128, "e4m3")
    table = ints([[2, 0], [1, 3]])
    out = tuple(torch.full((40, 2, 128), 7.0, dtype=BF16, device=DEV) for _ in range(2))
    pkg.cache_read(cache, table, ints([3, 20, 30]), out=out)
    for o, x in zip(out, values):
        assert torch.equal(o[3:20].double(), sequence(x, table, 0, 17, 16))
        assert torch.equal(o[20:30].double(), sequence(x, table, 1, 10, 16))
        assert (o[:3] == 7).all() and (o[30:] == 7).all()
    before = [x.clone() for x in cache]
    k, v = rows(g, 9, 2, 128)
    pkg.cache_write(cache, k, v, table, ints([5, 8]), ints([2, 3, 6]))  # tokens 0, 1 and 6 .. 8 belong to nobody
    same = [(x.view(torch.uint8) == y.view(torch.uint8)) for x, y in zip(cache, before)]
    assert same[2].sum() >= same[2].numel() - 4 * 2
    assert same[0][2, :, :4].all() and same[0][2, :, 5:].all() and same[0][1, :, 8:].all() and same[0][3].all()


def test_no_tokens():
    cache = pkg.kv_cache(2, 16, 1, 64, "bf16", DEV)
    empty = torch.empty(0, 1, 64, dtype=BF16, device=DEV)
    pkg.cache_write(cache, empty, empty, ints([[0]]), ints([0]), ints([0, 0]))
    k, v = pkg.cache_read(cache, ints([[0]]), ints([0, 0]), 0)
    assert k.shape == (0, 1, 64)


# ------------------------------------------------------------------ attention of one token


def check_decode(q, cache, values, table, held, page, kind, scale=None, out=None, lse=None):
    B, H, d = q.shape
    Hk = cache.k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o = torch.empty_like(out, dtype=torch.float64) if out is not None else None
    bound, want, lbound = torch.zeros_like(o), torch.zeros_like(lse, dtype=torch.float64), torch.zeros_like(lse, dtype=torch.float64)
    for b, n in enumerate(held):
        k, v = (sequence(x, table, b, n, page) for x in values)
        for h in range(H):
            kh = h // (H // Hk)
            see = torch.ones(1, n, dtype=torch.bool, device=DEV)
            oo, bo, ll, bl = ref.attention(q[b, h][None], k[:, kh], v[:, kh], see, scale, half_weights=kind == "e4m3")
            o[b, h], bound[b, h], want[b, h], lbound[b, h] = oo[0], bo[0], ll[0], bl[0]
    ref.within(out, o, bound, "O")
    ref.within(lse, want, lbound, "LSE")


DECODE = [
    # kind, page, H, Hk, d, lengths
    ("bf16", 16, 1, 1, 64, [1]),
    ("e4m3", 16, 1, 1, 128, [1]),
    ("bf16", 64, 8, 8, 128, [63, 64, 65, 0, 1]),
    ("e4m3", 64, 8, 8, 64, [0, 15, 16, 17, 128, 129]),
    ("bf16", 32, 24, 8, 128, [1000, 33, 2]),
    ("e4m3", 32, 24, 8, 128, [1000, 33, 2]),
    ("bf16", 16, 16, 1, 64, [777]),          # 16 heads share a key head
    ("e4m3", 256, 16, 1, 128, [5000, 1]),
    ("bf16", 128, 21, 1, 128, [300, 40]),    # 21 of them: two chunks of heads, the second in part
    ("e4m3", 64, 40, 1, 64, [511]),
    ("bf16", 64, 7, 7, 64, [9, 0, 0, 200]),
    ("e4m3", 16, 14, 2, 128, [4097, 31, 16]),
    ("bf16", 64, 4, 2, 128, [30011]),        # cut over many CTAs, joined in two steps
    ("e4m3", 64, 2, 1, 64, [60001, 3]),
    ("bf16", 16, 2, 1, 64, [i * 13 % 90 for i in range(300)]),
]


@pytest.mark.parametrize("kind,page,H,Hk,d,held", DECODE)
def test_cache_attention(kind, page, H, Hk, d, held):
    g = gen(5)
    table, n_pages = paged(g, held, page)
    cache, values = filled(g, n_pages, page, Hk, d, kind)
    q = draw(g, len(held), H, d).to(BF16)
    out, lse = pkg.cache_attention(q, cache, table, ints(held))
    check_decode(q, cache, values, table, held, page, kind, out=out, lse=lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_cache_attention_views_scale_and_spread_scores(kind):
    g = gen(6)
    held, page, H, Hk, d = [200, 77, 500], 16, 12, 4, 128
    table, n_pages = paged(g, held, page, width=64)
    cache, values = filled(g, n_pages, page, Hk, d, kind)
    q = (draw(g, 3, H + 8, d) * 4).to(BF16)[:, 3:3 + H]     # scores of some tens: the maximum is raised often
    out = torch.empty(3, 2, H, d, dtype=BF16, device=DEV)[:, 1]
    out, lse = pkg.cache_attention(q, cache, table, ints(held), 0.2, out=out)
    check_decode(q, cache, values, table, held, page, kind, scale=0.2, out=out, lse=lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_cache_attention_is_blind_behind_the_end(kind):
    """NaN in the rows behind a sequence's last token, and in pages that are not its own, does not reach it"""
    g = gen(7)
    held, page, H, Hk, d = [70, 1, 16, 0], 64, 8, 2, 128
    table, n_pages = paged(g, held, page)
    cache, values = filled(g, n_pages, page, Hk, d, kind)
    q = draw(g, 4, H, d).to(BF16)
    a, la = pkg.cache_attention(q, cache, table, ints(held))
    own = torch.zeros(n_pages, page, dtype=torch.bool, device=DEV)
    for b, n in enumerate(held):
        for t in range(n):
            own[table[b, t // page].long(), t % page] = True
    other = ~own[:, None, :].expand(n_pages, Hk, page)
    for x in cache[:2]:
        x.view(torch.int16 if kind == "bf16" else torch.uint8)[other] = 0x7FC0 if kind == "bf16" else 0x7F
    for x in cache[2:]:
        if x is not None:
            x[other] = 255
    b, lb = pkg.cache_attention(q, cache, table, ints(held))
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert (a[3] == 0).all() and (la[3] == float("-inf")).all()


def test_cache_attention_values_of_very_different_size():
    """8-bit rows whose exponents differ by 40: weights are rounded relative to the largest product"""
    g = gen(8)
    held, page, H, Hk, d = [300], 16, 4, 1, 64
    table, n_pages = paged(g, held, page)
    cache, values = filled(g, n_pages, page, Hk, d, "e4m3")
    shift = torch.randint(-20, 21, cache.v_exp.shape, generator=g, device=DEV)
    cache.v_exp.copy_((cache.v_exp.long() + shift).to(torch.uint8))
    values[1] *= torch.pow(2.0, shift.double())[..., None]
    q = draw(g, 1, H, d).to(BF16)
    out, lse = pkg.cache_attention(q, cache, table, ints(held))
    check_decode(q, cache, values, table, held, page, "e4m3", out=out, lse=lse)


def test_a_result_does_not_depend_on_the_other_sequences_order():
    """the same call twice, bit for bit, and with the workspace of other calls before it"""
    g = gen(9)
    held, page = [4000, 1, 999, 2500], 64
    table, n_pages = paged(g, held, page)
    cache, _ = filled(g, n_pages, page, 4, 128, "e4m3")
    q = draw(g, 4, 8, 128).to(BF16)
    ws = pkg.cache_workspace(4, 4, 8, 4, 128, DEV)
    a = pkg.cache_attention(q, cache, table, ints(held), ws=ws)
    for _ in range(3):
        b = pkg.cache_attention(q, cache, table, ints(held), ws=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        pkg.cache_attention(q[:1], cache, table[:1], ints(held[:1]), ws=ws)


# ------------------------------------------------------------------ what only the device sees


def test_bad_pages_and_lengths_are_reported():
    g = gen(10)
    cache, _ = filled(g, 4, 16, 2, 64, "bf16")
    q = draw(g, 2, 2, 64).to(BF16)
    k, v = rows(g, 2, 2, 64)
    for table, held in (([[0, 4], [1, 1]], [17, 5]), ([[0, 1], [-1, 2]], [17, 5]), ([[0, 1], [2, 3]], [33, 5]),
                        ([[0, 1], [2, 3]], [17, -1])):
        ws = pkg.cache_workspace(2, 2, 2, 2, 64, DEV)
        for call in (lambda: pkg.cache_attention(q, cache, ints(table), ints(held), ws=ws),
                     lambda: pkg.cache_write(cache, k, v, ints(table), ints(held), ws=ws)):
            with pytest.raises(bb.BsaError) as e:
                call()
            assert e.value.code == bb.ERR_INVALID_ARG
            pkg.cache_check(ws)  # cleared
    with pytest.raises(bb.BsaError):
        pkg.cache_read(cache, ints([[0, 9]]), ints([0, 20]), 20)
    with pytest.raises(bb.BsaError):
        pkg.cache_read(cache, ints([[0, 1]]), ints([0, 40]), 40)     # longer than its table
    with pytest.raises(bb.BsaError):
        pkg.cache_read(cache, ints([[0, 1]]), ints([0, 40]), 20)     # leaves its tensor
    # a sequence that is well formed beside one that is not gets its result
    table, held = ints([[0, 1], [2, 3]]), [20, -3]
    ws = pkg.cache_workspace(2, 2, 2, 2, 64, DEV)
    out, lse = pkg.cache_attention(q, cache, table, ints(held), ws=ws, check=False)
    check_decode(q[:1], cache, [x.double() for x in cache[:2]], table, [20], 16, "bf16", out=out[:1], lse=lse[:1])
    assert (out[1] == 0).all() and (lse[1] == float("-inf")).all()
    with pytest.raises(bb.BsaError):
        pkg.cache_check(ws)


# ------------------------------------------------------------------ large


def test_large_calls_take_eight_rows_a_thread():
    """8-bit calls of many rows, written and read with eight heads a thread, heads that are no multiple of it"""
    g = gen(11)
    for Hk, d, n in ((12, 128, 5000), (9, 64, 9000)):
        table, n_pages = paged(g, [n, 7], 64)
        cache = pkg.kv_cache(n_pages, 64, Hk, d, "e4m3", DEV)
        k, v = rows(g, n + 7, Hk, d)
        pkg.cache_write(cache, k, v, table, ints([n, 7]), starts([n, 7]))
        for got, x in zip(pkg.cache_read(cache, table, starts([n, 7]), n + 7), (k, v)):
            assert torch.equal(got.double(), ref.e4m3_rows(x)[0])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kind):
    """a cache of more than 2^32 bytes a tensor, the sequences' pages at its end"""
    g = gen(12)
    Hk, d, page = 8, 128, 256
    row = Hk * page * d * (2 if kind == "bf16" else 1)
    n_pages = (1 << 32) // row + 40
    cache = pkg.kv_cache(n_pages, page, Hk, d, kind, DEV)
    held = [1000, 300]
    table = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    table[0, :4] = torch.arange(n_pages - 4, n_pages, device=DEV)
    table[1, :2] = torch.tensor([n_pages - 9, 3], device=DEV)
    k, v = rows(g, sum(held), Hk, d)
    pkg.cache_write(cache, k, v, table, ints(held), starts(held))
    got = pkg.cache_read(cache, table, starts(held), sum(held))
    held_values = [x.double() if kind == "bf16" else ref.e4m3_rows(x)[0] for x in (k, v)]
    assert all(torch.equal(a.double(), b) for a, b in zip(got, held_values))
    q = draw(g, 2, Hk, d).to(BF16)
    out, lse = pkg.cache_attention(q, cache, table, ints(held))
    at = 0
    for b, n in enumerate(held):
        for h in range(Hk):
            see = torch.ones(1, n, dtype=torch.bool, device=DEV)
            o, bo, l, bl = ref.attention(q[b, h][None], held_values[0][at:at + n, h], held_values[1][at:at + n, h], see, d ** -0.5,
                                         half_weights=kind == "e4m3")
            ref.within(out[b, h][None], o, bo, "O")
            ref.within(lse[b, h][None], l, bl, "LSE")
        at += n


def test_cache_attention_keeps_infinities_and_nan_of_its_own_keys():
    g = gen(13)
    held, page, H, Hk, d = [90, 90], 16, 4, 2, 64
    table, n_pages = paged(g, held, page)
    cache, values = filled(g, n_pages, page, Hk, d, "bf16")
    q = draw(g, 2, H, d).to(BF16)
    p, r = table[0, 70 // page].long(), 70 % page
    cache.v[p, 0, r, 5] = float("inf")
    cache.v[p, 1, r, 9] = float("nan")
    out, lse = pkg.cache_attention(q, cache, table, ints(held))
    check_decode(q[1:], cache, values, table[1:], held[1:], page, "bf16", out=out[1:], lse=lse[1:])
    assert (out[0, :2, 5] == float("inf")).all() and out[0, 2:, 9].isnan().all()
    keep = torch.ones(H, d, dtype=torch.bool, device=DEV)
    keep[:2, 5] = keep[2:, 9] = False
    assert out[0][keep].isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("d,H,held", [(64, 4, [300]), (128, 16, [5000, 17]), (128, 3, [40000])])
@pytest.mark.parametrize("large", [20, 60, 80])
def test_weights_of_zeros_and_of_tiny_values_count(d, H, held, large):
    """8-bit rows of zeros and of the least exponent among large ones: their weights are part of the sum all the same"""
    g = gen(14)
    page = 32
    table, n_pages = paged(g, held, page)
    cache, values = filled(g, n_pages, page, 1, d, "e4m3")
    kind = torch.randint(0, 3, cache.v_exp.shape, generator=g, device=DEV)
    kind[:, :, page // 2:] = torch.where(kind[:, :, page // 2:] == 2, 0, kind[:, :, page // 2:])  # tiles without a large one
    data = values[1] * torch.pow(2.0, -(cache.v_exp.double() - 127))[..., None]
    data = torch.where((kind == 0)[..., None], 0.0, data)
    exps = torch.where(kind == 2, cache.v_exp.long() + large, 27)
    cache.v.copy_(data.float())
    cache.v_exp.copy_(exps.to(torch.uint8))
    values[1] = data * torch.pow(2.0, (exps - 127).double())[..., None]
    q = draw(g, len(held), H, d).to(BF16)
    out, lse = pkg.cache_attention(q, cache, table, ints(held))
    check_decode(q, cache, values, table, held, page, "e4m3", out=out, lse=lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_thousands_of_sequences(kind):
    """more than the CTAs, most of them empty or of few tokens"""
    g = gen(15)
    B, H, Hk, d, page = 5000, 2, 1, 64, 16
    held = torch.randint(-20, 40, (B,), generator=g, device=DEV).clamp(min=0).tolist()
    held[4990] = 700
    table, n_pages = paged(g, held, page)
    cache, values = filled(g, n_pages, page, Hk, d, kind)
    q = draw(g, B, H, d).to(BF16)
    out, lse = pkg.cache_attention(q, cache, table, ints(held))
    some = torch.randperm(B, generator=g, device=DEV)[:150].tolist() + [0, 4990, B - 1]
    check_decode(q[some].contiguous(), cache, values, table[some], [held[b] for b in some], page, kind, out=out[some], lse=lse[some])
    empty = torch.tensor(held, device=DEV) == 0
    assert (out[empty] == 0).all() and (lse[empty] == float("-inf")).all()


@pytest.mark.parametrize("d,H,held", [(64, 4, [300]), (128, 16, [5000, 17]), (128, 3, [40000])])
@pytest.mark.parametrize("large", [24, 45, 84, 118])
@pytest.mark.parametrize("level,lift", [(-30, 0), (-40, 5), (-60, 0), (-60, 9), (-200, 5), (0, 9), (60, 0), (200, 5)])
def test_weights_count_at_any_level_of_the_scores(d, H, held, large, level, lift):
    """8-bit rows: zeros and the least exponent, and one in fifty of them large. Every score is moved by `level`, and the large
    rows' by `lift` more: a row's weight is part of the sum wherever the scores lie and however small its value is beside
    another's (of up to 2^127)"""
    g = gen(16)
    page = 32
    table, n_pages = paged(g, held, page)
    cache, values = filled(g, n_pages, page, 1, d, "e4m3")
    kind = torch.randint(0, 50, cache.v_exp.shape, generator=g, device=DEV)
    big = kind == 49
    k = draw(g, *values[0].shape)
    k[..., 0], k[..., 1] = -8.0, torch.where(big, 1.0, 0.0)
    k, e = ref.e4m3_rows(k.to(BF16))
    cache.k.copy_((k / ((e.long() - 127 + 1023) << 52).view(torch.float64)[..., None]).float())
    cache.k_exp.copy_(e)
    data = values[1] * torch.pow(2.0, -(cache.v_exp.double() - 127))[..., None]
    data = torch.where((kind < 25)[..., None], 0.0, data)
    exps = torch.where(big, cache.v_exp.long() + large, 27).clamp(max=246)
    cache.v.copy_(data.float())
    cache.v_exp.copy_(exps.to(torch.uint8))
    values = [k, data * torch.pow(2.0, (exps - 127).double())[..., None]]
    q = draw(g, len(held), H, d)
    q[..., 0], q[..., 1] = -level * d ** 0.5 / 8, lift * d ** 0.5
    q = q.to(BF16)
    out, lse = pkg.cache_attention(q, cache, table, ints(held))
    check_decode(q, cache, values, table, held, page, "e4m3", out=out, lse=lse)


def test_scores_rise_while_the_values_become_smaller():
    """the running maximum of scores and values together stays, that of the scores alone rises by a hundred, within one CTA's
    share too; and a key that is not finite"""
    g = gen(17)
    B, n, page, H, d = 150, 1200, 64, 2, 64
    at = torch.arange(n, device=DEV)
    k, v = draw(g, n, 1, d), draw(g, n, 1, d) * torch.pow(2.0, 60 - at * 0.125)[:, None, None]
    k[:, 0, 0] = at * (8.0 / n)                   # scores of up to 100, 144 as powers of two
    k, v = k.to(BF16), v.to(BF16)
    table, n_pages = paged(g, [n, n], page)
    cache = pkg.kv_cache(n_pages, page, 1, d, "e4m3", DEV)
    other = k.clone()
    other[700, 0, 3] = INF
    pkg.cache_write(cache, torch.cat((k, other)), torch.cat((v, v)), table, ints([n, n]), ints([0, n, 2 * n]))
    table = torch.cat((table, table[:1].expand(B - 2, -1)))  # all but one read the same pages
    q = draw(g, B, H, d)
    q[..., 0] = 100.0
    q = q.to(BF16)
    out, lse = pkg.cache_attention(q, cache, table, ints([n] * B))
    assert out[1].isnan().all() and lse[1].isnan().all()
    keep = torch.arange(B, device=DEV) != 1
    k, v = (ref.e4m3_rows(x)[0][:, 0] for x in (k, v))
    see = torch.ones(1, n, dtype=torch.bool, device=DEV).expand(B - 1, n)
    for h in range(H):
        o, bo, l, bl = ref.attention(q[keep, h], k, v, see, d ** -0.5, half_weights=True)
        ref.within(out[keep, h], o, bo, "O")
        ref.within(lse[keep, h], l, bl, "LSE")


MALFORMED = [
    # tokens, cu, well-formed sequences where cu nowhere decreases (else it is unspecified what is moved)
    (50, [0, 50, 40], []), (8, [0, 5, 3, 8], []), (8, [0, 8, 12], [0]), (12, [0, 8, 4, 12], []), (8, [-3, 0, 8], [1]), (8, [9, 9], []),
    (8, [3, 2, 2], []), (8, [0, 8, 3], []), (3, [0] * 299 + [-1] + [0] * 300 + [3], []), (0, [0, 4], []), (0, [-1, 0], []),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,cu,sound", MALFORMED)
def test_malformed_sequences_are_reported_wherever_they_are(T, cu, sound, kind):
    """also those that no token falls in"""
    g = gen(18)
    B = len(cu) - 1
    cache, values = filled(g, B * 4, 16, 2, 64, kind)
    table = torch.randperm(B * 4, generator=g, device=DEV).to(torch.int32).view(B, 4)
    ws = pkg.cache_workspace(T, B, 2, 2, 64, DEV)
    k, v = rows(g, T, 2, 64)

    def reported(call):
        with pytest.raises(bb.BsaError) as e:
            call()
        assert e.value.code == bb.ERR_INVALID_ARG
        pkg.cache_check(ws)

    out = tuple(torch.full((T, 2, 64), 7.0, dtype=BF16, device=DEV) for _ in range(2))
    reported(lambda: pkg.cache_read(cache, table, ints(cu), out=out, ws=ws))
    for b in sound:
        for o, x in zip(out, values):
            assert torch.equal(o[cu[b]:cu[b + 1]].double(), sequence(x, table, b, cu[b + 1] - cu[b], 16))
    reported(lambda: pkg.cache_write(cache, k, v, table, ints([60] * B), ints(cu), ws=ws))
    for b in sound:
        n = cu[b + 1] - cu[b]
        got = pkg.cache_read(cache, table[b:b + 1], ints([0, 60]), 60, ws=ws)
        for o, x in zip(got, (k, v)):
            want = x[cu[b]:cu[b + 1]]
            assert torch.equal(o[60 - n:].double(), want.double() if kind == "bf16" else ref.e4m3_rows(want)[0])


@pytest.mark.parametrize("lens,cu", [([-1, 8], [0, 0, 8]), ([65, 8], [0, 0, 8]), ([8, 7], [0, 0, 8]), ([8, -2 ** 31], [0, 8, 8]),
                                     ([2 ** 31 - 1, 64], [0, 0, 8]), ([-5], [0, 0]), ([5, 65], None), ([0, 5], None)])
def test_lengths_of_sequences_without_new_tokens_are_looked_at(lens, cu):
    g = gen(19)
    cache, _ = filled(g, 8, 16, 2, 64, "bf16")
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)[:len(lens)]
    T = len(lens) if cu is None else cu[-1]
    k, v = rows(g, T, 2, 64)
    with pytest.raises(bb.BsaError) as e:
        pkg.cache_write(cache, k, v, table, ints(lens), None if cu is None else ints(cu))
    assert e.value.code == bb.ERR_INVALID_ARG


def test_zeros_keep_their_sign():
    """and what is rounded to zero keeps its own, in either form of the 8-bit kernels"""
    g = gen(20)
    for T, Hk, d in ((40, 3, 64), (5000, 12, 128)):
        x = draw(g, T, Hk, d)
        x[..., ::3] = -0.0
        x[..., 1::3] *= 2.0 ** -30
        x[..., 4::9] *= 2.0 ** -100   # subnormal
        x[T // 2] = -0.0
        x = x.to(BF16)
        table, n_pages = paged(g, [T], 64)
        cache = pkg.kv_cache(n_pages, 64, Hk, d, "e4m3", DEV)
        pkg.cache_write(cache, x, x, table, ints([T]), ints([0, T]))
        want = ref.e4m3_rows(x)[0]
        for got in pkg.cache_read(cache, table, ints([0, T]), T):
            assert torch.equal(got.double(), want) and torch.equal(got.signbit(), want.signbit())
