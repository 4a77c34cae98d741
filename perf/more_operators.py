"""Cases of attention over packed prompts and paged caches: a cache of keys and values written (quantised to 8 bits or
not) and read back, the attention of one new token per sequence over it, and the attention over whole prompts.

Where ``own`` is false, ``run`` computes an operator in plain torch operations in 32 bits; where it is true, it calls
the framework. ``exact`` gives the same from the definitions in 64 bits.
"""
import torch

own = False

E4M3_MAX = 448.0
MAX_EXP, MIN_EXP, EXP_BIAS = 119, -100, 127
PROMPT_PAIRS = 32768 * 32768 * 16 // 2   # (query, key) pairs of all heads in the largest listed prompt
SCORES = 1 << 31                         # scores that the plain form holds at a time
CACHE_VALUES = 65536 * 16 * 128 * 2      # values of K in the largest listed caches


# ------------------------------------------------------------------ cases


def _case(name, op, lens, H, Hk, d, **more):
    """lens: a sequence's new tokens (prompt, write) or its tokens in the cache (decode, read)"""
    case = {"op": op, "lens": ",".join(str(n) for n in lens), "H": H, "Hk": Hk, "d": d}
    case.update({"past": "", "causal": True, "fused": True} if op == "prompt" else
                {"kind": "bf16", "page": 64, "past": "", "fused": True})
    case.update(more)
    return dict(case, name=name) if name else case


def _spaced(lo, hi, n):
    """n lengths between lo and hi, evenly spaced on the logarithm, in an order that mixes long and short ones"""
    got = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]
    return [got[i * 37 % n] for i in range(n)] if n % 37 else got


def listed():
    return [
        # four text prompts of a caption, of the image model's heads: latency of a call
        _case("prompt text", "prompt", [77, 12, 128, 33], 24, 24, 64),
        # six prompts of text and image tokens packed together, three query heads to a key head
        _case("prompt packed", "prompt", [4224, 1000, 2777, 513, 3333, 4096], 24, 8, 128),
        # one long prompt of the sweep's heads
        _case("prompt long", "prompt", [32768], 16, 16, 128, fused=False),
        # the next frame of a video: 1024 tokens that see each other and 31 frames before them
        _case("prompt frame", "prompt", [1024], 16, 4, 128, past="31744", causal=False, fused=False),
        # one caption being written: latency of a call
        _case("decode one", "decode", [333], 24, 24, 64),
        # 64 sequences of very different lengths, 8-bit cache, three query heads to a key head
        _case("decode batch fp8", "decode", _spaced(100, 8192, 64), 24, 8, 128, kind="fp8"),
        # two long videos, a key head per query head
        _case("decode long", "decode", [65536, 40001], 16, 16, 128, page=256),
        # one key head for all query heads
        _case("decode shared", "decode", _spaced(9000, 30001, 8), 16, 1, 128, kind="fp8", page=32),
        # the new token of each of 64 sequences
        _case("append", "write", [1] * 64, 24, 8, 128, past=",".join(str(n) for n in _spaced(31, 511, 64)), page=16),
        # prompts quantised into the cache, and read back
        _case("write fp8", "write", [8192, 4224, 777, 2500], 24, 8, 128, kind="fp8", past="0,64,1000,0"),
        # a frame of each of four sequences read back, pages of 16
        _case("read short", "read", [256, 1, 77, 300], 24, 24, 64, page=16),
        # a long 8-bit cache read back for the next chunk
        _case("read long fp8", "read", [65536], 16, 16, 128, kind="fp8"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "write", "read"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 5, 8, 16, 24])
    H = Hk * rng.choice([g for g in (1, 1, 2, 3, 4, 7, 8, 16) if Hk * g <= 64])
    B = rng.choice([1, 1, 2, 3, 8, 17])
    if op == "prompt":
        chunk, causal = rng.random() < 0.3, rng.random() < 0.75
        most = int(((2 if causal else 1) * PROMPT_PAIRS / (B * H)) ** 0.5)
        most = min(32768, most)
        # with earlier tokens: a chunk of at most an eighth of the longest prompt, over a context of at most all of it
        longest = _spread(rng, 1, most // 8 if chunk else most)
        lens = [max(1, int(longest * rng.choice([1.0, 0.9, 0.5, 0.25]))) for _ in range(B)]
        lens[rng.randrange(B)] = longest
        past = [_spread(rng, 1, most) for _ in lens] if chunk else []
        return _case(None, op, lens, H, Hk, d, past=",".join(str(n) for n in past), causal=causal,
                     fused=rng.random() < 0.5 and not past)
    kind, page = rng.choice(["bf16", "fp8"]), rng.choice([16, 32, 64, 128, 256])
    if op == "decode":
        B = rng.choice([1, 2, 7, 16, 64, 129])
    longest = _spread(rng, 1, min(131072, CACHE_VALUES // (2 * B * Hk * d)))
    lens = [max(1, int(longest * rng.choice([1.0, 0.7, 0.3, 0.05]))) for _ in range(B)]
    lens[rng.randrange(B)] = longest
    past = ""
    if op == "write" and rng.random() < 0.6:
        past = ",".join(str(rng.choice([0, 1, 15, 64, 333])) for _ in lens)
    return _case(None, op, lens, H, Hk, d, kind=kind, page=page, past=past, fused=rng.random() < 0.6)


def _lens(case, key="lens"):
    return [int(n) for n in case[key].split(",")] if case[key] else [0] * len(_lens(case))


def _pairs(case):
    """visible (query, key) pairs of one head"""
    if case["op"] == "decode":
        return sum(_lens(case))
    n = 0
    for q, past in zip(_lens(case), _lens(case, "past")):
        n += q * past + (q * (q + 1) // 2 if case["causal"] else q * q)
    return n


def work(case):
    tokens, H, Hk, d = sum(_lens(case)), case["H"], case["Hk"], case["d"]
    if case["op"] == "prompt":
        keys = tokens + sum(_lens(case, "past"))
        return {"bytes": 4 * tokens * H * d + 4 * keys * Hk * d + 4 * tokens * H, "flops": 4 * d * H * _pairs(case)}
    cached = 2 * tokens * Hk * (2 * d if case["kind"] == "bf16" else d + 1)  # K and V in the cache
    if case["op"] == "decode":
        B = len(_lens(case))
        return {"bytes": cached + 4 * B * H * d + 4 * B * H, "flops": 4 * d * H * _pairs(case)}
    packed = 4 * tokens * Hk * d
    if case["op"] == "read" or case["kind"] == "bf16":
        return {"bytes": packed + cached, "flops": 0}
    return {"bytes": 2 * (packed + cached), "flops": 4 * tokens * Hk * d}  # written, then read back


# ------------------------------------------------------------------ inputs


def _starts(lens, device):
    """int32 [B + 1]: where each sequence begins among the packed tokens"""
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=device)


def _power(e):
    """2^e in fp32, e int32 in [-126, 127]: from its bits, since pow may be off by a unit in the last place"""
    return ((e + EXP_BIAS) << 23).view(torch.float32)


def _quantised(x):
    """(e4m3 data, byte of the exponent) of rows x [..., d]: data * 2^(byte - 127) is the row"""
    x = x.float()
    a = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1)
    e = torch.where(a > 0, e - torch.where(m <= 0.875, 9, 8), MIN_EXP).clamp(MIN_EXP, MAX_EXP).int()
    y = (x * _power(-e)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    y = torch.where(x.isfinite(), y, float("nan"))
    return y.to(torch.float8_e4m3fn), (e + EXP_BIAS).to(torch.uint8)


def _values(data, exps):
    return data.float() if exps is None else data.float() * _power(exps.int() - EXP_BIAS)[..., None]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    H, Hk, d = case["H"], case["Hk"], case["d"]
    lens, past = _lens(case), _lens(case, "past")
    tokens = sum(lens)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def keys(n):
        """keys with a few large channels, values of tokens of different size: [n, Hk, d] each"""
        k, v = normal(n, Hk, d), normal(n, Hk, d)
        big = torch.randperm(d, generator=gen, device=dev)[: d // 32]
        k[..., big] *= 3.0
        return k.bfloat16(), (v * torch.exp(0.5 * normal(n, Hk, 1))).bfloat16()

    s = {"case": case}
    if case["op"] == "prompt":
        total = tokens + sum(past)
        k, v = keys(total)
        q = normal(tokens, H, d).bfloat16()
        if case["fused"]:  # views of one projection
            q, k, v = torch.cat((q, k, v), dim=1).split([H, Hk, Hk], dim=1)
        s.update(q=q, k=k, v=v, cu_q=_starts(lens, dev), cu_k=_starts([n + p for n, p in zip(lens, past)], dev))
        s["out"] = torch.empty(tokens, H, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(H, tokens, device=dev)
        if own:
            import block_sparse_attention_mean_gb300 as pkg
            s["ws"] = pkg.cache_workspace(tokens, len(lens), H, Hk, d, dev)
        return s
    # a cache whose pages belong to the sequences in no order, a few of them to none
    page, B = case["page"], len(lens)
    held = [n + p for n, p in zip(lens, past)]
    wide = max(-(-n // page) for n in held)
    used = sum(-(-n // page) for n in held)
    order = torch.randperm(used + 3, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(B, wide, dtype=torch.int32, device=dev)
    col = torch.arange(wide, device=dev)
    count = torch.tensor([-(-n // page) for n in held], device=dev)
    table[col < count[:, None]] = order[:used]
    k, v = keys((used + 3) * page)
    pages = (used + 3, page, Hk, d)
    k, v = (x.view(pages).transpose(1, 2).contiguous() for x in (k, v))  # [pages, Hk, page, d]
    s["cache"] = (k, v, None, None)
    if case["kind"] == "fp8":
        (k, ke), (v, ve) = _quantised(k), _quantised(v)
        s["cache"] = (k, v, ke, ve)
    s["table"], s["held"] = table, torch.tensor(held, dtype=torch.int32, device=dev)
    if case["op"] == "decode":
        s["q"] = normal(B, H, d).bfloat16()
        if case["fused"]:
            s["q"] = torch.cat((s["q"], normal(B, 2 * Hk, d).bfloat16()), dim=1)[:, :H]
        s["out"], s["lse"] = torch.empty(B, H, d, dtype=torch.bfloat16, device=dev), torch.empty(B, H, device=dev)
    else:
        if case["op"] == "write":
            k, v = keys(tokens)
            if case["fused"]:
                k, v = torch.cat((normal(tokens, H, d).bfloat16(), k, v), dim=1).split([H, Hk, Hk], dim=1)[1:]
            s["k"], s["v"] = k, v
            s["cu_held"] = _starts(held, dev)
        s["cu"], s["tokens"], s["cached"] = _starts(lens, dev), tokens, sum(held)
        n = s["tokens"] if case["op"] == "read" else s["cached"]
        if case["op"] == "read" or case["kind"] == "fp8":
            s["out"] = tuple(torch.empty(n, Hk, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    if own:
        import block_sparse_attention_mean_gb300 as pkg
        s["kv"] = pkg.KvCache(*s["cache"])
        s["ws"] = pkg.cache_workspace(B, B, H, Hk, d, dev)
    return s


# ------------------------------------------------------------------ plain forms


def _padded(x, cu, longest):
    """packed rows [T, heads, d] as fp32 [B, heads, longest, d]; rows past a sequence's end are zeros"""
    at = torch.arange(longest, device=x.device)
    there = at < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + at).clamp(max=max(0, x.shape[0] - 1))
    return torch.where(there[..., None, None], x[rows].float(), 0.0).transpose(1, 2)


def _softmax_rows(q, k, v, visible):
    """q [B, Hk, rows, d], k and v [B, Hk, keys, d], visible [B, 1, rows or 1, keys]: (O, LSE)"""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(q.shape[-1] ** -0.5)
    s.masked_fill_(~visible, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return o, (m + total.log()).squeeze(-1)


def _plain_prompt(s):
    case, cu_q, cu_k = s["case"], s["cu_q"], s["cu_k"]
    H, Hk, d = case["H"], case["Hk"], case["d"]
    g = H // Hk
    n_q, n_k = _lens(case), [n + p for n, p in zip(_lens(case), _lens(case, "past"))]
    Lq, Lk, B = max(n_q), max(n_k), len(n_q)
    q, k, v = _padded(s["q"], cu_q, Lq), _padded(s["k"], cu_k, Lk), _padded(s["v"], cu_k, Lk)
    len_q, len_k = ((cu[1:] - cu[:-1])[:, None, None, None] for cu in (cu_q, cu_k))
    key = torch.arange(Lk, device=q.device)
    q = q.reshape(B, Hk, g, Lq, d)
    part = max(1, SCORES // (B * H * Lk))
    got = []
    for at in range(0, Lq, part):  # as many query rows at a time as the scores have room for
        i = torch.arange(at, min(at + part, Lq), device=q.device).repeat(g)[:, None]
        last = i + len_k - len_q if case["causal"] else len_k - 1
        visible = (key <= last) & (key < len_k)
        o, lse = _softmax_rows(q[:, :, :, at:at + part].reshape(B, Hk, -1, d), k, v, visible)
        got.append((o.view(B, H, -1, d), lse.view(B, H, -1)))
    o, lse = (torch.cat(x, dim=2) for x in zip(*got))
    real = torch.arange(Lq, device=q.device) < len_q[:, 0, 0]
    return o.transpose(1, 2)[real].bfloat16(), lse.transpose(1, 2)[real].T.contiguous()


def _gathered(data, exps, table):
    """pages of the table as fp32 [B, Hk, tokens, d]"""
    x = _values(data[table], None if exps is None else exps[table])  # [B, pages, Hk, page, d]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_decode(s):
    k, v, ke, ve = s["cache"]
    case = s["case"]
    B, H, Hk, d = len(_lens(case)), case["H"], case["Hk"], case["d"]
    k, v = _gathered(k, ke, s["table"]), _gathered(v, ve, s["table"])
    visible = torch.arange(k.shape[2], device=k.device) < s["held"][:, None, None, None]
    o, lse = _softmax_rows(s["q"].float().reshape(B, Hk, H // Hk, d), k, v, visible)
    return o.reshape(B, H, d).bfloat16(), lse.reshape(B, H)


def _places(cu, first, table, page, tokens):
    """(page, row in it) of each packed token; a sequence's tokens follow each other from `first` [B]"""
    t = torch.arange(tokens, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t.to(cu.dtype), right=True)
    at = first[b] + t - cu[b]
    return table[b, at // page], at % page


def _plain_read(s, cu, tokens):
    k, v, ke, ve = s["cache"]
    p, r = _places(cu, torch.zeros_like(cu[1:]), s["table"], s["case"]["page"], tokens)
    return tuple(_values(x[p, :, r], None if e is None else e[p, :, r]).bfloat16() for x, e in ((k, ke), (v, ve)))


def _plain_write(s):
    k, v, ke, ve = s["cache"]
    cu = s["cu"]
    p, r = _places(cu, s["held"] - (cu[1:] - cu[:-1]), s["table"], s["case"]["page"], s["tokens"])
    for x, data, exps in ((s["k"], k, ke), (s["v"], v, ve)):
        if exps is None:
            data[p, :, r] = x
        else:
            y, e = _quantised(x)
            data.view(torch.uint8)[p, :, r] = y.view(torch.uint8)
            exps[p, :, r] = e
    return (k, v) if ke is None else _plain_read(s, s["cu_held"], s["cached"])


# ------------------------------------------------------------------ one pass


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "read":
            return _plain_read(s, s["cu"], s["tokens"])
        return {"prompt": _plain_prompt, "decode": _plain_decode, "write": _plain_write}[case["op"]](s)
    import block_sparse_attention_mean_gb300 as pkg
    if case["op"] == "prompt":
        return pkg.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"], out=s["out"],
                                    lse=s["lse"], ws=s["ws"], check=False)
    if case["op"] == "decode":
        return pkg.cache_attention(s["q"], s["kv"], s["table"], s["held"], out=s["out"], lse=s["lse"], ws=s["ws"],
                                   check=False)
    if case["op"] == "read":
        return pkg.cache_read(s["kv"], s["table"], s["cu"], out=s["out"], ws=s["ws"], check=False)
    pkg.cache_write(s["kv"], s["k"], s["v"], s["table"], s["held"], s["cu"], ws=s["ws"], check=False)
    if case["kind"] == "bf16":
        return s["cache"][:2]
    return pkg.cache_read(s["kv"], s["table"], s["cu_held"], out=s["out"], ws=s["ws"], check=False)


# ------------------------------------------------------------------ definitions in 64 bits


def _exact_rows(q, k, v, last):
    """q [rows, d] of one head over k, v [keys, d]; row i sees the keys up to last[i] (none below zero)"""
    s = (q @ k.T) / q.shape[-1] ** 0.5
    s = s.masked_fill(torch.arange(k.shape[0], device=q.device) > last[:, None], float("-inf"))
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - torch.where(lse.isfinite(), lse, 0.0)[:, None]) @ v, lse


def _exact_prompt(case, s):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    g = case["H"] // case["Hk"]
    at_q = at_k = 0
    for n, past in zip(_lens(case), _lens(case, "past")):
        for h in range(case["H"]):
            k, v = (s[x][at_k:at_k + n + past, h // g].double() for x in "kv")
            for lo in range(0, n, 4096):
                hi = min(n, lo + 4096)
                last = torch.arange(lo, hi, device="cuda") + past
                last = last if case["causal"] else torch.full_like(last, n + past - 1)
                keys = int(past + hi) if case["causal"] else n + past
                o[at_q + lo:at_q + hi, h], lse[h, at_q + lo:at_q + hi] = _exact_rows(
                    s["q"][at_q + lo:at_q + hi, h].double(), k[:keys], v[:keys], last)
        at_q, at_k = at_q + n, at_k + n + past
    return o, lse


def _exact_cached(s, b, n):
    """the first n tokens of sequence b in 64 bits: K and V [n, Hk, d]"""
    page = s["case"]["page"]
    ids = s["table"][b, : -(-n // page)].long()
    got = []
    for data, exps in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        x = data[ids].double()
        if exps is not None:
            x = x * _power64(exps[ids].long() - EXP_BIAS)[..., None]
        got.append(x.permute(0, 2, 1, 3).flatten(0, 1)[:n])
    return got


def _power64(e):
    return ((e + 1023) << 52).view(torch.float64)


def _exact_e4m3(x):
    """rows x [..., d] as the values that the cache holds for them"""
    x = x.double()
    a = x.abs().amax(-1, keepdim=True)
    e = torch.full(a.shape, MIN_EXP, dtype=torch.int64, device=x.device)
    for i in range(MIN_EXP, MAX_EXP):  # one more wherever the row does not fit yet
        e += a > E4M3_MAX * 2.0 ** i
    unit = _power64(e)
    y = x / unit
    step = _power64(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].long() - 4)  # three bits behind the first
    return torch.round(y / step) * step * unit


def exact(case, seed):
    if case["op"] == "prompt" and _pairs(case) * case["H"] * case["d"] > 6e12 / 4:
        return None
    s = prepare(case, seed)
    lens, past = _lens(case), _lens(case, "past")
    if case["op"] == "prompt":
        return _exact_prompt(case, s)
    if case["op"] == "decode":
        g = case["H"] // case["Hk"]
        o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), s["lse"].double()
        for b, n in enumerate(lens):
            k, v = _exact_cached(s, b, n)
            for h in range(case["Hk"]):
                rows = slice(h * g, (h + 1) * g)
                o[b, rows], lse[b, rows] = _exact_rows(s["q"][b, rows].double(), k[:, h], v[:, h],
                                                       torch.full((g,), n, device="cuda"))
        return o, lse
    if case["op"] == "read":
        got = [_exact_cached(s, b, n) for b, n in enumerate(lens)]
        return tuple(torch.cat(x) for x in zip(*got))
    at, got = 0, []
    pool = [x.double() for x in s["cache"][:2]] if case["kind"] == "bf16" else None
    for b, (n, p) in enumerate(zip(lens, past)):
        new = [s[x][at:at + n].double() for x in "kv"]
        at += n
        if pool is None:
            got.append([torch.cat((old, _exact_e4m3(x))) for old, x in zip(_exact_cached(s, b, p), new)])
            continue
        for i in range(n):
            place = s["table"][b, (p + i) // case["page"]].long()
            for x, y in zip(pool, new):
                x[place, :, (p + i) % case["page"]] = y[i]
    return tuple(pool) if pool is not None else tuple(torch.cat(x) for x in zip(*got))
