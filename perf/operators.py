"""Cases of the operators around the attention: rotary positions with several axes (bsa_rotary and its
backward pass) and the gated norm between two sub-blocks (bsa_gated_norm and its backward pass).

Where ``own`` is false, ``run`` computes an operator in plain torch operations in 32 bits (angles in 64);
where it is true, it calls the framework. ``exact`` gives the same from the definitions in 64 bits.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
MAX_ELEMENTS = 65536 * 16 * 128  # elements of one tensor of the largest listed cases


# ------------------------------------------------------------------ cases


def _rotary(name, op, dt, B, H, Hk, N, d, axes, **more):
    case = {"op": op, "dt": dt, "B": B, "H": H, "Hk": Hk, "N": N, "d": d, "axes": axes, "interleaved": True,
            "norm": True, "fused": True, "n_text": 0, "grid": "", "far": 0}
    case.update(more)
    return dict(case, name=name) if name else case


def _gated(name, op, stream, branch, mod, B, F, N, C, **more):
    case = {"op": op, "stream": stream, "branch": branch, "mod": mod, "B": B, "F": F, "N": N, "C": C,
            "post": "none", "post_affine": "none", "pre": "layer", "pre_affine": "none", "gate": True,
            "modulate": True, "alpha": 1.0, "branch_in": True}
    case.update(more)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one head pair of the small fp32 problem, positions along the sequence only: latency of a call
        _rotary("rotary small fp32", "rotary", "fp32", 1, 2, 2, 512, 64, "64", norm=False, fused=False),
        # text-to-image: 128 text tokens at the origin, 64 x 64 patches on two axes, fused projection
        _rotary("rotary image", "rotary", "bf16", 2, 24, 24, 4224, 64, "32,32", n_text=128, grid="64,64"),
        # video: 256 text tokens, 16 x 32 x 32 latent tokens on three axes of unequal width
        _rotary("rotary video", "rotary", "bf16", 1, 24, 24, 16640, 128, "44,42,42", n_text=256, grid="16,32,32"),
        # the longest video, channel halves as pairs
        _rotary("rotary long", "rotary", "bf16", 1, 16, 16, 65536, 128, "16,56,56", interleaved=False,
                grid="64,32,32"),
        # training on a short clip of odd length, keys and values shared by four query heads
        _rotary("rotary grad odd", "rotary_backward", "bf16", 2, 8, 2, 777, 128, "32,48,48", grid="7,11,11"),
        # training on the video shape
        _rotary("rotary grad video", "rotary_backward", "bf16", 1, 24, 24, 16640, 128, "44,42,42", n_text=256,
                grid="16,32,32"),
        # the first norm of a block on the text tokens alone: latency of a call
        _gated("norm text", "gated_norm", "bf16", "bf16", "bf16", 1, 1, 128, 1536, branch_in=False, gate=False),
        # between attention and feed-forward on the image shape
        _gated("norm image", "gated_norm", "bf16", "bf16", "bf16", 2, 1, 4224, 1536),
        # a sandwich block (norm after the branch, with weight) on the longest video, one modulation a frame
        _gated("norm long sandwich", "gated_norm", "bf16", "bf16", "bf16", 1, 64, 65536, 2048, post="rms",
               post_affine="weight", pre="rms", pre_affine="weight"),
        # fp32 residual stream and modulation, bf16 branch, odd number of tokens
        _gated("norm fp32 stream", "gated_norm", "fp32", "bf16", "fp32", 1, 1, 16385, 2048, pre_affine="bias"),
        # training, image shape
        _gated("norm grad image", "gated_norm_backward", "bf16", "bf16", "bf16", 2, 1, 4224, 1536),
        # training, sandwich block on the video shape, one modulation for each of 16 frames
        _gated("norm grad video", "gated_norm_backward", "bf16", "bf16", "bf16", 1, 16, 16384, 2048, post="rms",
               post_affine="weight", pre="rms", pre_affine="weight"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_backward", "gated_norm", "gated_norm_backward"])
    # a backward pass of a case costs more than its forward: its sizes stay lower
    limit = MAX_ELEMENTS if op in ("rotary", "gated_norm") else MAX_ELEMENTS // 4
    B = rng.choice([1, 1, 1, 2, 3])
    if op.startswith("rotary"):
        d, dt = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "fp32"])
        limit = limit if dt == "bf16" else limit // 2
        Hk = rng.choice([1, 2, 5, 8, 12, 16, 24])
        H = Hk * rng.choice([1, 1, 1, 4]) if Hk <= 8 else Hk
        N = _spread(rng, 1, max(1, min(65536, limit // (B * H * d))))
        n_axes = rng.choice([1, 2, 3, 3, 4])
        interleaved = rng.random() < 0.5
        rot = d if rng.random() < 0.7 else rng.choice([16, 32, 48])
        cuts = sorted(rng.sample(range(1, rot // 2), n_axes - 1))
        axes = [2 * (b - a) for a, b in zip([0] + cuts, cuts + [rot // 2])]
        grid = [rng.randint(1, 40) for _ in axes]
        return _rotary(None, op, dt, B, H, Hk, N, d,
                       ",".join(str(a) for a in axes), interleaved=interleaved, norm=rng.random() < 0.7,
                       fused=rng.random() < 0.6, n_text=min(N, rng.choice([0, 0, 77, 256])),
                       grid=",".join(str(g) for g in grid), far=rng.choice([0, 0, 1000, 1000000]))
    stream, branch = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
    limit = limit if stream == "bf16" else limit // 2
    C = 8 * _spread(rng, 8, 1024)
    N = _spread(rng, 1, max(1, min(65536, limit // (B * C))))
    F = rng.choice([f for f in (1, 1, 2, 7, 16, N) if N % f == 0 and N <= 2 ** 40])
    F = 1 if F == N and N > 4096 else F
    pre = rng.choice(["layer", "rms", "layer", "rms", "none"])
    branch_in = pre == "none" or rng.random() < 0.8
    post = rng.choice(["none", "rms", "layer"]) if branch_in else "none"
    affine = ["none", "weight", "bias"]
    return _gated(None, op, stream, branch, rng.choice(["bf16", "fp32"]), B, F, N, C, post=post,
                  post_affine="none" if post == "none" else rng.choice(affine), pre=pre,
                  pre_affine="none" if pre == "none" else rng.choice(affine),
                  gate=branch_in and rng.random() < 0.8, modulate=pre != "none" and rng.random() < 0.8,
                  alpha=rng.choice([1.0, 0.5]), branch_in=branch_in)


def work(case):
    if case["op"].startswith("rotary"):
        tokens, d, size = case["B"] * case["N"], case["d"], 2 if case["dt"] == "bf16" else 4
        qk, v = tokens * (case["H"] + case["Hk"]) * d, tokens * case["Hk"] * d
        passes = 2 * (qk + v) + (qk if case["op"] == "rotary_backward" and case["norm"] else 0)
        n_axes = len(case["axes"].split(","))
        return {"bytes": passes * size + 4 * case["N"] * n_axes, "flops": 10 * qk}
    cells = case["B"] * case["N"] * case["C"]
    stream, branch = (2 if case[k] == "bf16" else 4 for k in ("stream", "branch"))
    pre, y = case["pre"] != "none", case["branch_in"]
    if case["op"] == "gated_norm":  # x, y read; h, z written
        size = stream + (branch + stream if y else 0) + (branch if pre else 0)
    else:  # dh, dz, h, y read; dx, dy written
        size = 2 * stream + (branch + stream if pre else 0) + (2 * branch if y else 0)
    rows = (int(case["gate"]) + 2 * int(case["modulate"])) * case["B"] * case["F"] * case["C"]
    rows *= 2 if case["op"] == "gated_norm_backward" else 1
    return {"bytes": cells * size + rows * (2 if case["mod"] == "bf16" else 4), "flops": 20 * cells}


# ------------------------------------------------------------------ inputs


def _positions(case, device):
    """int32 [N, axes]: text tokens count along the first axis, the others run over the grid, last axis first."""
    axes = [int(a) for a in case["axes"].split(",")]
    grid = [int(g) for g in case["grid"].split(",")] if case["grid"] else [1] * len(axes)
    i = torch.arange(case["N"], device=device) - case["n_text"]
    text = i < 0
    pos = []
    rest = i.clamp(min=0)
    for g in reversed(grid[1:]):
        pos.append(rest % g)
        rest = rest // g
    pos.append(rest + case["far"])
    pos = torch.stack(pos[::-1], dim=1)
    pos[text] = 0
    pos[text, 0] = (i + case["n_text"])[text]
    return pos.to(torch.int32)


def _inv_freq(case):
    """Frequency (64 bits) and axis of every pair: 10000^(-2 j / dim) along each axis."""
    freq, axis = [], []
    for a, dim in enumerate(int(x) for x in case["axes"].split(",")):
        freq += [10000.0 ** (-2.0 * j / dim) for j in range(dim // 2)]
        axis += [a] * (dim // 2)
    return freq, axis


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)

    def normal(*shape, dt=torch.float32, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale + mean).to(dt)

    s = {"case": case}
    B, N = case["B"], case["N"]
    if case["op"].startswith("rotary"):
        H, Hk, d, dt = case["H"], case["Hk"], case["d"], DTYPES[case["dt"]]

        def three(fill):
            """q, k, v as [B, N, heads, d]: views of one fused projection, or three tensors"""
            if case["fused"]:
                return fill(B, N, H + 2 * Hk, d).split([H, Hk, Hk], dim=2)
            return fill(B, N, H, d), fill(B, N, Hk, d), fill(B, N, Hk, d)

        def heads_first(fill):
            return fill(B, H, N, d), fill(B, Hk, N, d), fill(B, Hk, N, d)

        def draws(*shape):
            return normal(*shape, dt=dt)

        def buffer(*shape):
            return torch.empty(*shape, dtype=dt, device=dev)

        s["qkv"] = three(draws)
        s["weights"] = (normal(d, scale=0.2, mean=1.0), normal(d, scale=0.2, mean=1.0)) if case["norm"] else (None, None)
        s["pos"] = _positions(case, dev)
        freq, axis = _inv_freq(case)
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor(axis, device=dev)
        s["out"] = heads_first(buffer) if case["op"] == "rotary" else three(buffer)
        if case["op"] == "rotary_backward":
            s["grads"] = heads_first(draws)
        if own:
            import block_sparse_attention_mean_gb300 as pkg
            s["plan"] = pkg.rotary_plan(d, [int(a) for a in case["axes"].split(",")], theta=10000.0,
                                        interleaved=case["interleaved"])
            if case["op"] == "rotary_backward":
                s["ws"] = pkg.rotary_workspace(B, N, d, dev)
        return s
    C, F = case["C"], case["F"]
    stream, branch, mod = (DTYPES[case[k]] for k in ("stream", "branch", "mod"))

    def residual():
        """a residual stream: some channels much larger than the others, and off zero"""
        x = normal(B, N, C)
        big = torch.randperm(C, generator=gen, device=dev)[: max(1, C // 64)]
        x[..., big] = x[..., big] * 8.0 + 4.0
        return x.to(stream)

    def weights(kind):
        return (normal(C, scale=0.1, mean=1.0) if kind != "none" else None,
                normal(C, scale=0.1) if kind == "bias" else None)

    # shift, scale and gate as views of one projection of the conditioning
    rows = normal(B, F, 3, C, dt=mod, scale=0.3)
    s["shift"], s["scale"] = (rows[:, :, 0], rows[:, :, 1]) if case["modulate"] else (None, None)
    s["gate"] = rows[:, :, 2] if case["gate"] else None
    s["post_w"], s["post_b"] = weights(case["post_affine"])
    s["pre_w"], s["pre_b"] = weights(case["pre_affine"])
    s["y"] = normal(B, N, C, dt=branch) if case["branch_in"] else None
    pre = case["pre"] != "none"
    if case["op"] == "gated_norm":
        s["x"] = residual()
        s["out"] = (torch.empty_like(s["x"]) if case["branch_in"] else None,
                    torch.empty(B, N, C, dtype=branch, device=dev) if pre else None)
    else:
        s["h"] = residual() if pre else None
        s["dh"] = normal(B, N, C, dt=stream)
        s["dz"] = normal(B, N, C, dt=branch) if pre else None
        s["out"] = (torch.empty(B, N, C, dtype=stream, device=dev) if pre else None,
                    torch.empty_like(s["y"]) if case["branch_in"] else None)
    if own:
        import block_sparse_attention_mean_gb300 as pkg
        s["post"] = pkg.NormSpec(case["post"], s["post_w"], s["post_b"], 1e-6) if case["post"] != "none" else None
        s["pre"] = pkg.NormSpec(case["pre"], s["pre_w"], s["pre_b"], 1e-6) if pre else None
        if case["op"] == "gated_norm_backward":
            s["ws"] = pkg.gated_norm_workspace(B, N, C, dev)
    return s


# ------------------------------------------------------------------ plain forms


def _rotate(u, cos, sin, interleaved):
    """u [..., d] with its first 2 * cos.shape[-1] channels turned by the angles"""
    p = cos.shape[-1]
    rest = u[..., 2 * p:]
    if interleaved:
        a, b = u[..., 0:2 * p:2], u[..., 1:2 * p:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = u[..., :p], u[..., p:2 * p]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _plain_rotary(s):
    case = s["case"]
    angle = s["pos"].double()[:, s["axis"]] * s["freq"]
    cos, sin = angle.cos().float()[None, :, None], angle.sin().float()[None, :, None]

    def one(x, w):
        u = x.float()
        if case["norm"]:
            u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6) * w
        return _rotate(u, cos, sin, case["interleaved"]).transpose(1, 2).to(x.dtype).contiguous()

    q, k, v = s["qkv"]
    return one(q, s["weights"][0]), one(k, s["weights"][1]), v.transpose(1, 2).contiguous()


def _plain_rotary_backward(s):
    case = s["case"]
    angle = s["pos"].double()[:, s["axis"]] * s["freq"]
    cos, sin = angle.cos().float()[None, :, None], angle.sin().float()[None, :, None]

    def one(dy, x, w):
        g = _rotate(dy.float().transpose(1, 2), cos, -sin, case["interleaved"])
        if not case["norm"]:
            return g.to(x.dtype), None
        x32 = x.float()
        r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + 1e-6)
        n = x32 * r
        dw = (g * n).sum((0, 1, 2))
        g = g * w
        return (r * (g - n * (g * n).mean(-1, keepdim=True))).to(x.dtype), dw

    dq, dk, dv = s["grads"]
    gq, gwq = one(dq, s["qkv"][0], s["weights"][0])
    gk, gwk = one(dk, s["qkv"][1], s["weights"][1])
    return gq, gk, dv.transpose(1, 2).contiguous(), gwq, gwk


def _normal_rows(x, kind):
    """the rows of x (fp32) normalised, and 1 / their scale"""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return x * r, r


def _affine(n, w, b):
    n = n if w is None else n * w
    return n if b is None else n + b


def _by_token(m, case):
    """a modulation [B, F, C] as fp32 [B, N, C] (or broadcastable to it)"""
    m = m.float()
    return m if case["F"] == 1 else m.repeat_interleave(case["N"] // case["F"], dim=1)


def _plain_gated_norm(s):
    case = s["case"]
    h = s["x"].float()
    if case["branch_in"]:
        u = s["y"].float()
        if case["post"] != "none":
            u = _affine(_normal_rows(u, case["post"])[0], s["post_w"], s["post_b"])
        if case["gate"]:
            u = u * _by_token(s["gate"], case)
        h = h + case["alpha"] * u
    z = None
    if case["pre"] != "none":
        z = _affine(_normal_rows(h, case["pre"])[0], s["pre_w"], s["pre_b"])
        if case["modulate"]:
            z = z * (1.0 + _by_token(s["scale"], case)) + _by_token(s["shift"], case)
        z = z.to(DTYPES[case["branch"]])
    return h.to(s["x"].dtype) if case["branch_in"] else None, z


def _frames(t, case):
    """sums of a [B, N, C] over the tokens of each frame: [B, F, C]"""
    return t.view(case["B"], case["F"], case["N"] // case["F"], case["C"]).sum(2)


def _norm_grad(g, n, r, kind):
    """gradient through the normalisation of rows, g arriving at n"""
    out = g - n * (g * n).mean(-1, keepdim=True)
    if kind == "layer":
        out = out - g.mean(-1, keepdim=True)
    return out * r


def _plain_gated_norm_backward(s):
    case = s["case"]
    out = dict.fromkeys(("dx", "dy", "dgate", "dscale", "dshift", "dpost_w", "dpost_b", "dpre_w", "dpre_b"))
    dh = s["dh"].float()
    mod = DTYPES[case["mod"]]
    if case["pre"] != "none":
        n, r = _normal_rows(s["h"].float(), case["pre"])
        g = s["dz"].float()
        if case["modulate"]:
            out["dshift"] = _frames(g, case).to(mod)
            out["dscale"] = _frames(g * _affine(n, s["pre_w"], s["pre_b"]), case).to(mod)
            g = g * (1.0 + _by_token(s["scale"], case))
        out["dpre_w"] = (g * n).sum((0, 1)) if s["pre_w"] is not None else None
        out["dpre_b"] = g.sum((0, 1)) if s["pre_b"] is not None else None
        g = g if s["pre_w"] is None else g * s["pre_w"]
        dh = dh + _norm_grad(g, n, r, case["pre"])
        out["dx"] = dh.to(s["dh"].dtype)
    if case["branch_in"]:
        g = dh * case["alpha"]
        m = s["y"].float()
        u, r = _normal_rows(m, case["post"]) if case["post"] != "none" else (m, None)
        if case["gate"]:
            out["dgate"] = _frames(g * _affine(u, s["post_w"], s["post_b"]), case).to(mod)
            g = g * _by_token(s["gate"], case)
        out["dpost_w"] = (g * u).sum((0, 1)) if s["post_w"] is not None else None
        out["dpost_b"] = g.sum((0, 1)) if s["post_b"] is not None else None
        if case["post"] != "none":
            g = g if s["post_w"] is None else g * s["post_w"]
            g = _norm_grad(g, u, r, case["post"])
        out["dy"] = g.to(s["y"].dtype)
    return out


# ------------------------------------------------------------------ one pass


def run(s):
    case = s["case"]
    if not own:
        return {"rotary": _plain_rotary, "rotary_backward": _plain_rotary_backward, "gated_norm": _plain_gated_norm,
                "gated_norm_backward": _plain_gated_norm_backward}[case["op"]](s)
    import block_sparse_attention_mean_gb300 as pkg
    if case["op"] == "rotary":
        q, k, v = s["qkv"]
        return pkg.rotary(s["plan"], q, k, v, positions=s["pos"], norm_eps=1e-6 if case["norm"] else None,
                          q_weight=s["weights"][0], k_weight=s["weights"][1], out=s["out"])
    if case["op"] == "rotary_backward":
        dq, dk, dv = s["grads"]
        q, k, _ = s["qkv"] if case["norm"] else (None, None, None)
        return pkg.rotary_backward(s["plan"], dq, dk, dv, positions=s["pos"], q=q, k=k,
                                   norm_eps=1e-6 if case["norm"] else None, q_weight=s["weights"][0],
                                   k_weight=s["weights"][1], out=s["out"], ws=s["ws"])
    if case["op"] == "gated_norm":
        return pkg.gated_norm(s["x"], s["y"], gate=s["gate"], alpha=case["alpha"], post=s["post"], pre=s["pre"],
                              scale=s["scale"], shift=s["shift"], out=s["out"])
    g = pkg.gated_norm_backward(s["dh"], s["dz"], s["h"], s["y"], gate=s["gate"], alpha=case["alpha"],
                                post=s["post"], pre=s["pre"], scale=s["scale"], shift=s["shift"], out=s["out"],
                                ws=s["ws"])
    return {"dx": g.dx if s["dz"] is not None else None, "dy": g.dy, "dgate": g.dgate, "dscale": g.dscale,
            "dshift": g.dshift, "dpost_w": g.dpost_weight, "dpost_b": g.dpost_bias, "dpre_w": g.dpre_weight,
            "dpre_b": g.dpre_bias}


# ------------------------------------------------------------------ definitions in 64 bits


def _exact_turned(case, s, x, w):
    """[B, heads, N, d] in 64 bits: the pairs as complex numbers, multiplied by exp(i angle)"""
    x = x.double()
    if case["norm"]:
        x = x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6).sqrt()
        x = x * w if w is not None else x
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device).expand(case["N"], len(s["freq"])).contiguous(),
                       s["pos"][:, s["axis"]].double() * s["freq"])[None, :, None]
    p = turn.shape[-1]
    if case["interleaved"]:
        z = torch.view_as_complex(x[..., :2 * p].unflatten(-1, (p, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :p].contiguous(), x[..., p:2 * p].contiguous()) * turn
        head = torch.cat((z.real, z.imag), -1)
    return torch.cat((head, x[..., 2 * p:]), -1).transpose(1, 2)


def _exact_rows(x, kind, w, b):
    if kind == "none":
        return x
    if kind == "layer":
        x = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + 1e-6).sqrt()
    else:
        x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    x = x * w if w is not None else x
    return x + b if b is not None else x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rotary"):
        q, k, v = s["qkv"]
        wq, wk = (None if w is None else w.double().requires_grad_(case["op"] == "rotary_backward") for w in s["weights"])
        if case["op"] == "rotary":
            return (_exact_turned(case, s, q, wq).contiguous(), _exact_turned(case, s, k, wk).contiguous(),
                    v.double().transpose(1, 2).contiguous())
        dq, dk, dv = s["grads"]

        def grads(x, w, dy):
            x = x.double().requires_grad_(True)
            got = torch.autograd.grad(_exact_turned(case, s, x, w), [x] if w is None else [x, w], dy.double())
            return got[0], got[1] if w is not None else None

        gq, gwq = grads(q, wq, dq)
        gk, gwk = grads(k, wk, dk)
        return gq, gk, dv.double().transpose(1, 2).contiguous(), gwq, gwk

    def wide(name):
        t = s.get(name)
        return None if t is None else t.double().requires_grad_(case["op"] == "gated_norm_backward")

    v = {n: wide(n) for n in ("gate", "scale", "shift", "post_w", "post_b", "pre_w", "pre_b", "y")}
    frame = torch.arange(case["N"], device="cuda") // (case["N"] // case["F"])

    def branch():
        u = _exact_rows(v["y"], case["post"], v["post_w"], v["post_b"])
        return case["alpha"] * (u * v["gate"][:, frame] if v["gate"] is not None else u)

    def normed(h):
        z = _exact_rows(h, case["pre"], v["pre_w"], v["pre_b"])
        return z * (1 + v["scale"][:, frame]) + v["shift"][:, frame] if case["modulate"] else z

    if case["op"] == "gated_norm":
        h = s["x"].double() + branch() if case["branch_in"] else s["x"].double()
        return h if case["branch_in"] else None, normed(h) if case["pre"] != "none" else None
    out = dict.fromkeys(("dx", "dy", "dgate", "dscale", "dshift", "dpost_w", "dpost_b", "dpre_w", "dpre_b"))

    def pull(value, arriving, names):
        """gradients of the named tensors (name in v: name of the output)"""
        names = {k: o for k, o in names.items() if v[k] is not None}
        out.update(zip(names.values(), torch.autograd.grad(value, [v[k] for k in names], arriving)))

    dh = s["dh"].double()
    if case["pre"] != "none":
        v["h"] = s["h"].double().requires_grad_(True)
        pull(normed(v["h"]), s["dz"].double(), {"h": "dx", "scale": "dscale", "shift": "dshift", "pre_w": "dpre_w",
                                                "pre_b": "dpre_b"})
        dh = out["dx"] = out["dx"] + dh
    if case["branch_in"]:
        pull(branch(), dh, {"y": "dy", "gate": "dgate", "post_w": "dpost_w", "post_b": "dpost_b"})
    return out
