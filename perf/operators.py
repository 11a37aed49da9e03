"""What is measured of the operators around the block's projections: the
modulated norm before a block, the gate, residual and norm after it (each
forward and backward), and the optimiser step (global gradient norm, AdamW
with 32-bit or 8-bit states over a list of tensors).

``run`` computes a case with the framework's calls where ``own`` is true and
in plain torch operations otherwise; ``exact`` computes it in 64 bits."""

import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "fp32": F32}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _acts(name, op, B, txt, img, C, norm="layer", post="none", x="bf16", y="bf16", mod="bf16", weights=False, alpha=1.0):
    return {"name": name, "op": op, "B": B, "txt": txt, "img": img, "C": C, "norm": norm, "post": post, "x": x, "y": y,
            "mod": mod, "weights": weights, "alpha": alpha}


def listed():
    return [
        # the smallest image of the test workloads, 8 x 8 tokens with 16 text tokens: launch latency
        _acts("modulation-fwd-8x8", "mod_fwd", 1, 16, 64, 256),
        # a 1024 x 1024 guidance pair: both streams' norm before the QKV projection
        _acts("modulation-fwd-1024", "mod_fwd", 2, 256, 4096, 2560),
        # a small odd grid with short prompts, RMS norm with learned weights over an fp32 residual stream
        _acts("modulation-bwd-ragged", "mod_bwd", 3, 77, 513, 1160, norm="rms", x="fp32", weights=True, mod="fp32"),
        # the same pair as above, in training
        _acts("modulation-bwd-1024", "mod_bwd", 2, 256, 4096, 2560),
        # one image row of tokens without text: the shortest residual step
        _acts("gate-fwd-13-tokens", "gate_fwd", 1, 0, 13, 512),
        # four samples at 1328 x 1328 (83 x 83 tokens), norms on both sides of the sublayer
        _acts("gate-fwd-1328-sandwich", "gate_fwd", 4, 256, 6889, 1920, norm="rms", post="rms", weights=True, alpha=0.5),
        # a ragged training batch with the residual stream kept in fp32, norms on both sides
        _acts("gate-bwd-ragged", "gate_bwd", 5, 41, 1365, 1096, post="rms", x="fp32", weights=True, alpha=0.7),
        # four samples at 1328 x 1328 in training: the largest activation pass
        _acts("gate-bwd-1328", "gate_bwd", 4, 256, 6889, 2560),
        # only the gains and norm weights are trained: a few small tensors, clipped
        {"name": "adamw-gains", "op": "adamw", "bits": 32, "wide": 0, "fine": 12, "least": 128, "most": 2560, "clip": True},
        # a fine-tune's adapter matrices: many tensors of odd sizes, 8-bit states
        {"name": "adamw-8bit-many", "op": "adamw", "bits": 8, "wide": 120, "fine": 60, "least": 1000, "most": 400000, "clip": False},
        # the projections of one block in both streams (8 matrices), clipped, 32-bit states
        {"name": "adamw-32bit-block", "op": "adamw", "bits": 32, "wide": 8, "fine": 12, "least": 2560, "most": 13107200, "clip": True},
        # the projections of several blocks, 8-bit states: the largest optimiser pass
        {"name": "adamw-8bit-blocks", "op": "adamw", "bits": 8, "wide": 32, "fine": 24, "least": 2048, "most": 12582913, "clip": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        bits = rng.choice([8, 32])
        most = _log(rng, 3000, 6000000)
        return {"op": "adamw", "bits": bits, "wide": rng.randint(0, 24), "fine": rng.randint(1, 24),
                "least": _log(rng, 1, 2000), "most": most, "clip": bits == 32 and rng.random() < 0.6}
    while True:
        B, txt, img = rng.randint(1, 8), rng.choice([0, _log(rng, 1, 512)]), _log(rng, 1, 8192)
        C = 8 * _log(rng, 8, 640)
        if B * (txt + img) * C <= 60_000_000:
            break
    op = rng.choice(["mod_fwd", "mod_bwd", "gate_fwd", "gate_bwd"])
    x, y = rng.choice([("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
    c = _acts("", op, B, txt, img, C, norm=rng.choice(["layer", "rms"]),
              post=rng.choice(["none", "rms", "layer"]) if op.startswith("gate") else "none", x=x, y=y,
              mod=rng.choice(["bf16", "fp32"]), weights=rng.random() < 0.5,
              alpha=round(rng.uniform(0.3, 1.5), 3) if op.startswith("gate") else 1.0)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
EPS = 1e-6
LR, BETAS, ADAM_EPS, STEP, SEED, MAX_NORM = 2e-4, (0.9, 0.95), 1e-8, 57, 1234567, 1.0
PAD = 512  # tensors of a list start at multiples of this in their flat buffer


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _sizes(c):
    """Element counts of a list's tensors: bf16 matrices with an fp32 master
    first (``wide`` of them, up to ``most``), then fp32 vectors (``fine``)."""
    at = lambda i: (0.618034 * (i + 1)) % 1.0  # noqa: E731
    spread = lambda i, lo, hi: int(round(lo * (hi / lo) ** at(i)))  # noqa: E731
    wide = [spread(i, max(c["least"], c["most"] // 9), c["most"]) for i in range(c["wide"])]
    return wide, [spread(i, c["least"], min(c["most"], 8 * c["least"])) for i in range(c["fine"])]


def _layout(c):
    wide, fine = _sizes(c)
    sizes = wide + fine
    starts, n = [], 0
    for s in sizes:
        starts.append(n)
        n += -(-s // PAD) * PAD
    n_wide = starts[len(wide)] if fine else n
    return sizes, starts, n, n_wide, len(wide)


def _activation(g, B, T, C, dtype, size=1.0):
    """A residual stream's values: channels of unlike sizes, a few far larger."""
    ch = torch.exp(0.5 * torch.randn(C, generator=g, device=DEV))
    ch = torch.where(torch.rand(C, generator=g, device=DEV) < 0.01, 20.0 * ch, ch)
    return ((torch.randn((B, T, C), generator=g, device=DEV) + 0.2) * ch * size).to(dtype)


def _prepare_norm(c, seed):
    g = _gen(seed)
    xt, yt, mt = TYPES[c["x"]], TYPES[c["y"]], TYPES[c["mod"]]
    B, C, gate, bwd = c["B"], c["C"], c["op"].startswith("gate"), c["op"].endswith("bwd")
    s = {"case": c, "n": []}
    for T in (c["txt"], c["img"]):
        if T == 0:
            s["n"].append(None)
            continue
        # the modulation projection's output: scale, shift, gate as columns of one tensor
        mod = (0.3 * torch.randn((B, 3 * C), generator=g, device=DEV)).to(mt)
        d = {"scale": mod[:, :C], "shift": mod[:, C:2 * C], "gate": mod[:, 2 * C:], "w": None, "w_post": None}
        if c["weights"]:
            d["w"] = 0.5 + torch.rand(C, generator=g, device=DEV)
        if gate and c["post"] != "none":
            d["w_post"] = 0.5 + torch.rand(C, generator=g, device=DEV)
        d["x"] = _activation(g, B, T, C, xt)
        if gate:
            d["h"] = _activation(g, B, T, C, yt, 0.5)
        if bwd:
            d["dy"] = torch.randn((B, T, C), generator=g, device=DEV).to(yt)
            d["dr"] = torch.randn((B, T, C), generator=g, device=DEV).to(xt)
            # what the forward left: statistics of the normalised rows (mean, 1 / deviation)
            d["stats"] = torch.stack(_stats(d["x"], c["norm"])[1:], -1).reshape(B, T, 2).contiguous()
            if c["post"] != "none":
                d["post_stats"] = torch.stack(_stats(d["h"], c["post"])[1:], -1).reshape(B, T, 2).contiguous()
        s["n"].append(d)
    for key in ("x", "h", "gate", "scale", "shift", "w", "w_post", "dy", "dr", "stats", "post_stats"):
        s[key] = tuple(None if d is None else d.get(key) for d in s["n"])  # (text, image)
    if own:
        import invariant_mmdit_joint_gb300 as pkg
        op = pkg.AdaLN(B, c["txt"], c["img"], C, norm=c["norm"], post=c["post"], x_dtype=xt, y_dtype=yt, mod_dtype=mt,
                       eps=EPS, alpha=c["alpha"], device=DEV)
        s["op"], s["out"] = op, None
    return s


def _flat_views(flat, sizes, starts):
    return [flat[a:a + n] for n, a in zip(sizes, starts)]


def _prepare_adamw(c, seed):
    g = _gen(seed)
    sizes, starts, n, n_wide, k = _layout(c)
    dev = torch.zeros(n, device=DEV)
    inside = torch.zeros(n + 1, device=DEV)  # 1 inside a tensor, 0 in the padding
    inside[torch.tensor(starts, device=DEV)] = 1.0
    ends = torch.tensor([a + m for a, m in zip(starts, sizes)], device=DEV)
    inside.index_add_(0, ends, torch.full((len(sizes),), -1.0, device=DEV))
    inside = inside.cumsum(0)[:n]
    del dev
    size = torch.exp(torch.randn(n // PAD, generator=g, device=DEV)).repeat_interleave(PAD) * (1e-3 if c["clip"] else 1e-4)
    grad = torch.randn(n, generator=g, device=DEV) * size * inside
    s = {"case": c, "p": 0.02 * torch.randn(n, generator=g, device=DEV) * inside,
         "g16": grad[:n_wide].to(BF16), "g32": grad[n_wide:].clone()}
    s["p16"] = s["p"][:n_wide].to(BF16)
    m = 0.3 * torch.randn(n, generator=g, device=DEV) * size * inside
    v = (size * inside).square() * torch.rand(n, generator=g, device=DEV) + 0.01 * (size * inside).square()
    if c["bits"] == 8:
        zero = torch.zeros(n, dtype=torch.int64, device=DEV)
        (s["m"], s["ms"]), (s["v"], s["vs"]) = _encode(m, zero, False), _encode(v, zero, True)
    else:
        s["m"], s["v"] = m, v
    # the random numbers' key of each tensor, its decay and its share of the rate
    s["decay"] = [0.01 if i < k else 0.0 for i in range(len(sizes))]
    s["share"] = [1.0 if i < k else 0.5 for i in range(len(sizes))]
    if own:
        import invariant_mmdit_joint_gb300 as pkg
        views = lambda t, a=0, b=len(sizes), d=1, off=0: [  # noqa: E731
            t[(starts[i] - off) // d:(starts[i] - off) // d + -(-sizes[i] // d)] for i in range(a, b)]
        p = views(s["p"])
        state = {"m": views(s["m"]), "v": views(s["v"])}
        if c["bits"] == 8:
            state.update(m_scale=views(s["ms"], d=32), v_scale=views(s["vs"], d=32))
        s["op"] = pkg.AdamW(views(s["p16"], 0, k) + p[k:], masters=p[:k] + [None] * (len(sizes) - k),
                            state_bits=c["bits"], lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=s["decay"],
                            lr_scale=s["share"], seed=SEED, grads=views(s["g16"], 0, k) + views(s["g32"], k, off=n_wide),
                            **state)
    return s


def prepare(case, seed):
    return _prepare_adamw(case, seed) if case["op"] == "adamw" else _prepare_norm(case, seed)


# ------------------------------------------------------------------ plain forms
def _stats(x, kind):
    """fp32 values, mean (0 for an RMS norm) and 1 / deviation of each row."""
    x = x.float()
    mean = x.mean(-1) if kind == "layer" else torch.zeros_like(x[..., 0])
    return x, mean, 1.0 / torch.sqrt((x - mean[..., None]).square().mean(-1) + EPS)


def _hat(x, mean, rstd):
    return (x - mean[..., None]) * rstd[..., None]


def _row(v):
    return v.float()[:, None, :]


def _weight(w):
    return 1.0 if w is None else w


def _modulate(x, d, c):
    xf, mean, rstd = _stats(x, c["norm"])
    y = _hat(xf, mean, rstd) * _weight(d["w"]) * (1.0 + _row(d["scale"])) + _row(d["shift"])
    return {"y": y.to(TYPES[c["y"]]), "stats": torch.stack((mean, rstd), -1)}


def _mod_fwd(d, c):
    return None if d is None else _modulate(d["x"], d, c)


def _gate_fwd(d, c):
    if d is None:
        return None
    u, more = d["h"].float(), {}
    if c["post"] != "none":
        u, mean, rstd = _stats(d["h"], c["post"])
        u, more = _hat(u, mean, rstd) * d["w_post"], {"post_stats": torch.stack((mean, rstd), -1)}
    r = (d["x"].float() + c["alpha"] * _row(d["gate"]) * u).to(TYPES[c["x"]])
    return {"r": r, **_modulate(r, d, c), **more}


def _norm_bwd(e, hat, rstd, kind):
    c1 = e.mean(-1, keepdim=True) if kind == "layer" else 0.0
    return rstd[..., None] * (e - c1 - hat * (e * hat).mean(-1, keepdim=True))


def _mod_bwd(d, c):
    if d is None:
        return None
    mean, rstd = d["stats"][..., 0], d["stats"][..., 1]
    hat, dy, more = _hat(d["x"].float(), mean, rstd), d["dy"].float(), 1.0 + _row(d["scale"])
    dx = d["dr"].float() + _norm_bwd(dy * more * _weight(d["w"]), hat, rstd, c["norm"])
    a = (dy * hat).sum(1)
    out = {"dx": dx, "dscale": a * _weight(d["w"]), "dshift": dy.sum(1)}
    if d["w"] is not None:
        out["dw"] = (more[:, 0] * a).sum(0)
    return out


def _gate_bwd(d, c):
    if d is None:
        return None
    out = _mod_bwd(d, c)
    u = d["h"].float()
    du = c["alpha"] * _row(d["gate"]) * out["dx"]
    if c["post"] == "none":
        dh, share = du, 1.0
    else:
        rstd = d["post_stats"][..., 1]
        u, share = _hat(u, d["post_stats"][..., 0], rstd), d["w_post"]
        dh = _norm_bwd(du * d["w_post"], u, rstd, c["post"])
    s = (out["dx"] * u).sum(1)
    out["dgate"] = c["alpha"] * share * s
    if c["post"] != "none":
        out["dw_post"] = c["alpha"] * (d["gate"].float() * s).sum(0)
    out["dh"] = dh.to(TYPES[c["y"]])
    return out


def _pairs(streams):
    """The two streams' results as (text, image) pairs by name."""
    names = sorted({k for d in streams if d is not None for k in d})
    return {k: tuple(None if d is None else d[k] for d in streams) for k in names}


def _norm(s):
    c = s["case"]
    form = {"mod_fwd": _mod_fwd, "mod_bwd": _mod_bwd, "gate_fwd": _gate_fwd, "gate_bwd": _gate_bwd}[c["op"]]
    out = _pairs([form(d, c) for d in s["n"]])
    if "dx" in out:
        out["dx"] = tuple(None if t is None else t.to(TYPES[c["x"]]) for t in out["dx"])
    return out


def _hash(x):
    """The 32-bit integer hash of Wellons' prospector search ("lowbias32")."""
    low = 0xFFFFFFFF
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & low
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & low
    return x ^ (x >> 16)


def _random(c):
    """32 random bits for every element, from the seed, the step, the tensor's
    place in the list and the element's index in it."""
    sizes, starts, n, _, _ = _layout(c)
    key = torch.arange(len(sizes), device=DEV)
    base = _hash(_hash(_hash(torch.full_like(key, SEED)) ^ STEP) ^ key)
    lengths = torch.tensor(starts[1:] + [n], device=DEV) - torch.tensor(starts, device=DEV)
    at = torch.arange(n, device=DEV) - torch.tensor(starts, device=DEV).repeat_interleave(lengths)
    return _hash((at * 0x9E3779B9 + base.repeat_interleave(lengths)) & 0xFFFFFFFF)


def _bits(x):
    return x.view(torch.int32)


def _encode(x, rand16, positive):
    """Values in blocks of 32 as e4m3 with one power-of-two scale a block,
    rounded up with the probability of the remainder (16 random bits)."""
    top = (_bits(x) & 0x7FFFFFFF).view(-1, 32).amax(1)
    e = ((top + 0x1FFFFF) >> 23).clamp_min(32)  # largest magnitude <= 1.75 * 2^(e - 127)
    y = x.abs().view(-1, 32) * _as_float((262 - e) << 23)[:, None]  # <= 448
    small = y < 2.0 ** -6
    t = torch.where(small, y + 2.0 ** -6, y)
    code = ((_bits(t) + ((rand16.view(-1, 32) << 4) | 8).int()) >> 20) - torch.where(small, 968, 960)
    if positive:
        code = torch.where(x.view(-1, 32) > 0, code.clamp_min(1), code)
    else:
        code = code | torch.where(_bits(x).view(-1, 32) < 0, 128, 0)
    return code.to(torch.uint8).view(-1).view(torch.float8_e4m3fn), (e - 8).to(torch.uint8)


def _as_float(bits):
    return bits.to(torch.int32).view(F32)


def _decode(code, scale):
    return (code.to(F32).view(-1, 32) * _as_float(scale.to(torch.int32) << 23)[:, None]).view(-1)


def _per_element(values, c):
    _, starts, n, _, _ = _layout(c)
    lengths = torch.tensor(starts[1:] + [n], device=DEV) - torch.tensor(starts, device=DEV)
    return torch.tensor(values, device=DEV).repeat_interleave(lengths)


def _scalars():
    return 1.0 - BETAS[0] ** STEP, math.sqrt(1.0 - BETAS[1] ** STEP)


def _adamw(s):
    c = s["case"]
    g = torch.cat((s["g16"].float(), s["g32"]))
    out = {}
    if c["clip"]:
        norm = g.double().square().sum().sqrt().float()
        factor = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
        out["norm"] = torch.stack((norm, factor))
        g = g * factor
    q = c["bits"] == 8
    m, v = (_decode(s["m"], s["ms"]), _decode(s["v"], s["vs"])) if q else (s["m"], s["v"])
    b1, b2 = (torch.tensor(b, device=DEV) for b in BETAS)
    one1, one2 = (torch.tensor(1.0 - b, device=DEV) for b in BETAS)
    m = b1 * m + one1 * g
    v = b2 * v + (one2 * g) * g
    c1, c2 = _scalars()
    rate = LR * _per_element(s["share"], c)
    u = m / (torch.sqrt(v) * (1.0 / c2) + ADAM_EPS)
    s["p"].sub_(rate * _per_element(s["decay"], c) * s["p"] + (rate / c1) * u)
    s["p16"].copy_(s["p"][: s["p16"].numel()])
    if q:
        rand = _random(c)
        for name, value, part in (("m", m, rand & 0xFFFF), ("v", v, rand >> 16)):
            code, scale = _encode(value, part, name == "v")
            s[name].view(torch.uint8).copy_(code.view(torch.uint8))
            s[name + "s"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return {**out, **{k: s[k] for k in ("p", "p16", "m", "v", "ms", "vs") if k in s}}


# ------------------------------------------------------------------ the framework's calls
def _own_norm(s):
    op, kind, w = s["op"], s["case"]["op"], s["w"]
    if kind == "mod_fwd":
        s["out"] = op.modulation(s["x"], s["scale"], s["shift"], w=w, out=s["out"])
    elif kind == "gate_fwd":
        s["out"] = op.gate_residual(s["x"], s["h"], s["gate"], s["scale"], s["shift"], w=w, w_post=s["w_post"], out=s["out"])
    elif kind == "mod_bwd":
        s["out"] = op.modulation_bwd(s["x"], s["scale"], s["stats"], s["dy"], s["dr"], w=w, out=s["out"])
    else:
        s["out"] = op.gate_residual_bwd(s["x"], s["h"], s["gate"], s["scale"], s["stats"], s["dy"], s["dr"], w=w,
                                        w_post=s["w_post"], post_stats=s["post_stats"], out=s["out"])
    return s["out"]


def _own_adamw(s):
    op, out, factor = s["op"], {}, None
    if s["case"]["clip"]:
        out["norm"] = op.grad_norm(MAX_NORM)
        factor = out["norm"][1:]
    op.step(STEP, grad_scale=factor)
    return {**out, **{k: s[k] for k in ("p", "p16", "m", "v", "ms", "vs") if k in s}}


def run(state):
    if state["case"]["op"] == "adamw":
        return _own_adamw(state) if own else _adamw(state)
    return _own_norm(state) if own else _norm(state)


# ------------------------------------------------------------------ work
def work(c):
    if c["op"] == "adamw":
        wide, fine = _sizes(c)
        nw, nf = sum(wide), sum(fine)
        states = 4 * (1 + 1 / 32) if c["bits"] == 8 else 16
        return {"bytes": nw * (2 + 8 + 2 + states) + nf * (4 + 8 + states), "flops": 16.0 * (nw + nf)}
    rows = c["B"] * (c["txt"] + c["img"])
    n, streams = rows * c["C"], (c["txt"] > 0) + (c["img"] > 0)
    x, y, m = (4 if c[k] == "fp32" else 2 for k in ("x", "y", "mod"))
    vec, post = streams * c["B"] * c["C"], c["post"] != "none"
    weights = streams * c["C"] * 4 * (c["weights"] + post)
    row = 8 * rows * (1 + post)
    if c["op"] == "mod_fwd":
        return {"bytes": n * (x + y) + 2 * vec * m + weights + row, "flops": 9.0 * n}
    if c["op"] == "gate_fwd":
        return {"bytes": n * (2 * x + 2 * y) + 3 * vec * m + weights + row, "flops": (12.0 + 8.0 * post) * n}
    if c["op"] == "mod_bwd":
        return {"bytes": n * (3 * x + y) + vec * (m + 8) + 2 * weights + row, "flops": 15.0 * n}
    return {"bytes": n * (3 * x + 3 * y) + vec * (2 * m + 12) + 2 * weights + row, "flops": (20.0 + 10.0 * post) * n}


# ------------------------------------------------------------------ 64 bits
F64 = torch.float64


def _exact_norm(x, kind):
    mean = x.sum(-1, keepdim=True) / x.shape[-1] if kind == "layer" else torch.zeros_like(x[..., :1])
    z = x - mean
    inv = ((z * z).sum(-1, keepdim=True) / x.shape[-1] + EPS) ** -0.5
    return z * inv, mean, inv


def _exact_stream(d, c):
    """One stream of a norm case, gradients by the chain rule on 64-bit values."""
    if d is None:
        return None
    gate, bwd = c["op"].startswith("gate"), c["op"].endswith("bwd")
    D = {k: v.to(F64) for k, v in d.items() if v is not None}
    C = c["C"]
    ones = torch.ones(C, dtype=F64, device=DEV)
    w, wp = D.get("w", ones), D.get("w_post", ones)
    a, b, gt = (D[k].unsqueeze(1) for k in ("scale", "shift", "gate"))
    res = {}
    if not bwd:
        r = D["x"]
        if gate:
            u = D["h"]
            if c["post"] != "none":
                z, mean, inv = _exact_norm(u, c["post"])
                u, res["post_stats"] = z * wp, torch.cat((mean, inv), -1)
            r = r + c["alpha"] * gt * u
            r = r.to(TYPES[c["x"]]).to(F64) if c["x"] == "bf16" else r
            res["r"] = r
        z, mean, inv = _exact_norm(r, c["norm"])
        return {**res, "y": z * w * (1 + a) + b, "stats": torch.cat((mean, inv), -1)}
    z, _, inv = _exact_norm(D["x"], c["norm"])
    e = D["dy"] * (w * (1 + a))
    through = e - z * ((e * z).sum(-1, keepdim=True) / C)
    if c["norm"] == "layer":
        through = through - e.sum(-1, keepdim=True) / C
    dx = D["dr"] + inv * through
    res = {"dx": dx, "dscale": (D["dy"] * z * w).sum(1), "dshift": D["dy"].sum(1)}
    if "w" in D:
        res["dw"] = (D["dy"] * (1 + a) * z).sum((0, 1))
    if gate:
        back = c["alpha"] * gt * dx
        if c["post"] == "none":
            res["dh"], res["dgate"] = back, c["alpha"] * (dx * D["h"]).sum(1)
        else:
            z, _, inv = _exact_norm(D["h"], c["post"])
            f = back * wp
            q = f - z * ((f * z).sum(-1, keepdim=True) / C)
            if c["post"] == "layer":
                q = q - f.sum(-1, keepdim=True) / C
            res["dh"] = inv * q
            res["dgate"] = c["alpha"] * (dx * z * wp).sum(1)
            res["dw_post"] = (back * z).sum((0, 1))
    return res


def _exact_round(x, seed_bits, positive):
    """e4m3 values and block scales of 64-bit values, rounded by the same random bits."""
    blocks, r = x.view(-1, 32), seed_bits.view(-1, 32).to(F64)
    top = blocks.abs().amax(1)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    e = torch.where(top > 1.75 * torch.exp2(e), e + 1, e)
    e = torch.where(top > 0, e, torch.full_like(e, -200)).clamp_min(32 - 127)
    y = blocks.abs() * torch.exp2(8 - e)[:, None]
    step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    q = torch.floor(y / step + (r * 16 + 8) / 2 ** 20) * step
    if positive:
        q = torch.where((blocks > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return (torch.sign(blocks) * q).view(-1), (e + 127 - 8).to(torch.uint8)


def _exact_adamw(c, s):
    g = torch.cat((s["g16"].to(F64), s["g32"].to(F64)))
    out = {}
    if c["clip"]:
        norm = torch.sqrt((g * g).sum())
        factor = min(1.0, MAX_NORM / (float(norm) + 1e-6))
        out["norm"] = torch.tensor([float(norm), factor], dtype=F64, device=DEV)
        g = g * factor
    if c["bits"] == 8:
        m, v = ((s[k].to(F64).view(-1, 32) * torch.exp2(s[k + "s"].to(F64) - 127)[:, None]).view(-1) for k in ("m", "v"))
    else:
        m, v = s["m"].to(F64), s["v"].to(F64)
    m = BETAS[0] * m + (1 - BETAS[0]) * g
    v = BETAS[1] * v + (1 - BETAS[1]) * g * g
    p, share, decay = s["p"].to(F64), _per_element(s["share"], c).to(F64), _per_element(s["decay"], c).to(F64)
    hat_m, hat_v = m / (1 - BETAS[0] ** STEP), v / (1 - BETAS[1] ** STEP)
    p = p - LR * share * (decay * p + hat_m / (torch.sqrt(hat_v) + ADAM_EPS))
    out.update(p=p, p16=p[: s["p16"].numel()])
    if c["bits"] == 8:
        rand = _random(c)
        (out["m"], out["ms"]), (out["v"], out["vs"]) = _exact_round(m, rand & 0xFFFF, False), _exact_round(v, rand >> 16, True)
    else:
        out.update(m=m, v=v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    return _pairs([_exact_stream(d, case) for d in s["n"]])
