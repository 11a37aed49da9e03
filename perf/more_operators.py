"""What is measured of the block's projections in 8-bit floating point and of the
update of their weights: the product y = x W^T + b with codes of 8 bits and a
power-of-two scale for each 128 of them (forward alone, or a training step's
share: weights quantised, forward, backward), an update made orthogonal by
Newton-Schulz products, and the whole Muon step over a list of matrices.

``run`` computes a case with the framework's calls where ``own`` is true and
in plain torch operations otherwise; ``exact`` computes it in 64 bits."""

import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _proj(name, op, B, txt, img, n_in, n_out, grad="e4m3"):
    return {"name": name, "op": op, "B": B, "txt": txt, "img": img, "n_in": n_in, "n_out": n_out, "grad": grad}


def _mats(name, op, count, kinds, rows, cols, x="fp32"):
    return {"name": name, "op": op, "count": count, "kinds": kinds, "rows": rows, "cols": cols, "x": x}


def listed():
    return [
        # the modulation projection of one sample's conditioning vector: one token, six outputs of the width
        _proj("fp8-one-token", "fwd", 1, 0, 1, 2560, 15360),
        # a short prompt through the second projection of an MLP: few tokens, long sums
        _proj("fp8-13-tokens", "fwd", 1, 13, 0, 10240, 2560),
        # a 1024 x 1024 guidance pair through the QKV projection
        _proj("fp8-qkv-1024", "fwd", 2, 256, 4096, 2560, 7680),
        # four samples at 1328 x 1328 through the first projection of an MLP: the largest product
        _proj("fp8-mlp-1328", "fwd", 4, 256, 6889, 2560, 10240),
        # short prompts and a small odd grid in training, gradients in the format with the wide range
        _proj("fp8-train-ragged", "train", 3, 77, 513, 1168, 2600, grad="e5m2"),
        # the guidance pair's QKV projection in training
        _proj("fp8-train-1024", "train", 2, 256, 4096, 2560, 7680),
        # one adapter matrix of rank 16
        _mats("orthogonal-adapter", "orth", 1, 1, 16, 1160),
        # one attention output projection's update
        _mats("orthogonal-2560", "orth", 1, 1, 2560, 2560, x="bf16"),
        # a fine-tune's adapters: many small matrices of odd sizes, tall and wide
        _mats("muon-adapters", "muon", 64, 8, 64, 2567),
        # the QKV and output projections of both streams of one block
        _mats("muon-attention", "muon", 4, 2, 2560, 7680, x="bf16"),
        # the MLP projections of two blocks: the largest update
        _mats("muon-mlp", "muon", 4, 1, 2560, 10240, x="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        op = rng.choice(["orth", "muon"])
        while True:
            c = _mats("", op, _log(rng, 1, 64), rng.randint(1, 8), _log(rng, 1, 4000), _log(rng, 1, 10240),
                      x=rng.choice(["bf16", "fp32"]))
            c["kinds"] = min(c["kinds"], c["count"])
            sizes = _shapes(c)
            if sum(r * k for r, k in sizes) <= 100_000_000 and sum(_products(r, k) for r, k in sizes) <= 4.3e12:
                break
    else:
        op = rng.choice(["fwd", "fwd", "train"])
        while True:
            c = _proj("", op, rng.randint(1, 8), rng.choice([0, _log(rng, 1, 512)]), _log(rng, 1, 8192),
                      16 * _log(rng, 4, 640), 8 * _log(rng, 8, 1920), grad=rng.choice(["e4m3", "e5m2"]))
            tokens = c["B"] * (c["txt"] + c["img"])
            if tokens * c["n_in"] * c["n_out"] <= (7e11 if op == "fwd" else 1.7e11) and tokens * (c["n_in"] + c["n_out"]) <= 3.6e8:
                break
    del c["name"]
    return c


def _shapes(c):
    """(rows, columns) of a list's matrices: ``kinds`` different ones in turn,
    the first as given, every other one turned over."""
    part = lambda j, n, k: n if j == 0 else max(1, int(n * (0.3 + 0.7 * ((k * j) % 1.0))))  # noqa: E731
    kinds = [(part(j, c["rows"], 0.618034), part(j, c["cols"], 0.414214)) for j in range(c["kinds"])]
    return [kinds[i % c["kinds"]][::-1 if i % c["kinds"] % 2 else 1] for i in range(c["count"])]


# ------------------------------------------------------------------ inputs
LR, MOMENTUM, DECAY, UPDATE_RMS = 2e-4, 0.95, 0.01, 0.2
ITERATIONS, POLY, TINY = 5, (3.4445, -4.7750, 2.0315), 1e-7
PAD = 512


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows(g, B, T, C, size=1.0):
    """A projection's input rows: channels of unlike sizes, a few far larger."""
    ch = torch.exp(0.5 * torch.randn(C, generator=g, device=DEV))
    ch = torch.where(torch.rand(C, generator=g, device=DEV) < 0.01, 20.0 * ch, ch)
    return (torch.randn((B, T, C), generator=g, device=DEV) * ch * size).to(BF16)


def _prepare_proj(c, seed):
    g = _gen(seed)
    s = {"case": c}
    live = [T > 0 for T in (c["txt"], c["img"])]
    pair = lambda make: tuple(make(T) if on else None for T, on in zip((c["txt"], c["img"]), live))  # noqa: E731
    s["w"] = pair(lambda T: (torch.randn((c["n_out"], c["n_in"]), generator=g, device=DEV) / math.sqrt(c["n_in"])).to(BF16))
    s["bias"] = pair(lambda T: (0.1 * torch.randn(c["n_out"], generator=g, device=DEV)).to(BF16))
    s["x"] = pair(lambda T: _rows(g, c["B"], T, c["n_in"]))
    if c["op"] == "train":
        # gradients of a mean loss: small, tokens of unlike sizes
        s["dy"] = pair(lambda T: (1e-4 * torch.randn((c["B"], T, c["n_out"]), generator=g, device=DEV)
                                  * torch.exp(torch.randn((c["B"], T, 1), generator=g, device=DEV))).to(BF16))
    if own:
        import invariant_mmdit_joint_gb300 as pkg
        s["op"] = pkg.Fp8Projection(c["B"], c["txt"], c["img"], c["n_in"], c["n_out"], grad_format=c["grad"], device=DEV)
        s["op"].set_weights(s["w"])
    elif c["op"] == "fwd":
        s["w8"] = tuple(None if w is None else _blocks(w, 128, 128, "e4m3") for w in s["w"])  # what a server keeps
    return s


def _prepare_mats(c, seed):
    g = _gen(seed)
    s = {"case": c}
    dtype = BF16 if c["x"] == "bf16" else F32

    def grad(r, k):  # noise under a few strong directions
        low = torch.randn((r, 4), generator=g, device=DEV) @ torch.randn((4, k), generator=g, device=DEV)
        return (1e-3 * (torch.randn((r, k), generator=g, device=DEV) + low)).to(dtype)

    shapes = _shapes(c)
    s["g"] = [grad(r, k) for r, k in shapes]
    if c["op"] == "muon":
        starts = [0]
        for r, k in shapes:  # matrices in one buffer of each kind, at multiples of PAD
            starts.append(starts[-1] + -(-r * k // PAD) * PAD)
        s["flat"] = {"p": 0.02 * torch.randn(starts[-1], generator=g, device=DEV),  # the weights in fp32
                     "m": 1e-3 * torch.randn(starts[-1], generator=g, device=DEV)}
        s["flat"]["p16"] = s["flat"]["p"].to(BF16)
        for k, t in s["flat"].items():
            s[k] = [t[a:a + n[0] * n[1]].view(n) for a, n in zip(starts, shapes)]
        s["share"] = [1.0 if i % 2 == 0 else 0.5 for i in range(len(shapes))]
        if own:
            import invariant_mmdit_joint_gb300 as pkg
            s["op"] = pkg.Muon(s["p16"], masters=s["p"], lr=LR, momentum=MOMENTUM, nesterov=True, weight_decay=DECAY,
                               lr_scale=s["share"], update_rms=UPDATE_RMS, iterations=ITERATIONS, coefficients=POLY,
                               eps=TINY, grads=s["g"], m=s["m"])
    return s


def prepare(case, seed):
    return _prepare_proj(case, seed) if case["op"] in ("fwd", "train") else _prepare_mats(case, seed)


# ------------------------------------------------------------------ plain forms
def _power(e):
    """2^e as fp32 for whole e in -126 .. 127."""
    return ((e + 127) << 23).view(F32)


def _blocks(x, tall, wide, kind):
    """fp32 values of x [rows, columns] after rounding to 8-bit codes with one
    power-of-two scale for each block of tall x wide: the smallest that
    brings the block's largest magnitude within the codes' largest."""
    rows, cols = x.shape
    dtype, room = (torch.float8_e4m3fn, 8) if kind == "e4m3" else (torch.float8_e5m2, 15)
    up = lambda n, k: -(-n // k) * k  # noqa: E731
    v = torch.nn.functional.pad(x.float(), (0, up(cols, wide) - cols, 0, up(rows, tall) - rows))
    v = v.view(v.shape[0] // tall, tall, v.shape[1] // wide, wide)
    top = v.abs().amax((1, 3), keepdim=True)
    # 1.75 * 2^room is the largest code: exponent of top, one more above 1.75 of its power of two
    e = ((top.view(torch.int32) + 0x1FFFFF) >> 23) - 127 - room
    e = e.clamp(-126, 126)
    v = (v * _power(-e)).to(dtype).float() * _power(e)
    return v.reshape(up(rows, tall), up(cols, wide))[:rows, :cols]


def _fwd(x, w8, bias):
    y = _blocks(x.reshape(-1, x.shape[-1]), 1, 128, "e4m3") @ w8.t() + bias.float()
    return y.to(BF16).view(*x.shape[:-1], w8.shape[0])


def _train(c, x, dy, w, bias):
    w8 = _blocks(w, 128, 128, "e4m3")
    rows, grads = x.reshape(-1, x.shape[-1]), dy.reshape(-1, dy.shape[-1])
    dx = _blocks(grads, 1, 128, c["grad"]) @ w8
    # the weights' gradient sums over tokens: its operands' blocks run along them
    dw = _blocks(grads, 128, 1, c["grad"]).t() @ _blocks(rows, 128, 1, "e4m3")
    return {"y": _fwd(x, w8, bias), "dx": dx.to(BF16).view(x.shape), "dw": dw, "db": grads.float().sum(0)}


def _both(streams):
    """The two streams' results as (text, image) pairs by name."""
    names = sorted({k for d in streams if d is not None for k in d})
    return {k: tuple(None if d is None else d[k] for d in streams) for k in names}


def _plain_proj(s):
    c = s["case"]
    if c["op"] == "fwd":
        return {"y": tuple(None if x is None else _fwd(x, w, b) for x, w, b in zip(s["x"], s["w8"], s["bias"]))}
    return _both([None if x is None else _train(c, x, dy, w, b)
                  for x, dy, w, b in zip(s["x"], s["dy"], s["w"], s["bias"])])


def _newton_schulz(u):
    x = u.float()
    x = x / (torch.sqrt((x * x).sum()) + TINY)
    turned = x.shape[0] > x.shape[1]
    if turned:
        x = x.t()
    a, b, c = POLY
    for _ in range(ITERATIONS):
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t() if turned else x


def _muon(s):
    def one(p, p16, m, g, share):
        g = g.float()
        m.mul_(MOMENTUM).add_(g)
        o = _newton_schulz(g + MOMENTUM * m)
        rate = LR * share
        p.sub_(rate * DECAY * p + (rate * UPDATE_RMS * math.sqrt(max(p.shape))) * o)
        p16.copy_(p)
    for args in zip(s["p"], s["p16"], s["m"], s["g"], s["share"]):
        one(*args)
    return s["flat"]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        if op == "fwd":
            return {"y": s["op"].forward(s["x"], s["bias"])["y"]}
        if op == "train":
            s["op"].set_weights(s["w"])
            f = s["op"].forward(s["x"], s["bias"], train=True)
            b = s["op"].backward(s["dy"], f)
            return {"y": f["y"], "dx": b["dx"], "dw": b["dw"], "db": b["db"]}
        if op == "orth":
            import invariant_mmdit_joint_gb300 as pkg
            return pkg.orthogonalize(s["g"], iterations=ITERATIONS, coefficients=POLY, eps=TINY)
        s["op"].step()
        return s["flat"]
    if op in ("fwd", "train"):
        return _plain_proj(s)
    if op == "orth":
        return [_newton_schulz(g).to(BF16) for g in s["g"]]
    return _muon(s)


# ------------------------------------------------------------------ work
def _products(r, k):
    """Operations of Newton-Schulz on [r, k]: the two symmetric products count one triangle."""
    r, k = min(r, k), max(r, k)
    return ITERATIONS * (r * (r + 1) * k + r * (r + 1) * r + 2 * r * r * k)


def work(case):
    c = case
    if c["op"] in ("orth", "muon"):
        sizes = _shapes(c)
        n, x = sum(r * k for r, k in sizes), 2 if c["x"] == "bf16" else 4
        # read the gradient, write the update; or gradient, momentum and weight read, the latter two and bf16 written
        return {"bytes": n * (x + (2 if c["op"] == "orth" else 18)), "flops": sum(_products(r, k) for r, k in sizes)}
    n_in, n_out, streams = c["n_in"], c["n_out"], (c["txt"] > 0) + (c["img"] > 0)
    tokens = c["B"] * (c["txt"] + c["img"])
    product = 2 * tokens * n_in * n_out
    if c["op"] == "fwd":  # weights in 8 bits
        return {"bytes": 2 * tokens * (n_in + n_out) + streams * n_in * n_out, "flops": product}
    return {"bytes": 4 * tokens * (n_in + n_out) + streams * n_in * n_out * (2 + 4), "flops": 3 * product}


# ------------------------------------------------------------------ exact
def _power64(e):
    """2^e, of which no library's power function may miss the last bit: halfway cases are many."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _coded(x, tall, wide, kind):
    """x (64 bits) on the grid of its blocks' codes, from the format: q significant
    bits down to the format's smallest step, halfway cases to even."""
    digits, low, top = (3, -6, 448.0) if kind == "e4m3" else (2, -14, 57344.0)
    out = torch.zeros_like(x)
    rows, cols = x.shape
    pad = torch.zeros((-(-rows // tall) * tall, -(-cols // wide) * wide), dtype=F64, device=x.device)
    pad[:rows, :cols] = x
    t = pad.unfold(0, tall, tall).unfold(1, wide, wide)  # [row blocks, column blocks, tall, wide]
    most = t.abs().amax((2, 3))
    _, e = torch.frexp(torch.where(most > 0, most, torch.ones_like(most)) / top)
    scale = _power64(e)  # most / top in [scale / 2, scale)
    scale = torch.where(most / top <= scale / 2, scale / 2, scale)
    scale = scale.clamp_min(2.0 ** -126)[:, :, None, None]
    v = t / scale
    _, k = torch.frexp(torch.where(v == 0, torch.full_like(v, 2.0 ** low), v))
    step = _power64(torch.clamp(k - 1, min=low) - digits)
    v = torch.round(v / step) * step * scale
    out.copy_(v.permute(0, 2, 1, 3).reshape(pad.shape)[:rows, :cols])
    return out


def _exact_proj(c, s):
    def one(i):
        if s["x"][i] is None:
            return None
        x, w, b = (s[k][i].to(F64) for k in ("x", "w", "bias"))
        rows, w = x.reshape(-1, c["n_in"]), _coded(w, 128, 128, "e4m3")
        res = {"y": (_coded(rows, 1, 128, "e4m3") @ w.t() + b).view(*x.shape[:-1], -1)}
        if c["op"] == "train":
            dy = s["dy"][i].to(F64).reshape(-1, c["n_out"])
            res["dx"] = (_coded(dy, 1, 128, c["grad"]) @ w).view(x.shape)
            res["dw"] = _coded(dy, 128, 1, c["grad"]).t() @ _coded(rows, 128, 1, "e4m3")
            res["db"] = dy.sum(0)
        return res
    return _both([one(0), one(1)])


def _exact_orthogonal(u):
    if u.shape[0] > u.shape[1]:
        return _exact_orthogonal(u.mT).mT
    x = u / (torch.linalg.vector_norm(u) + TINY)
    a, b, c = POLY
    eye = torch.eye(u.shape[0], dtype=F64, device=u.device)
    for _ in range(ITERATIONS):
        s = torch.mm(x, x.mT)
        x = torch.mm(a * eye + torch.mm(b * eye + c * s, s), x)
    return x


def exact(case, seed):
    c = case
    if c["op"] in ("fwd", "train"):
        if 2 * c["B"] * (c["txt"] + c["img"]) * c["n_in"] * c["n_out"] * (3 if c["op"] == "train" else 1) > 2e13:
            return None
        return _exact_proj(c, prepare(c, seed))
    s = prepare(c, seed)
    if c["op"] == "orth":
        return [_exact_orthogonal(g.to(F64)) for g in s["g"]]
    out = {k: t.to(F64) for k, t in s["flat"].items()}
    at = 0
    for p, m, g, share in zip(s["p"], s["m"], s["g"], s["share"]):
        g, rate = g.to(F64), LR * share
        m = MOMENTUM * m.to(F64) + g
        o = _exact_orthogonal(g + MOMENTUM * m)
        p = p.to(F64) * (1.0 - rate * DECAY) - rate * UPDATE_RMS * math.sqrt(max(p.shape)) * o
        for k, t in (("p", p), ("p16", p), ("m", m)):
            out[k][at:at + t.numel()] = t.flatten()
        at += -(-p.numel() // PAD) * PAD
    return out
