"""adaln_modulation and adaln_gate_residual on the GPU against their 64-bit
definitions, forward and backward, within each value's own error bound: the
fp32 bound that comes with the definition, plus half a step of the output's
type (bf16 2^-8, fp32 2^-24, relative)."""

import numpy as np
import pytest

import invariant_mmdit_joint_gb300 as pkg
from oracle import block_ops as O
from tests import _helpers as Hh

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def types(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def half_step(t):
    import torch
    return torch.finfo(t.dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_near(got, ref, where):
    """|got - value| <= bound + half a step of got's type."""
    value, bound = ref
    g = f64(got)
    assert g.shape == value.shape, where
    err = np.abs(g - value)
    tol = bound * (1 + 1e-6) + half_step(got) * (np.abs(value) + bound) + 1e-37
    assert np.all(err <= tol), (where, float(np.max(err / tol)), np.unravel_index(np.argmax(err / tol), err.shape))


class Case:
    """Inputs of one call, (text, image) pairs on the device."""

    def __init__(self, dev, B, txt, img, C, norm="layer", post="none", x="bf16", y="bf16", mod="bf16", weights=True,
                 alpha=0.75, seed=1, offset=0.5, pack=6):
        import torch
        self.__dict__.update(B=B, T=(txt, img), C=C, norm=norm, post=post, alpha=alpha, dev=dev, weights=weights)
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.op = pkg.AdaLN(B, txt, img, C, norm=norm, post=post, x_dtype=types(x), y_dtype=types(y),
                            mod_dtype=types(mod), eps=EPS, alpha=alpha, device=dev)

        def r(*shape):
            return torch.randn(shape, generator=g, device=dev)

        def pair(f):
            return tuple(f(T) if T else None for T in self.T)
        spread = torch.exp(r(C))
        self.x = pair(lambda T: ((r(B, T, C) + offset) * spread).to(types(x)))
        self.h = pair(lambda T: (r(B, T, C) + offset).to(types(y)))
        self.dy = pair(lambda T: r(B, T, C).to(types(y)))
        self.dr = pair(lambda T: r(B, T, C).to(types(x)))
        mods = pair(lambda T: (0.4 * r(B, pack * C)).to(types(mod)))
        self.scale, self.shift, self.gate = (tuple(None if m is None else m[:, i * C:(i + 1) * C] for m in mods)
                                             for i in range(3))
        self.w = pair(lambda T: 0.5 + torch.rand(C, generator=g, device=dev)) if weights else None
        self.w_post = pair(lambda T: 0.5 + torch.rand(C, generator=g, device=dev)) if weights and post != "none" else None

    def np(self, name, i, absent=None):
        pair = getattr(self, name)
        if pair is None or pair[i] is None:
            return np.full(self.C, absent) if name.startswith("w") else np.full((self.B, self.C), absent)
        return f64(pair[i])


SHAPES = [
    # B, text, image tokens, C: one token, one column group, odd counts, a warp's edge, two passes of columns
    (1, 0, 1, 8), (2, 1, 0, 8), (3, 1, 2, 264), (1, 16, 64, 256), (2, 5, 131, 1160), (5, 9, 33, 136),
    (1, 3, 17, 4096), (2, 2, 5, 4104), (1, 1, 3, 8192), (2, 31, 1037, 200),
    # each number of threads at its edges
    (1, 2, 5, 512), (2, 3, 4, 1288), (1, 5, 6, 2048), (2, 1, 3, 2056), (2, 3, 9, 2568),
    (1, 2, 7, 5120), (2, 5, 3, 5128), (1, 3, 6, 6144), (2, 2, 3, 6152),
]
KINDS = [
    dict(norm="layer", post="none", x="bf16", y="bf16", mod="bf16", weights=False, alpha=1.0),
    dict(norm="rms", post="rms", x="bf16", y="bf16", mod="fp32"),
    dict(norm="layer", post="layer", x="fp32", y="bf16", mod="bf16"),
    dict(norm="rms", post="layer", x="fp32", y="fp32", mod="fp32", alpha=-1.25),
    dict(norm="layer", post="rms", x="fp32", y="fp32", mod="bf16", weights=False),
]


def check_stats(got, x, kind, where):
    mean, rstd, me, re = O.stats(x, kind, EPS)
    g = f64(got)
    assert np.all(np.abs(g[..., 0] - mean) <= me + 2 * O.U * np.abs(mean)), where
    assert np.all(np.abs(g[..., 1] - rstd) <= re + 2 * O.U * rstd), where


def check_modulation(c, out, x, i, where):
    y, err, _, _ = O.modulation(x, c.np("scale", i), c.np("shift", i), c.np("w", i, 1.0), c.norm, EPS)
    assert_near(out["y"][i], (y, err), (where, "y"))
    check_stats(out["stats"][i], x, c.norm, where)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "-".join(str(v) for v in k.values()))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(dev, shape, kind):
    c = Case(dev, *shape, **kind)
    # modulation
    m = c.op.modulation(c.x, c.scale, c.shift, w=c.w)
    b = c.op.modulation_bwd(c.x, c.scale, m["stats"], c.dy, c.dr, w=c.w)
    nodr = c.op.modulation_bwd(c.x, c.scale, m["stats"], c.dy, None, w=c.w)
    # gate, residual and the next modulation
    f = c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w=c.w, w_post=c.w_post)
    q = c.op.gate_residual_bwd(f["r"], c.h, c.gate, c.scale, f["stats"], c.dy, c.dr, w=c.w, w_post=c.w_post,
                               post_stats=f.get("post_stats"))
    plain = c.op.gate_residual(c.x, c.h, c.gate, None, None, w_post=c.w_post, want_y=False)
    last = c.op.gate_residual_bwd(f["r"], c.h, c.gate, None, None, None, c.dr, w_post=c.w_post,
                                  post_stats=f.get("post_stats"))
    for i in (0, 1):
        if c.T[i] == 0:
            assert all(v[i] is None for o in (m, b, f, q) for k, v in o.items() if k in ("y", "r", "dx", "dscale"))
            continue
        where = (shape, kind, i)
        x, h, dy, dr = (f64(getattr(c, k)[i]) for k in ("x", "h", "dy", "dr"))
        check_modulation(c, m, x, i, where)
        sc, w, wp, gt = c.np("scale", i), c.np("w", i, 1.0), c.np("w_post", i, 1.0), c.np("gate", i)
        st = f64(m["stats"][i])
        for got, res in ((b, dr), (nodr, 0.0 * dr)):
            ref = O.modulation_backward(x, sc, w, st[..., 0], st[..., 1], dy, res, c.norm)
            assert set(got) == {"dx", "dscale", "dshift"} | ({"dw"} if c.weights else set())
            for k in got:
                assert_near(got[k][i], ref[k], (where, "modulation", k))
        r, err, post = O.residual(x, h, gt, wp, c.post, c.alpha, EPS)
        assert_near(f["r"][i], (r, err), (where, "r"))
        assert Hh.bits_equal(plain["r"][i], f["r"][i])
        r = f64(f["r"][i])
        check_modulation(c, f, r, i, where)
        ps = None
        if c.post != "none":
            check_stats(f["post_stats"][i], h, c.post, where)
            g = f64(f["post_stats"][i])
            ps = (g[..., 0], g[..., 1])
        st = f64(f["stats"][i])
        ref = O.gate_residual_backward(r, h, gt, sc, w, wp, st[..., 0], st[..., 1], ps, dy, dr, c.norm, c.post, c.alpha)
        for k in q:
            assert_near(q[k][i], ref[k], (where, "gate", k))
        ref = O.gate_residual_backward(r, h, gt, sc, w, wp, None, None, ps, None, dr, c.norm, c.post, c.alpha)
        assert set(last) == {"dx", "dh", "dgate"} | ({"dw_post"} if c.w_post else set())
        for k in last:
            assert_near(last[k][i], ref[k], (where, "residual alone", k))


def test_large_mean_and_tiny_variance(dev):
    """Rows far from zero: the variance is taken about the mean, so nothing cancels; constant rows stay finite."""
    import torch
    C = 1024
    c = Case(dev, 1, 0, 4, C, x="fp32", y="fp32", mod="fp32", weights=False)
    x = torch.full((1, 4, C), 1000.0, device=dev)
    x[0, 1] += torch.randn(C, device=dev) * 0.01
    x[0, 2] = 0.0
    x[0, 3, ::2] = -1000.0
    got = c.op.modulation((None, x), c.scale, c.shift)
    xs = f64(x)
    check_modulation(c, got, xs, 1, "offset rows")
    # a constant row is its shift exactly
    for row in (0, 2):
        assert torch.equal(got["y"][1][0, row], c.shift[1][0])


def test_non_finite_rows_stay_in_their_row(dev):
    import torch
    c = Case(dev, 2, 3, 5, 264, post="rms")
    clean = c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w=c.w, w_post=c.w_post)
    x = tuple(t.clone() for t in c.x)
    x[0][1, 2, 7], x[1][0, 0, 0] = float("inf"), float("nan")
    got = c.op.gate_residual(x, c.h, c.gate, c.scale, c.shift, w=c.w, w_post=c.w_post)
    for i, bad in ((0, (1, 2)), (1, (0, 0))):
        assert torch.isnan(got["y"][i][bad]).any()
        keep = torch.ones(got["y"][i].shape[:2], dtype=torch.bool)
        keep[bad] = False
        assert Hh.bits_equal(got["y"][i][keep.to(dev)], clean["y"][i][keep.to(dev)])


@pytest.mark.parametrize("T", [1, 3, 40, 700, 2100, 4100, 6200])
def test_a_sample_does_not_depend_on_its_batch(dev, T):
    """Rows, statistics and per-sample gradients of a sample alone, first and last in a batch: the same bytes."""
    B = 5
    c = Case(dev, B, 0, T, 520, post="rms")
    f = c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w=c.w, w_post=c.w_post)
    q = c.op.gate_residual_bwd(f["r"], c.h, c.gate, c.scale, f["stats"], c.dy, c.dr, w=c.w, w_post=c.w_post,
                               post_stats=f["post_stats"])
    one = pkg.AdaLN(1, 0, T, 520, post="rms", eps=EPS, alpha=c.alpha, device=dev)

    def only(pair, b):
        return (None, pair[1][b:b + 1].contiguous())
    for b in (0, B - 1):
        g = one.gate_residual(*(only(p, b) for p in (c.x, c.h, c.gate, c.scale, c.shift)), w=c.w, w_post=c.w_post)
        for k in f:
            assert Hh.bits_equal(g[k][1][0], f[k][1][b]), k
        p = one.gate_residual_bwd(g["r"], only(c.h, b), only(c.gate, b), only(c.scale, b), g["stats"], only(c.dy, b),
                                  only(c.dr, b), w=c.w, w_post=c.w_post, post_stats=g["post_stats"])
        for k in ("dx", "dh", "dgate", "dscale", "dshift"):
            assert Hh.bits_equal(p[k][1][0], q[k][1][b]), k


def test_streams_are_independent_and_runs_repeat(dev):
    """Text and image in one call give the bytes of each alone, and a second run the first's."""
    c = Case(dev, 2, 77, 300, 640, post="layer")
    both = c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w=c.w, w_post=c.w_post)
    args = dict(w=c.w, w_post=c.w_post)
    grads = [c.op.gate_residual_bwd(both["r"], c.h, c.gate, c.scale, both["stats"], c.dy, c.dr,
                                    post_stats=both["post_stats"], **args) for _ in range(2)]
    for k in grads[0]:
        for i in (0, 1):
            assert Hh.bits_equal(grads[0][k][i], grads[1][k][i]), k
    for i in (0, 1):
        T = [0, 0]
        T[i] = c.T[i]
        one = pkg.AdaLN(2, *T, 640, post="layer", eps=EPS, alpha=c.alpha, device=dev)

        def only(pair):
            return (pair[0], None) if i == 0 else (None, pair[1])
        got = one.gate_residual(*(only(p) for p in (c.x, c.h, c.gate, c.scale, c.shift)), w=only(c.w),
                                w_post=only(c.w_post))
        for k in both:
            assert Hh.bits_equal(got[k][i], both[k][i]), k
        back = one.gate_residual_bwd(got["r"], only(c.h), only(c.gate), only(c.scale), got["stats"], only(c.dy),
                                     only(c.dr), w=only(c.w), w_post=only(c.w_post), post_stats=got["post_stats"])
        for k in back:
            assert Hh.bits_equal(back[k][i], grads[0][k][i]), k


def test_in_place_residual_and_gradient(dev):
    """r may be x and dx may be dr."""
    c = Case(dev, 3, 9, 130, 1160, post="rms")
    a = (c.x, c.h, c.gate, c.scale, c.shift)
    want = c.op.gate_residual(*a, w=c.w, w_post=c.w_post)
    wantb = c.op.gate_residual_bwd(want["r"], c.h, c.gate, c.scale, want["stats"], c.dy, c.dr, w=c.w, w_post=c.w_post,
                                   post_stats=want["post_stats"])
    out = {k: tuple(t.clone() for t in v) for k, v in want.items()}
    out["r"] = c.x
    got = c.op.gate_residual(*a, w=c.w, w_post=c.w_post, out=out)
    assert got["r"][1].data_ptr() == c.x[1].data_ptr()
    outb = {k: tuple(t.clone().zero_() for t in v) for k, v in wantb.items()}
    outb["dx"] = c.dr
    gotb = c.op.gate_residual_bwd(got["r"], c.h, c.gate, c.scale, got["stats"], c.dy, c.dr, w=c.w, w_post=c.w_post,
                                  post_stats=got["post_stats"], out=outb)
    for a, b in ((got, want), (gotb, wantb)):
        for k in b:
            for i in (0, 1):
                assert Hh.bits_equal(a[k][i], b[k][i]), k


def test_absent_modulation_is_the_plain_norm(dev):
    import torch
    c = Case(dev, 2, 4, 21, 136, x="fp32", y="fp32", mod="fp32", weights=False)
    zeros = tuple(torch.zeros_like(s) for s in c.scale)
    ones = tuple(torch.ones_like(s) for s in c.scale)
    a = c.op.gate_residual(c.x, c.h, None, None, None)
    b = c.op.gate_residual(c.x, c.h, ones, zeros, zeros)
    for k in a:
        for i in (0, 1):
            assert torch.equal(a[k][i], b[k][i]), k
    a = c.op.gate_residual_bwd(a["r"], c.h, None, None, a["stats"], c.dy, c.dr)
    b = c.op.gate_residual_bwd(b["r"], c.h, ones, zeros, b["stats"], c.dy, c.dr)
    for k in a:
        for i in (0, 1):
            assert torch.equal(a[k][i], b[k][i]), k


def test_rows_behind_the_tensors_stay(dev):
    """Outputs inside larger buffers: nothing before or behind them is written."""
    import torch
    c = Case(dev, 2, 3, 11, 264, post="rms")
    f = c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w=c.w, w_post=c.w_post)
    q = c.op.gate_residual_bwd(f["r"], c.h, c.gate, c.scale, f["stats"], c.dy, c.dr, w=c.w, w_post=c.w_post,
                               post_stats=f["post_stats"])
    guards = []

    def guarded(t):
        pad = 64
        buf = torch.full((t.numel() + 2 * pad,), -7.5, dtype=t.dtype, device=dev)
        guards.append((buf, pad, t.numel()))
        return buf[pad:pad + t.numel()].view(t.shape)
    out = {k: tuple(guarded(t) for t in v) for k, v in f.items()}
    c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w=c.w, w_post=c.w_post, out=out)
    outb = {k: tuple(guarded(t) for t in v) for k, v in q.items()}
    c.op.gate_residual_bwd(f["r"], c.h, c.gate, c.scale, f["stats"], c.dy, c.dr, w=c.w, w_post=c.w_post,
                           post_stats=f["post_stats"], out=outb)
    for got, want in ((out, f), (outb, q)):
        for k in want:
            for i in (0, 1):
                assert Hh.bits_equal(got[k][i], want[k][i]), k
    for buf, pad, n in guards:
        assert bool((buf[:pad] == -7.5).all()) and bool((buf[pad + n:] == -7.5).all())


def test_graph_replay_and_other_streams(dev):
    import torch
    c, d = (Case(dev, 2, 40, 300, 640, post="rms", seed=s) for s in (3, 4))
    names = ("x", "h", "gate", "scale", "shift", "dy", "dr")

    def step(k, out=None):
        f = c.op.gate_residual(k["x"], k["h"], k["gate"], k["scale"], k["shift"], w=c.w, w_post=c.w_post,
                               out=None if out is None else out[0])
        q = c.op.gate_residual_bwd(f["r"], k["h"], k["gate"], k["scale"], f["stats"], k["dy"], k["dr"], w=c.w,
                                   w_post=c.w_post, post_stats=f["post_stats"], out=None if out is None else out[1])
        return f, q
    ins = [{n: getattr(k, n) for n in names} for k in (c, d)]
    want = [step(k) for k in ins]
    cap = {n: tuple(t.clone() if t.is_contiguous() else t.clone(memory_format=torch.contiguous_format)
                    for t in ins[0][n]) for n in names}
    outs = step(cap)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step(cap, outs)
    torch.cuda.current_stream().wait_stream(s)
    for which in (1, 0, 1):
        for n in names:
            for i in (0, 1):
                cap[n][i].copy_(ins[which][n][i])
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want[which]):
            for k in ref:
                for i in (0, 1):
                    assert Hh.bits_equal(got[k][i], ref[k][i]), (which, k)
    # a stream given by hand, with nothing on the current one to order it
    torch.cuda.synchronize()
    f = c.op.gate_residual(*(ins[0][n] for n in names[:5]), w=c.w, w_post=c.w_post, stream=s)
    s.synchronize()
    for k in f:
        assert Hh.bits_equal(f[k][1], want[0][0][k][1]), k


def test_a_bf16_residual_rounds_its_product(dev):
    """r = bf16(x + round(round(alpha * gate) * h)), so that ties stay ties."""
    import torch
    g = torch.Generator(device=dev).manual_seed(3)
    x, h = (torch.randn(1, 300, 1096, generator=g, device=dev).bfloat16() for _ in range(2))
    gate = (0.4 * torch.randn(1, 1096, generator=g, device=dev)).bfloat16()
    op = pkg.AdaLN(1, 0, 300, 1096, alpha=0.7, device=dev)
    r = op.gate_residual((None, x), (None, h), (None, gate), None, None, want_y=False)["r"][1]
    share = torch.tensor(0.7, device=dev) * gate.float()
    assert Hh.bits_equal(r, (x.float() + share[:, None] * h.float()).bfloat16())


def test_results_on_a_stream_given_by_hand(dev):
    """Buffers the call allocates must not be memory that the current stream still writes."""
    import torch
    c = Case(dev, 2, 40, 900, 1280, seed=5)
    want = c.op.modulation(c.x, c.scale, c.shift)
    grads = c.op.modulation_bwd(c.x, c.scale, want["stats"], c.dy, c.dr)
    again = Case(dev, 2, 40, 900, 1280, seed=5)  # whose workspace does not exist yet
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for run, ref in ((lambda: again.op.modulation(c.x, c.scale, c.shift, stream=s), want),
                     (lambda: again.op.modulation_bwd(c.x, c.scale, want["stats"], c.dy, c.dr, stream=s.cuda_stream), grads)):
        junk = [torch.empty(n, dtype=torch.uint8, device=dev) for n in (2 ** 26, 2 ** 22, 2 ** 22, 2 ** 18, 2 ** 18, 2 ** 14)]
        for _ in range(50):
            for j in junk:
                j.fill_(0x55)
        del j, junk
        got = run()
        torch.cuda.synchronize()
        for k in ref:
            for i in (0, 1):
                assert Hh.bits_equal(got[k][i], ref[k][i]), (k, i)


def test_offsets_past_32_bits(dev):
    """An activation of more than 2^32 bytes and 2^31 elements: the last rows are computed like the first."""
    import torch
    B, T, C = 3, 180_000, 4096
    op = pkg.AdaLN(B, 0, T, C, device=dev)
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    x = torch.empty((B, T, C), dtype=torch.bfloat16, device=dev)
    assert x.numel() > 2 ** 31
    tile = torch.randn((1, 1000, C), generator=g, device=dev).bfloat16()
    for b in range(B):
        for t in range(0, T, 1000):
            x[b, t:t + 1000] = tile[0]
    mod = torch.randn((1, 2 * C), generator=g, device=dev).bfloat16().expand(B, 2 * C).contiguous()
    scale, shift = (None, mod[:, :C]), (None, mod[:, C:])
    out = op.modulation((None, x), scale, shift)
    small = pkg.AdaLN(1, 0, 1000, C, device=dev).modulation((None, tile), (None, mod[:1, :C].contiguous()),
                                                          (None, mod[:1, C:].contiguous()))
    for b, t in ((0, 0), (1, 90_000), (2, T - 1000)):
        assert Hh.bits_equal(out["y"][1][b, t:t + 1000], small["y"][1][0])
    back = op.modulation_bwd((None, x), scale, out["stats"], (None, x), None, out=None)
    sb = pkg.AdaLN(1, 0, 1000, C, device=dev)
    sbk = sb.modulation_bwd((None, tile), (None, mod[:1, :C].contiguous()), small["stats"], (None, tile), None)
    for b, t in ((0, 0), (2, T - 1000)):
        assert Hh.bits_equal(back["dx"][1][b, t:t + 1000], sbk["dx"][1][0])


def test_the_trace_names_the_kernels(dev):
    c = Case(dev, 1, 3, 5, 64)
    with pkg.op_trace() as t:
        m = c.op.modulation(c.x, c.scale, c.shift)
        c.op.modulation_bwd(c.x, c.scale, m["stats"], c.dy, c.dr)
    assert [(r["op"], r["status"], r["kernels"]) for r in t.records] == [
        ("adaln_modulation", 0, ["adaln_fwd_kernel"]),
        ("adaln_modulation backward", 0, ["adaln_bwd_kernel", "adaln_fold_kernel"])]


def test_the_trace_and_the_timing_name_the_weights_kernel(dev):
    """A backward that writes a weight's gradient launches a third kernel, with or without another sum."""
    c = Case(dev, 2, 3, 5, 64, post="rms")
    m = c.op.modulation(c.x, c.scale, c.shift, w=c.w)
    f = c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w_post=c.w_post)
    three = ["adaln_bwd_kernel", "adaln_fold_kernel", "adaln_weight_kernel"]
    pkg.rlk_kernel_timing(True)
    with pkg.op_trace() as t:
        c.op.modulation_bwd(c.x, c.scale, m["stats"], c.dy, c.dr, w=c.w)
        c.op.modulation_bwd(c.x, c.scale, m["stats"], c.dy, c.dr)
        c.op.gate_residual_bwd(f["r"], c.h, c.gate, c.scale, f["stats"], c.dy, c.dr, w_post=c.w_post,
                               post_stats=f["post_stats"])
    counts = {k: pkg.rlk_kernel_timing_read(k)[1] for k in ("adaln_fwd", "adaln_bwd", "adaln_fold", "adaln_weight")}
    pkg.rlk_kernel_timing(False)
    assert [r["kernels"] for r in t.records] == [three, three[:2], three]
    assert counts == {"adaln_fwd": 0, "adaln_bwd": 3, "adaln_fold": 3, "adaln_weight": 2}


def butterfly(x, first):
    """What a sum by exchanges with lanes xor first .. 1 leaves in a lane, fp32."""
    while first:
        x = x + x[..., np.arange(x.shape[-1]) ^ first]
        first //= 2
    return x[..., 0]


@pytest.mark.parametrize("T, rows", [(20, 1), (300, 4), (2500, 8), (4200, 8)])
def test_token_sums_run_in_the_stated_order(dev, T, rows):
    """dshift = sum_t dy bit by bit: rows of a chunk, every 32nd chunk, the runs."""
    f = np.float32
    c = Case(dev, 2, 0, T, 264, x="fp32", y="fp32")
    m = c.op.modulation(c.x, c.scale, c.shift, w=c.w)
    got = c.op.modulation_bwd(c.x, c.scale, m["stats"], c.dy, None, w=c.w)["dshift"][1].cpu().numpy()
    dy = c.dy[1].cpu().numpy()
    chunks = -(-T // rows)
    part = np.zeros((2, chunks, 264), f)
    for t in range(T):
        part[:, t // rows] += dy[:, t]
    runs = np.zeros((2, 32, 264), f)
    for j in range(chunks):
        runs[:, j % 32] += part[:, j]
    want = runs[:, 0]
    for k in range(1, 32):
        want = want + runs[:, k]
    assert want.dtype == f
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("C", [64, 520, 1024, 1032, 2568, 8192])
def test_row_sums_run_in_the_stated_order(dev, C):
    """A LayerNorm row's mean bit by bit: a thread's columns in pairs, its warp's
    mean, the warps' means (times their columns) by exchanges, 1 / C in two parts."""
    f, n = np.float32, 7
    c = Case(dev, 1, 0, n, C, weights=False)
    got = c.op.modulation(c.x, c.scale, c.shift)["stats"][1][0, :, 0].cpu().numpy()
    x = c.x[1][0].float().cpu().numpy()
    groups, per = C // 8, 1 if C <= 1024 else 2
    threads = -(-(-(-groups // per)) // 32) * 32
    held = np.zeros((threads * per, 8), f)
    sums = np.zeros((n, threads), f)
    for j in range(per):
        for t in range(threads):
            at = j * threads + t
            if at >= groups:
                continue
            held[at] = 1
            p = np.zeros((n, 2), f)
            for i in range(4):
                p = p + x[:, 8 * at + 2 * i:8 * at + 2 * i + 2]
            pair = p[:, 0] + p[:, 1]
            sums[:, t] = pair if j == 0 else sums[:, t] + pair
    warps = threads // 32
    width = held.reshape(per, warps, 32 * 8).sum((0, 2))  # columns of a warp
    mean = butterfly(sums.reshape(n, warps, 32), 16) * (f(1) / np.maximum(width, f(1)))
    if warps > 1:
        slots = np.zeros((n, 16), f)
        slots[:, :warps] = mean * width
        s = butterfly(slots, 8)
        inv = f(1) / f(C)
        exact = np.longdouble  # (more bits than a product of two fp32 values has)
        low = f(f(exact(1) - exact(f(C)) * exact(inv))) / f(C)
        mean = (exact(s) * exact(inv) + exact(s * low)).astype(f)
    else:
        mean = mean[:, 0]
    assert mean.dtype == f
    np.testing.assert_array_equal(got, mean)


WIDE = [
    # the last width of each number of columns a thread and threads a CTA, and the first of the next
    1024, 1032, 1288, 2048, 2056, 2560, 2568, 4096, 4104, 5120, 5128, 6144, 6152, 8192]
WIDE_KINDS = [
    dict(norm="layer", post="none", x="bf16", y="bf16", mod="bf16", weights=False, alpha=1.0),
    dict(norm="layer", post="rms", x="bf16", y="bf16", mod="bf16"),
    dict(norm="rms", post="layer", x="fp32", y="bf16", mod="bf16"),
    dict(norm="layer", post="none", x="fp32", y="fp32", mod="fp32", alpha=-1.25),
]


def column_sum(got, terms, shares, where):
    """A sum over tokens in 64 bits on the device: each term has at most six roundings, the sum T + 8, its factor two."""
    import torch
    value = shares * terms.sum(1)
    tol = (terms.shape[1] + 16) * O.U * shares.abs() * terms.abs().sum(1)
    bad = (got.double() - value).abs() > tol + 1e-37
    assert not bool(bad.any()), (where, int(bad.sum()))


@pytest.mark.parametrize("kind", WIDE_KINDS, ids=lambda k: "-".join(str(v) for v in k.values()))
@pytest.mark.parametrize("C", WIDE)
def test_many_rows_of_wide_columns(dev, C, kind):
    """More rows than CTAs, so that each goes through its ring and its exchange
    buffers several times and from sample to sample and stream to stream: every
    row has the bytes of calls of a few rows (one a CTA, which are held against the
    definition above), the column sums are held against 64 bits on the device."""
    import torch
    B, T = 3, (90, 1250 if C <= 2560 else 610)
    c = Case(dev, B, *T, C, **kind)
    m = c.op.modulation(c.x, c.scale, c.shift, w=c.w)
    b = c.op.modulation_bwd(c.x, c.scale, m["stats"], c.dy, c.dr, w=c.w)
    f = c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w=c.w, w_post=c.w_post)
    post = dict(w_post=c.w_post, post_stats=f.get("post_stats"))
    q = c.op.gate_residual_bwd(f["r"], c.h, c.gate, c.scale, f["stats"], c.dy, c.dr, w=c.w, **post)
    last = c.op.gate_residual_bwd(f["r"], c.h, c.gate, None, None, None, c.dr, **post)
    n = 25  # tokens of a sample in a call of few rows
    few = pkg.AdaLN(B, 0, n, C, norm=c.norm, post=c.post, x_dtype=c.op.x_dtype, y_dtype=c.op.y_dtype,
                    mod_dtype=c.op.mod_dtype, eps=EPS, alpha=c.alpha, device=dev)
    for i in (0, 1):
        side = lambda pair: None if pair is None else (None, pair[i])  # noqa: E731
        for t in {0, 17, T[i] // 2, T[i] - n}:
            def some(pair):
                return None if pair is None else (None, pair[i][:, t:t + n].contiguous())
            x, h, dy, dr = (some(p) for p in (c.x, c.h, c.dy, c.dr))
            mods = [side(p) for p in (c.gate, c.scale, c.shift)]
            m1 = few.modulation(x, *mods[1:], w=side(c.w))
            b1 = few.modulation_bwd(x, mods[1], m1["stats"], dy, dr, w=side(c.w))
            f1 = few.gate_residual(x, h, *mods, w=side(c.w), w_post=side(c.w_post))
            p1 = dict(w_post=side(c.w_post), post_stats=f1.get("post_stats"))
            q1 = few.gate_residual_bwd(f1["r"], h, *mods[:2], f1["stats"], dy, dr, w=side(c.w), **p1)
            l1 = few.gate_residual_bwd(f1["r"], h, mods[0], None, None, None, dr, **p1)
            for got, ref, names in ((m, m1, ("y", "stats")), (b, b1, ("dx",)), (f, f1, list(f1)), (q, q1, ("dx", "dh")),
                                    (last, l1, ("dx", "dh"))):
                for k in names:
                    assert Hh.bits_equal(got[k][i][:, t:t + n].contiguous(), ref[k][1]), (i, t, k)
        row = lambda pair, absent: torch.full((B, C), absent, dtype=torch.float64, device=dev) if pair is None \
            else pair[i].double().expand(B, C)  # noqa: E731

        def hat(v, stats):
            s = stats[i].double()
            return (v[i].double() - s[..., :1]) * s[..., 1:]
        w, wp, gate = row(c.w, 1.0), row(c.w_post, 1.0), row(c.gate, 1.0)
        for got, rows, stats in ((b, c.x, m["stats"]), (q, f["r"], f["stats"])):
            z = c.dy[i].double() * hat(rows, stats)
            column_sum(got["dscale"][i], z, w, (i, "dscale"))
            column_sum(got["dshift"][i], c.dy[i].double(), torch.ones_like(w), (i, "dshift"))
            if c.w is not None:
                column_sum(got["dw"][i][None], z.reshape(1, -1, C) * (1 + row(c.scale, 0.0)).repeat_interleave(T[i], 0)[None],
                           w[:1] * 0 + 1, (i, "dw"))
        hh = c.h[i].double() if c.post == "none" else hat(c.h, f["post_stats"])
        # the residual's gradient alone is d itself, and with fp32 rows dx is
        for got, d in ((last, c.dr[i]), (q, q["dx"][i])) if c.op.x_dtype == torch.float32 else ((last, c.dr[i]),):
            z = d.double() * hh
            column_sum(got["dgate"][i], z, c.alpha * wp, (i, "dgate"))
            if c.w_post is not None:
                column_sum(got["dw_post"][i][None], z.reshape(1, -1, C) * gate.repeat_interleave(T[i], 0)[None],
                           w[:1] * 0 + c.alpha, (i, "dw_post"))


def test_forms_that_only_the_c_entries_take(dev):
    """Gradients' rows further apart than C, a backward that wants dw but neither
    dscale nor dshift, dgate alone, weights of one stream alone: the bytes of the class."""
    import torch
    c = Case(dev, 3, 20, 150, 520, post="rms")
    B, C = c.B, c.C
    f = c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w=c.w, w_post=c.w_post)
    want = c.op.gate_residual_bwd(f["r"], c.h, c.gate, c.scale, f["stats"], c.dy, c.dr, w=c.w, w_post=c.w_post,
                                  post_stats=f["post_stats"])
    sums = {"dgate": B, "dscale": B, "dshift": B, "dw": 1, "dw_post": 1}
    stride = 3 * C + 4
    sh = pkg.AdalnShape.from_buffer_copy(c.op.shape)
    sh.mod_stride, sh.dmod_stride = c.scale[0].stride(0), stride
    ws = torch.empty(pkg.rlk_adaln_workspace_bytes(sh), dtype=torch.uint8, device=dev)
    ptr = lambda t: t.data_ptr()  # noqa: E731
    for names in (tuple(sums), ("dw",), ("dw_post",), ("dgate",), ("dshift", "dw_post"), ()):
        io, grad, got = [], [], []
        for i in (0, 1):
            # the three rows of a sample side by side in one buffer
            rows = torch.full((B, stride), -3.0, device=dev)
            outs = {k: rows[:, j * C:(j + 1) * C] for j, k in enumerate(("dgate", "dscale", "dshift"))}
            outs.update(dw=torch.empty(C, device=dev), dw_post=torch.empty(C, device=dev),
                        dx=torch.empty_like(c.x[i]), dh=torch.empty_like(c.h[i]))
            got.append((rows, outs))
            io.append(pkg.AdalnIo(h=ptr(c.h[i]), gate=ptr(c.gate[i]), scale=ptr(c.scale[i]), w=ptr(c.w[i]),
                                  w_post=ptr(c.w_post[i]), r=ptr(f["r"][i]), stats=ptr(f["stats"][i]),
                                  post_stats=ptr(f["post_stats"][i])))
            grad.append(pkg.AdalnGrad(dy=ptr(c.dy[i]), dr=ptr(c.dr[i]), dx=ptr(outs["dx"]), dh=ptr(outs["dh"]),
                                      **{k: ptr(outs[k]) for k in names}))
        pkg.rlk_adaln_gate_residual_bwd(sh, io, grad, ws)
        torch.cuda.synchronize()
        for i, (rows, outs) in enumerate(got):
            for k in ("dx", "dh", *names):
                assert Hh.bits_equal(outs[k].contiguous(), want[k][i]), (names, i, k)
            for k in {"dgate", "dscale", "dshift"} - set(names):
                assert bool((outs[k] == -3.0).all()), (names, i, k)
            assert bool((rows[:, 3 * C:] == -3.0).all())
    # weights of one stream alone: of the other they are 1
    ones = torch.ones(C, device=dev)
    for i in (0, 1):
        alone = lambda pair: tuple(t if j == i else None for j, t in enumerate(pair))  # noqa: E731
        full = lambda pair: tuple(t if j == i else ones for j, t in enumerate(pair))  # noqa: E731
        res = []
        for pick in (alone, full):
            g = c.op.gate_residual(c.x, c.h, c.gate, c.scale, c.shift, w=pick(c.w), w_post=pick(c.w_post))
            res.append((g, c.op.gate_residual_bwd(g["r"], c.h, c.gate, c.scale, g["stats"], c.dy, c.dr, w=pick(c.w),
                                                  w_post=pick(c.w_post), post_stats=g["post_stats"])))
        for a, b in zip(*res):
            assert set(a) == set(b)
            for k in a:
                for j in (0, 1):
                    assert Hh.bits_equal(a[k][j], b[k][j]), (i, k, j)


@pytest.mark.parametrize("T, C, rows", [(5119, 520, 8), (6032, 520, 16), (6032, 512, 8), (4096, 1288, 16)])
def test_chunks_of_long_streams_by_their_rule(dev, T, C, rows):
    """dshift bit by bit on both sides of the rule for narrow rows."""
    f = np.float32
    g = Case(dev, 1, 0, T, C, x="fp32", y="fp32", weights=False)
    m = g.op.modulation(g.x, g.scale, g.shift)
    got = g.op.modulation_bwd(g.x, g.scale, m["stats"], g.dy, None)["dshift"][1][0].cpu().numpy()
    dy = g.dy[1][0].cpu().numpy()
    part = np.zeros((-(-T // rows), C), f)
    for t in range(T):
        part[t // rows] += dy[t]
    runs = np.zeros((32, C), f)
    for j, p in enumerate(part):
        runs[j % 32] += p
    want = runs[0]
    for r in runs[1:]:
        want = want + r
    np.testing.assert_array_equal(got, want)
