"""Projections in 8-bit floating point on the GPU: codes and scales bit by bit
against the format's definition, products and column sums against 64 bits within
a bound derived from the arithmetic, a row's bytes whatever the other rows, and
the class as a training step uses it."""

import ctypes

import numpy as np
import pytest

import invariant_mmdit_joint_gb300 as pkg
from oracle import projection_ops as O
from tests import _helpers as Hh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def f64(t):
    return t.detach().double().cpu().numpy()


def rows_of(dev, rows, cols, seed, dtype="bf16", size=1.0):
    """Channels of unlike sizes, a few zeros and a row of them."""
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = size * torch.randn((rows, cols), generator=g, device=dev) * torch.exp(2 * torch.randn(cols, generator=g, device=dev))
    x[:, cols // 2] = 0.0
    if rows > 3:
        x[2] = 0.0
    return x.bfloat16() if dtype == "bf16" else x


class Codes:
    """A matrix's codes and scales, as a call wrote them."""

    def __init__(self, dev, rows, cols, fill=0xA5):
        import torch
        self.rows, self.cols = rows, cols
        self.q = torch.full((rows, pkg.rlk_fp8_row_bytes(cols)), fill, dtype=torch.uint8, device=dev)
        self.s = torch.full((rows, pkg.rlk_fp8_scale_row_bytes(cols)), fill, dtype=torch.uint8, device=dev)

    def values(self, fmt):
        import torch
        v = self.q[:, :self.cols].view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).double().cpu().numpy()
        return v * np.exp2(np.repeat(self.exponents().astype(np.float64), 128, 1)[:, :self.cols])

    def exponents(self):
        return self.s[:, :-(-self.cols // 128)].cpu().numpy().astype(np.int64) - 127


def quantize(dev, x, fmt="e4m3", square=False, want="qts", stride=None):
    """(as it is, turned, column sums) of one matrix."""
    import torch
    rows, cols = x.shape
    q = Codes(dev, rows, cols) if "q" in want else None
    t = Codes(dev, cols, rows) if "t" in want else None
    sums = torch.full((cols,), 7.0, device=dev) if "s" in want else None
    ws = torch.empty(pkg.rlk_fp8_quant_workspace_bytes(rows, cols), dtype=torch.uint8, device=dev) if "s" in want else None
    p = pkg._ptr
    item = pkg.Fp8Quant(p(x), p(q and q.q), p(q and q.s), p(t and t.q), p(t and t.s), p(sums), p(ws), rows, cols, x.stride(0),
                        int(x.dtype == torch.float32), pkg.FP8_FORMATS[fmt], int(square), 0)
    pkg.rlk_fp8_quantize((pkg.Fp8Quant * 1)(item))
    torch.cuda.synchronize()
    return q, t, sums


def gemm(dev, a, b, fa="e4m3", fb="e4m3", bias=None, dtype=None, out=None, accumulate=False):
    import torch
    dtype = dtype or torch.bfloat16
    d = torch.full((a.rows, b.rows), 7.0, dtype=dtype, device=dev) if out is None else out
    item = pkg.Fp8Product(a.q.data_ptr(), a.s.data_ptr(), b.q.data_ptr(), b.s.data_ptr(), pkg._ptr(bias), d.data_ptr(), a.rows,
                          b.rows, a.cols, d.stride(0), pkg.FP8_FORMATS[fa], pkg.FP8_FORMATS[fb], int(dtype == torch.float32),
                          int(accumulate))
    pkg.rlk_fp8_gemm((pkg.Fp8Product * 1)(item))
    pkg.rlk_joint_attn_check_status()
    return d


def assert_product(got, ref, bound, where=""):
    import torch
    err = np.abs(f64(got) - ref)
    half = torch.finfo(got.dtype).eps / 2
    tol = bound + half * (np.abs(ref) + bound) + 2.0 ** -133
    assert np.all(err <= tol), (where, float(np.max(err / tol)), np.argwhere(err > tol)[:4])


SIZES = [(1, 8), (1, 128), (7, 136), (128, 128), (129, 264), (300, 1000), (257, 2600)]


@pytest.mark.parametrize("rows, cols", SIZES)
@pytest.mark.parametrize("fmt, dtype, square", [("e4m3", "bf16", False), ("e5m2", "fp32", False), ("e4m3", "fp32", True),
                                                ("e5m2", "bf16", True)])
def test_codes(dev, rows, cols, fmt, dtype, square):
    x = rows_of(dev, rows, cols, rows + cols, dtype)
    q, t, sums = quantize(dev, x, fmt, square)
    ref, exps = O.quantize(f64(x), 128 if square else 1, 128, fmt)
    assert np.array_equal(q.values(fmt), ref)
    assert np.array_equal(q.exponents(), np.repeat(exps, 128, 0)[:rows] if square else exps)
    ref, exps = O.quantize(f64(x), 128, 128 if square else 1, fmt)
    assert np.array_equal(t.values(fmt), ref.T)
    assert np.array_equal(t.exponents(), np.repeat(exps, 128, 1)[:, :cols].T if square else exps.T)
    # 8 rows, 16 runs, rows / 128 tiles: that many fp32 additions at most
    tol = np.abs(f64(x)).sum(0) * (8 + 16 + rows / 128) * 2.0 ** -24
    assert np.all(np.abs(f64(sums) - f64(x).sum(0)) <= tol)
    # nothing behind the scales; behind a row's codes nothing, or zeros where turned
    assert bool((q.s[:, -(-cols // 128):] == 0xA5).all()) and bool((t.s[:, -(-rows // 128):] == 0xA5).all())
    assert bool((q.q[:, cols:] == 0xA5).all()) and bool((t.q[:, rows:] == 0).all())


def test_codes_at_the_edges(dev):
    """The largest and smallest magnitudes, halfway cases, infinities and NaN, alone and among others."""
    import torch
    x = torch.zeros((9, 256), device=dev)
    x[0] = torch.linspace(-448, 448, 256, device=dev)
    x[1, :128] = 448.0 * 2.0 ** 100
    x[1, 128:] = torch.tensor(448.0 * 2.0 ** 100, device=dev) * (1 + 2.0 ** -20)  # one power more
    x[2] = 3.0e38
    x[3] = torch.arange(256, device=dev) * 2.0 ** -149
    x[4] = torch.arange(256, device=dev) * 2.0 ** -130
    x[5, 3], x[5, 4:9] = float("inf"), 1.0
    x[6, 200], x[6, 130] = float("nan"), -2.0
    x[7, :] = float("-inf")
    x[8] = (torch.arange(256, device=dev) % 64) * 0.125 + 16.0  # many ties
    for fmt in ("e4m3", "e5m2"):
        for want, tall, wide in (("q", 1, 128), ("t", 128, 1)):
            q, t, _ = quantize(dev, x, fmt, want=want)
            ref, exps = O.quantize(f64(x), tall, wide, fmt)
            got = q if want == "q" else t
            assert np.array_equal(got.values(fmt), ref if want == "q" else ref.T, equal_nan=True), (fmt, want)
            assert np.array_equal(got.exponents(), exps if want == "q" else exps.T)


def test_codes_of_a_strided_view(dev):
    x = rows_of(dev, 40, 512, 5)
    part = x[:, 128:328]
    q, t, _ = quantize(dev, part)
    ref, _ = O.quantize(f64(part), 1, 128)
    assert np.array_equal(q.values("e4m3"), ref)


def operands(dev, m, n, k, seed, fa="e4m3", square=True):
    a, _, _ = quantize(dev, rows_of(dev, m, k, seed), fa, want="q")
    b, _, _ = quantize(dev, rows_of(dev, n, k, seed + 1, size=0.1), square=square, want="q")
    return a, b


@pytest.mark.parametrize("m, n, k", [(1, 8, 8), (1, 136, 512), (16, 128, 520), (17, 256, 1024), (64, 384, 1032), (65, 200, 128),
                                     (224, 128, 2048), (225, 136, 640), (700, 1000, 1160), (3, 128, 5000)])
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
def test_product(dev, m, n, k, fa):
    import torch
    a, b = operands(dev, m, n, k, m + n + k, fa, square=n % 16 == 0)
    bias = torch.randn(n, device=dev).bfloat16()
    va, vb = a.values(fa), b.values("e4m3")
    bound = O.product_bound(va, vb, f64(bias))
    ref = va @ vb.T + f64(bias)
    assert_product(gemm(dev, a, b, fa, bias=bias), ref, bound, "bf16")
    assert_product(gemm(dev, a, b, fa, bias=bias, dtype=torch.float32), ref, bound, "fp32")


@pytest.mark.parametrize("k", [1, 17, 127, 129, 513])
def test_product_of_turned_operands(dev, k):
    """Weights' gradients: the sum over any number of tokens; added to what is there."""
    import torch
    x, dy = rows_of(dev, k, 136, 3), rows_of(dev, k, 72, 4, size=1e-4)
    _, xt, _ = quantize(dev, x, want="t")
    _, yt, _ = quantize(dev, dy, "e5m2", want="t")
    vx, vy = xt.values("e4m3"), yt.values("e5m2")
    dw = gemm(dev, yt, xt, "e5m2", dtype=torch.float32)
    assert_product(dw, vy @ vx.T, O.product_bound(vy, vx), "dw")
    twice = gemm(dev, yt, xt, "e5m2", dtype=torch.float32, out=dw.clone(), accumulate=True)
    assert Hh.bits_equal(twice, dw + dw)


def test_product_into_a_wider_tensor(dev):
    """Rows of d further apart; columns and rows beside it stay as they are."""
    import torch
    a, b = operands(dev, 70, 136, 256, 9)
    big = torch.full((74, 200), 3.0, dtype=torch.bfloat16, device=dev)
    gemm(dev, a, b, out=big[2:72, 32:168])
    assert Hh.bits_equal(big[2:72, 32:168].contiguous(), gemm(dev, a, b))
    big[2:72, 32:168] = 3.0
    assert bool((big == 3.0).all())


def test_a_nan_stays_in_its_row(dev):
    x = rows_of(dev, 20, 256, 11)
    x[4, 7] = float("nan")
    x[9, 200] = float("inf")
    a, _, _ = quantize(dev, x, want="q")
    b, _, _ = quantize(dev, rows_of(dev, 128, 256, 12), square=True, want="q")
    d = f64(gemm(dev, a, b))
    assert np.isnan(d[[4, 9]]).all() and np.isfinite(np.delete(d, [4, 9], 0)).all()


@pytest.mark.parametrize("k", [200, 2560, 10240])
def test_rows_do_not_depend_on_their_number(dev, k):
    """Each width of the accumulator and each split of the sums gives a row the same bytes."""
    import torch
    n = 264
    x = rows_of(dev, 500, k, 21)
    a, b = operands(dev, 500, n, k, 21)
    a, _, _ = quantize(dev, x, want="q")
    full = gemm(dev, a, b, dtype=torch.float32)
    for rows in (slice(0, 1), slice(3, 4), slice(0, 16), slice(5, 22), slice(100, 164), slice(200, 265), slice(499, 500)):
        part, _, _ = quantize(dev, x[rows], want="q")
        assert Hh.bits_equal(gemm(dev, part, b, dtype=torch.float32), full[rows].contiguous()), rows


def test_long_sums_of_few_tokens(dev):
    """K past what the CTAs of a cluster hold for 16 tokens, and for 64."""
    import torch
    for rows, k in ((2, 45056), (2, 45200), (40, 12288), (40, 12400)):
        x, w = rows_of(dev, 300, k, 31), rows_of(dev, 72, k, 32, size=0.1)
        a, _, _ = quantize(dev, x, want="q")
        b, _, _ = quantize(dev, w, square=True, want="q")
        few, _, _ = quantize(dev, x[:rows], want="q")
        got = gemm(dev, few, b, dtype=torch.float32)
        assert Hh.bits_equal(got, gemm(dev, a, b, dtype=torch.float32)[:rows].contiguous()), (rows, k)
        va, vb = few.values("e4m3"), b.values("e4m3")
        assert_product(got, va @ vb.T, O.product_bound(va, vb), (rows, k))


@pytest.mark.parametrize("m, n, k", [(1, 8, 8), (1, 15360, 2560), (16, 136, 12288), (13, 2560, 10240), (5, 264, 1160), (16, 128, 128),
                                     (2, 200, 4104)])
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
def test_few_rows_rounded_on_the_way(dev, m, n, k, fa):
    """bf16 rows as the operand: the bytes of rounding them first."""
    import torch
    x = rows_of(dev, m, k, m + k)
    if m > 2:
        x[1, 3], x[2, k - 1] = float("nan"), float("-inf")
    a, _, _ = quantize(dev, x, fa, want="q")
    b, _, _ = quantize(dev, rows_of(dev, n, k, 7, size=0.1), square=True, want="q")
    bias = torch.randn(n, device=dev).bfloat16()
    for dtype in (torch.bfloat16, torch.float32):
        want = gemm(dev, a, b, fa, bias=bias, dtype=dtype)
        got = torch.full((m, n), 7.0, dtype=dtype, device=dev)
        item = pkg.Fp8Product(x.data_ptr(), None, b.q.data_ptr(), b.s.data_ptr(), bias.data_ptr(), got.data_ptr(), m, n, k, n,
                              pkg.FP8_FORMATS[fa], 0, int(dtype == torch.float32), 0, 1, 0)
        pkg.rlk_fp8_gemm((pkg.Fp8Product * 1)(item))
        pkg.rlk_joint_attn_check_status()
        assert Hh.bits_equal(torch.nan_to_num(got), torch.nan_to_num(want)) and bool((got.isnan() == want.isnan()).all())


def test_places_past_32_bits(dev):
    """An input and an output of more than 2^31 elements: the last rows as if they were alone."""
    import torch
    rows, k = 270000, 8192
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    x = torch.empty((rows, k), dtype=torch.bfloat16, device=dev)
    x[-300:] = torch.randn((300, k), generator=g, device=dev).bfloat16()
    x[:-300] = 0.5
    op, last = (pkg.Fp8Projection(1, 0, t, k, n, device=dev) for t, n in ((rows, 8192), (300, 8192)))
    w = (torch.randn((8192, k), generator=g, device=dev) / k ** 0.5).bfloat16()
    op.set_weights((None, w))
    last.set_weights((None, w))
    y = op.forward((None, x.unsqueeze(0)))["y"][1][0, -300:].clone()
    assert Hh.bits_equal(y, last.forward((None, x[None, -300:].contiguous()))["y"][1][0])
    del op, x
    # (turned operands: column sums over that many rows)
    torch.cuda.empty_cache()


def test_products_of_one_launch(dev):
    """Eight unlike products at once give what each gives alone."""
    import torch
    sizes = [(1, 64, 128), (300, 136, 512), (16, 8, 8), (0, 64, 64), (77, 1000, 640), (5, 256, 2000), (224, 128, 128), (31, 40, 48)]
    ops = [operands(dev, max(m, 1), n, k, i, square=n % 16 == 0) for i, (m, n, k) in enumerate(sizes)]
    alone = [gemm(dev, a, b) for a, b in ops]
    out = [torch.full_like(t, 5.0) for t in alone]
    items = (pkg.Fp8Product * 8)(*[
        pkg.Fp8Product(a.q.data_ptr(), a.s.data_ptr(), b.q.data_ptr(), b.s.data_ptr(), None, o.data_ptr(), m, n, k, n, 0, 0, 0, 0)
        for (a, b), o, (m, n, k) in zip(ops, out, sizes)])
    pkg.rlk_fp8_gemm(items)
    pkg.rlk_joint_attn_check_status()
    for t, o, (m, n, k) in zip(alone, out, sizes):
        assert Hh.bits_equal(o[:m].contiguous(), t[:m].contiguous())
    assert bool((out[3] == 5.0).all())


def make(dev, B, T, n_in, n_out, seed=0, **kw):
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    on = lambda f: tuple(f(t) if t else None for t in T)  # noqa: E731
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    op = pkg.Fp8Projection(B, *T, n_in, n_out, device=dev, **kw)
    w = on(lambda t: (rnd(n_out, n_in) / n_in ** 0.5).bfloat16())
    b = on(lambda t: rnd(n_out).bfloat16())
    x = on(lambda t: rnd(B, t, n_in).bfloat16())
    dy = on(lambda t: (1e-3 * rnd(B, t, n_out)).bfloat16())
    return op, w, b, x, dy


@pytest.mark.parametrize("B, T, n_in, n_out, grad", [(2, (13, 70), 264, 136, "e5m2"), (1, (0, 1), 128, 768, "e4m3"),
                                                     (3, (5, 0), 1160, 72, "e4m3"), (1, (150, 330), 256, 640, "e5m2")])
def test_projection(dev, B, T, n_in, n_out, grad):
    op, w, b, x, dy = make(dev, B, T, n_in, n_out, grad_format=grad)
    op.set_weights(w)
    f = op.forward(x, b, train=True)
    r = op.backward(dy, f)
    pkg.rlk_joint_attn_check_status()
    for i in (0, 1):
        if not T[i]:
            assert f["y"][i] is None and r["dw"][i] is None
            continue
        xv, gv, wv = f64(x[i]).reshape(-1, n_in), f64(dy[i]).reshape(-1, n_out), O.quantize(f64(w[i]), 128, 128)[0]
        x8, g8 = O.quantize(xv, 1, 128)[0], O.quantize(gv, 1, 128, grad)[0]
        xt, gt = O.quantize(xv, 128, 1)[0].T, O.quantize(gv, 128, 1, grad)[0].T
        bias = f64(b[i])
        assert_product(f["y"][i].view(-1, n_out), x8 @ wv.T + bias, O.product_bound(x8, wv, bias), "y")
        assert_product(r["dx"][i].view(-1, n_in), g8 @ wv, O.product_bound(g8, wv.T), "dx")
        assert_product(r["dw"][i], gt @ xt.T, O.product_bound(gt, xt), "dw")
        assert np.all(np.abs(f64(r["db"][i]) - gv.sum(0)) <= np.abs(gv).sum(0) * (24 + len(gv) / 128) * 2.0 ** -24)


def test_projection_gradients_agree_with_differences(dev):
    """dx, dw and db are the derivatives of the rounded product: on values that the codes hold exactly, the product's
    differences are exact."""
    import torch
    n_in, n_out, t = 24, 16, 6
    op = pkg.Fp8Projection(1, 0, t, n_in, n_out, out_dtype=torch.float32, device=dev)
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    whole = lambda *s: torch.randint(-4, 5, s, generator=g, device=dev).bfloat16()  # noqa: E731  (exact in e4m3)
    w, x, dy, b = whole(n_out, n_in), whole(1, t, n_in), whole(1, t, n_out), whole(n_out)
    op.set_weights((None, w))
    f = op.forward((None, x), (None, b), train=True)
    r = op.backward((None, dy), f)

    def loss(x, w, b):
        op.set_weights((None, w))
        return float((op.forward((None, x), (None, b))["y"][1] * dy.float()).sum())
    base = loss(x, w, b)
    for name, t0, grad in (("x", x, r["dx"][1]), ("w", w, r["dw"][1]), ("b", b, r["db"][1])):
        for at in (0, t0.numel() // 3, t0.numel() - 1):
            moved = t0.clone()
            moved.view(-1)[at] += 1.0
            args = {"x": x, "w": w, "b": b, name: moved}
            assert loss(**args) - base == float(grad.reshape(-1)[at]), (name, at)


def test_projection_reuses_and_accumulates(dev):
    op, w, b, x, dy = make(dev, 2, (3, 40), 256, 128)
    op.set_weights(w)
    f = op.forward(x, b, train=True)
    r = op.backward(dy, f)
    again = op.backward(dy, f, out={k: tuple(t.clone() for t in r[k]) for k in r}, accumulate=True)
    for i in (0, 1):
        assert Hh.bits_equal(again["dw"][i], r["dw"][i] * 2) and Hh.bits_equal(again["dx"][i], r["dx"][i])
    only = op.backward(dy, None, want=("db",))
    assert Hh.bits_equal(only["db"][1], r["db"][1]) and set(only) == {"db"}
    y = [t.clone() for t in f["y"]]
    f2 = op.forward(x, b, train=True, out=f)
    assert f2["y"][0] is f["y"][0] and all(Hh.bits_equal(p, q) for p, q in zip(y, f2["y"]))
    assert all(Hh.bits_equal(p, q) for p, q in zip(y, op.forward(x, b)["y"]))


def test_projection_captured_and_on_another_stream(dev):
    import torch
    op, w, b, x, dy = make(dev, 1, (33, 260), 384, 264)
    op.set_weights(w)
    f = op.forward(x, b, train=True)
    r = op.backward(dy, f)
    want = [t.clone() for t in (*f["y"], *r["dx"], *r["dw"], *r["db"])]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        op.set_weights(w)
        op.forward(x, b, train=True, out=f)
        op.backward(dy, f, out=r)
    for _ in range(2):
        for t in (*f["y"], *r["dx"], *r["dw"], *r["db"]):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(Hh.bits_equal(p, q) for p, q in zip(want, (*f["y"], *r["dx"], *r["dw"], *r["db"])))
    f2 = op.forward(x, b, train=True, stream=s)
    r2 = op.backward(dy, f2, stream=s)
    s.synchronize()
    assert all(Hh.bits_equal(p, q) for p, q in zip(want, (*f2["y"], *r2["dx"], *r2["dw"], *r2["db"])))


def test_few_tokens_captured_and_beside_each_other(dev):
    """The product of few tokens starts before the tokens are rounded: captured and replayed on inputs that change, and
    two projections on two streams at once, give what each gives alone."""
    import torch
    made = [make(dev, 1, T, n_in, n_out, seed=i) for i, (T, n_in, n_out) in enumerate((((1, 16), 2560, 1536), ((5, 60), 1160, 4096)))]
    for op, w, *_ in made:
        op.set_weights(w)
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    inputs = [[tuple(torch.randn(t.shape, generator=g, device=dev).bfloat16() for t in x) for _ in range(6)] for _, _, _, x, _ in made]
    want = [[[t.clone() for t in m[0].forward(x, m[2])["y"]] for x in xs] for m, xs in zip(made, inputs)]
    for m, xs, ys in zip(made, inputs, want):
        op, _, b, x, _ = m
        out = op.forward(x, b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                op.forward(x, b, out=out)
        for new, y in zip(xs, ys):
            for t, n in zip(x, new):
                t.copy_(n)
            graph.replay()
            torch.cuda.synchronize()
            assert all(Hh.bits_equal(p, q) for p, q in zip(out["y"], y))
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    got = [[m[0].forward(x, m[2], stream=s)["y"] for x in xs for _ in (0, 1)] for m, xs, s in zip(made, inputs, streams)]
    torch.cuda.synchronize()
    for ys, zs in zip(want, got):
        for i, z in enumerate(zs):
            assert all(Hh.bits_equal(p, q) for p, q in zip(ys[i // 2], z))
    pkg.rlk_joint_attn_check_status()


def test_trace(dev):
    import torch
    op, w, b, x, dy = make(dev, 1, (0, 20), 128, 128)
    op.set_weights(w)
    with pkg.op_trace() as t:
        op.backward(dy, op.forward(x, b, train=True))
        torch.cuda.synchronize()
    assert [(k["entry_point"], k["kernels"]) for k in t.records] == [
        ("rlk_fp8_quantize", ["fp8_quant_kernel"]), ("rlk_fp8_gemm", ["fp8_gemm_kernel"]),
        ("rlk_fp8_quantize", ["fp8_quant_kernel", "fp8_fold_kernel"]), ("rlk_fp8_gemm", ["fp8_gemm_kernel"])]


def test_null_handles_fail(dev):
    assert pkg.lib().rlk_fp8_gemm(None, 1, None) == 1 and pkg.lib().rlk_fp8_quantize(None, 1, None) == 1
    assert pkg.lib().rlk_fp8_gemm((pkg.Fp8Product * 1)(), 0, ctypes.c_void_p()) == 1
