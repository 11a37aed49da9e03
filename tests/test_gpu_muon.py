"""Muon and its orthogonal update on the GPU against 64 bits.

Tolerances: the kernels keep X, A and B in fp16. The oracle runs the same
products with those roundings and without them; their distance d is what storage
alone does, and the kernels' own roundings (halfway cases and fp32 sums that
fall on the other side) are another draw of the same size. So, in the Frobenius
norm, |gpu - exact| <= 2 d + the output's rounding, and no more than the documented
2^-9 |X| beside the output's rounding for matrices like gradients."""

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


def gradient(dev, rows, cols, seed, dtype="fp32", low=4):
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.float64)  # noqa: E731
    x = 1e-3 * (rnd(rows, cols) + rnd(rows, low) @ rnd(low, cols))
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def assert_orthogonal(got, u, where="", half=2.0 ** -9, **kw):
    norm = np.linalg.norm
    exact = O.orthogonal(u, **kw)
    d = norm(O.orthogonal(u, stored=True, **kw) - exact)
    if min(u.shape) <= 16:
        d = max(d, *(norm(O.orthogonal(u, stored=True, lead=f, **kw) - exact) for f in (1.1, 1.23, 1.37, 1.52, 1.71, 1.83, 1.97)))
    err = norm(f64(got) - exact)
    # a value's rounding to bf16 is off by half * 2 at most
    tol = 2 * d + 2 * half * norm(exact) + 1e-30
    assert err <= tol, (where, err / max(norm(exact), 1e-300), d / max(norm(exact), 1e-300))


SHAPES = [(1, 1), (1, 9), (9, 1), (16, 1160), (1160, 16), (64, 64), (130, 70), (128, 256), (257, 300), (300, 257), (520, 264),
          (385, 1025)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_orthogonalize(dev, dtype):
    """Every size of the list at once, and each alone to the byte."""
    import torch
    xs = [gradient(dev, r, c, i, dtype) for i, (r, c) in enumerate(SHAPES)]
    xs += [gradient(dev, 130, 70, 50, dtype), gradient(dev, 70, 130, 51, dtype)]
    got = pkg.orthogonalize(xs)
    pkg.rlk_joint_attn_check_status()
    for x, o in zip(xs, got):
        assert o.dtype == torch.bfloat16
        assert_orthogonal(o, f64(x), tuple(x.shape))
        assert Hh.bits_equal(pkg.orthogonalize([x])[0], o), tuple(x.shape)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 8])
def test_iterations(dev, n):
    x = gradient(dev, 200, 333, n)
    poly = (1.5, -0.5, 0.0) if n == 3 else (3.4445, -4.7750, 2.0315)
    assert_orthogonal(pkg.orthogonalize([x], iterations=n, coefficients=poly)[0], f64(x), n, iterations=n, coefficients=poly)


def test_larger_matrix_within_the_documented_error(dev):
    x = gradient(dev, 768, 1536, 7, "bf16")
    got, exact = f64(pkg.orthogonalize([x])[0]), O.orthogonal(f64(x))
    # bf16's rounding of the output, at most 2^-8 of a value
    assert np.linalg.norm(got - exact) <= (2.0 ** -9 + 2.0 ** -8) * np.linalg.norm(exact)


def test_degenerate_matrices(dev):
    """Zero, one entry, one direction, tiny and large magnitudes; an empty one among others."""
    import torch
    zero = torch.zeros((40, 50), device=dev)
    one = zero.clone()
    one[7, 9] = 3.0
    rank1 = torch.outer(torch.arange(1, 41, device=dev).float(), torch.linspace(-1, 1, 50, device=dev))
    x = gradient(dev, 40, 50, 1)
    empty = torch.zeros((0, 50), device=dev)
    got = pkg.orthogonalize([zero, one, rank1, x * 1e-12, x * 1e15, empty])
    assert bool((got[0] == 0).all()) and got[5].shape == (0, 50)
    for o, u, eps in ((got[1], one, 1e-7), (got[2], rank1, 1e-7), (got[3], x * 1e-12, 1e-7), (got[4], x * 1e15, 1e-7)):
        assert_orthogonal(o, f64(u), eps=eps)
    x[3, 3] = float("nan")
    assert bool(torch.isnan(pkg.orthogonalize([x])[0]).all())


def state(dev, shapes, seed, bf16=True, dtype="bf16"):
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    p32 = [0.02 * torch.randn(s, generator=g, device=dev) for s in shapes]
    m = [1e-3 * torch.randn(s, generator=g, device=dev) for s in shapes]
    grads = [gradient(dev, *s, seed + i, dtype) for i, s in enumerate(shapes)]
    params = [p.bfloat16() if bf16 else p.clone() for p in p32]
    return params, (p32 if bf16 else None), m, grads


@pytest.mark.parametrize("bf16, dtype, nesterov", [(True, "bf16", True), (False, "fp32", False), (True, "fp32", False)])
def test_step(dev, bf16, dtype, nesterov):
    import torch
    shapes = [(64, 130), (257, 333), (330, 164), (5, 700), (64, 130)]
    params, masters, m, grads = state(dev, shapes, 3, bf16, dtype)
    p0, m0 = [f64(t) for t in (masters or params)], [f64(t) for t in m]
    decay, share = [0.0, 0.1, 0.02, 0.5, 0.0], [1.0, 0.5, 2.0, 1.0, 0.0]
    opt = pkg.Muon(params, masters=masters, lr=0.03, momentum=0.9, nesterov=nesterov, weight_decay=decay, lr_scale=share, m=m,
                   grads=grads)
    scale = torch.tensor([0.25], device=dev)
    opt.step(grad_scale=scale)
    pkg.rlk_joint_attn_check_status()
    for i, s in enumerate(shapes):
        g, rate = f64(grads[i]) * 0.25, 0.03 * share[i]
        args = (p0[i], m0[i], g, rate, 0.9, nesterov, decay[i], 0.2)
        p, mm, x = O.muon(*args)
        # momentum: one rounding of g', one of the sum
        assert np.all(np.abs(f64(m[i]) - mm) <= 2.0 ** -23 * (np.abs(0.9 * m0[i]) + np.abs(g)) + 2.0 ** -148)
        w = (masters or params)[i]
        step = rate * 0.2 * np.sqrt(max(s))
        d = np.linalg.norm(O.muon(*args, stored=True)[2] - x)
        # the products' and the rates' roundings: three of the step, two of the decay, one of p; X from an fp32 u
        tol = step * (2 * d + 3 * 2.0 ** -24 * np.linalg.norm(x)) + 2.0 ** -24 * (2 + 2 * rate * decay[i]) * np.linalg.norm(p0[i])
        assert np.linalg.norm(f64(w) - p) <= tol, (i, s)
        if bf16:
            assert Hh.bits_equal(params[i], w.bfloat16())


def test_step_with_device_rate_and_bad_scale(dev):
    """A rate on the device gives the number's bytes; a factor that is not finite changes nothing."""
    import torch
    shapes = [(100, 40), (40, 96), (300, 200), (129, 1001)]
    runs = []
    for lr in (0.01, torch.tensor([0.01], device=dev)):
        params, masters, m, grads = state(dev, shapes, 9)
        opt = pkg.Muon(params, masters=masters, m=m, grads=grads, weight_decay=0.0)
        opt.step(lr=lr)
        runs.append([*params, *masters, *m])
    for a, b in zip(*runs):
        assert np.linalg.norm(f64(a) - f64(b)) <= 2.0 ** -7 * np.linalg.norm(f64(a))  # (bf16 neighbours at most)
    before = [t.clone() for t in runs[1]]
    for bad in (float("nan"), float("inf")):
        opt.step(grad_scale=torch.tensor([bad], device=dev))
    assert all(Hh.bits_equal(a, b) for a, b in zip(before, runs[1]))


def test_list_order_and_many_sizes(dev):
    """More sizes than a launch's groups and more matrices than a pass's list: the same bytes as alone."""
    shapes = [(8 + 3 * (i % 11), 200 - 13 * (i % 11)) for i in range(90)]
    xs = [gradient(dev, *s, i) for i, s in enumerate(shapes)]
    got = pkg.orthogonalize(xs)
    back = pkg.orthogonalize(xs[::-1])[::-1]
    for i in range(0, 90, 7):
        assert Hh.bits_equal(got[i], pkg.orthogonalize([xs[i]])[0])
    assert all(Hh.bits_equal(a, b) for a, b in zip(got, back))


SMALL = [(1, 12289), (64, 12288), (12289, 64), (64, 513), (65, 512), (128, 4096), (4097, 128), (128, 4100), (100, 513), (17, 4097), (2, 1)]


def test_edges_of_the_small_kernel(dev):
    """The widest matrices that one kernel takes and the next ones, one column a CTA's slice and one more; odd rows and
    aligned ones, tall and wide; among others and alone."""
    xs = [gradient(dev, *s, i, "bf16" if i % 2 else "fp32") for i, s in enumerate(SMALL)]
    got = pkg.orthogonalize(xs)
    pkg.rlk_joint_attn_check_status()
    for x, o in zip(xs, got):
        assert_orthogonal(o, f64(x), tuple(x.shape))
        assert Hh.bits_equal(pkg.orthogonalize([x])[0], o), tuple(x.shape)


def test_values_that_the_first_look_misses(dev):
    """X's scale in fp16 comes from a part of the matrix: values far above and below it elsewhere."""
    import torch
    for shape in ((60, 700), (700, 60), (100, 900)):
        for size in (1e-7, 1.0, 1e6):
            x = gradient(dev, *shape, 5)
            x[: shape[0] // 2] *= size
            x[:, -3:] *= 1e-3
            assert_orthogonal(pkg.orthogonalize([x])[0], f64(x), (shape, size))
        z = torch.zeros(shape, device=dev)
        z[-1, -1] = 2.0
        assert_orthogonal(pkg.orthogonalize([z])[0], f64(z), shape)


def test_two_optimisers_at_once(dev):
    """Objects of their own on two streams: small and large matrices."""
    import torch
    shapes = [(64, 700), (300, 260), (100, 2000), (260, 513)]
    want, got = [], []
    for run in (0, 1):
        objects = []
        for seed in (1, 2):
            params, masters, m, grads = state(dev, shapes, seed)
            objects.append((pkg.Muon(params, masters=masters, m=m, grads=grads), [*params, *masters, *m]))
        streams = [torch.cuda.Stream(), torch.cuda.Stream()] if run else [None, None]
        torch.cuda.synchronize()
        for _ in range(3):
            for (opt, _), s in zip(objects, streams):
                opt.step(stream=s)
        torch.cuda.synchronize()
        (got if run else want).extend(t for _, ts in objects for t in ts)
    assert all(Hh.bits_equal(a, b) for a, b in zip(want, got))
    pkg.rlk_joint_attn_check_status()


def test_captured_step(dev):
    import torch
    shapes = [(64, 200), (300, 130), (100, 5000), (200, 260)]
    params, masters, m, grads = state(dev, shapes, 4)
    opt = pkg.Muon(params, masters=masters, m=m, grads=grads)
    lr = torch.tensor([0.02], device=dev)
    first = [t.clone() for t in (*masters, *m)]
    opt.step(lr=lr)
    opt.step(lr=lr)
    want = [t.clone() for t in (*params, *masters, *m)]
    for t, k in zip((*masters, *m), first):
        t.copy_(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        opt.step(lr=lr)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert all(Hh.bits_equal(a, b) for a, b in zip(want, (*params, *masters, *m)))


def test_other_stream_and_workspace_of_its_own(dev):
    import torch
    x = gradient(dev, 200, 264, 8)
    want = pkg.orthogonalize([x])[0]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [pkg.orthogonalize([x], stream=s)[0] for _ in range(3)]
    s.synchronize()
    assert all(Hh.bits_equal(want, o) for o in got)


def test_projection_trained_by_muon(dev):
    """The projections as they are trained: weights to codes, forward, backward, clipped Muon step, weights again."""
    import torch
    B, T, n_in, n_out = 2, (9, 40), 136, 264
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    w = tuple((rnd(n_out, n_in) / n_in ** 0.5).bfloat16() for _ in T)
    bias = tuple(torch.zeros(n_out, device=dev, dtype=torch.bfloat16) for _ in T)
    op = pkg.Fp8Projection(B, *T, n_in, n_out, device=dev)
    muon, adam = pkg.Muon(w, lr=0.02, weight_decay=0.01), pkg.AdamW(bias, lr=0.02)
    x = tuple(rnd(B, t, n_in).bfloat16() for t in T)
    for step in (1, 2):
        op.set_weights(w)
        f = op.forward(x, bias, train=True)
        dy = tuple((1e-2 * t).contiguous() for t in f["y"])  # towards smaller outputs
        r = op.backward(dy, f)
        clip = adam.grad_norm(max_norm=0.5, grads=r["db"])[1:]
        p0, m0 = [f64(t) for t in muon.masters], [f64(t) for t in muon.m]
        muon.step(grads=r["dw"], grad_scale=clip)
        adam.step(step, grad_scale=clip)
        pkg.rlk_joint_attn_check_status()
        for i in (0, 1):
            gt = O.quantize(f64(dy[i]).reshape(-1, n_out), 128, 1)[0].T
            xt = O.quantize(f64(x[i]).reshape(-1, n_in), 128, 1)[0].T
            assert np.all(np.abs(f64(r["dw"][i]) - gt @ xt.T) <= O.product_bound(gt, xt) + 2.0 ** -24 * np.abs(gt @ xt.T))
            args = (p0[i], m0[i], f64(r["dw"][i]) * float(clip), 0.02, 0.95, True, 0.01, 0.2)
            p, _, ex = O.muon(*args)
            d = np.linalg.norm(O.muon(*args, stored=True)[2] - ex)
            step_size = 0.02 * 0.2 * np.sqrt(max(p.shape))
            tol = step_size * (2 * d + 2.0 ** -22 * np.linalg.norm(ex)) + 2.0 ** -22 * np.linalg.norm(p)
            assert np.linalg.norm(f64(muon.masters[i]) - p) <= tol
            assert Hh.bits_equal(w[i], muon.masters[i].bfloat16())
    y = op.forward(x, bias)["y"]
    op.set_weights(w)
    assert not Hh.bits_equal(op.forward(x, bias)["y"][1], y[1])  # the new weights' codes


@pytest.mark.parametrize("rows, cols", [(16, 1160), (1000, 33), (64, 2567), (128, 1000), (130, 845), (300, 1000), (768, 400)])
def test_what_fp16_leaves_of_independent_entries(dev, rows, cols):
    """X is rounded to fp16 six times, each by 2^-11 of a value at most, 2^-11 / sqrt(3) of it in the mean square: 6.9e-4
    in all. The roundings of A's and B's parts are fewer bits of less than that, as much again at most: sqrt(2) 6.9e-4
    < 2^-10. (A and B rounded whole leave 1.3e-3 and more.)"""
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(rows)
    x = torch.randn((rows, cols), generator=g, device=dev)
    p = torch.zeros_like(x)
    pkg.Muon([p], lr=1.0, momentum=0.0, nesterov=False, weight_decay=0.0, update_rms=1.0, grads=[x]).step()
    pkg.rlk_joint_attn_check_status()
    got, exact = -f64(p) / np.sqrt(max(rows, cols)), O.orthogonal(f64(x))
    assert np.linalg.norm(got - exact) <= 2.0 ** -10 * np.linalg.norm(exact)


@pytest.mark.parametrize("poly", [(2.0, -1.5, 0.5), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0), (1.0, 0.0, 0.0), (3.0, -3.2, 1.2)])
@pytest.mark.parametrize("rows, cols", [(1, 9), (40, 50), (100, 700), (257, 300)])
def test_other_polynomials(dev, poly, rows, cols):
    x = gradient(dev, rows, cols, 11)
    assert_orthogonal(pkg.orthogonalize([x], coefficients=poly)[0], f64(x), (poly, rows, cols), coefficients=poly)
