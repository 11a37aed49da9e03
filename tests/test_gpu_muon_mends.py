"""Calls of Muon and of the orthogonal update that the operators' first tests do not make."""

import numpy as np
import pytest

import invariant_mmdit_joint_gb300 as pkg
from oracle import projection_ops as O
from tests import _helpers as Hh
from tests.test_gpu_muon import assert_orthogonal, f64, gradient, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


@pytest.mark.parametrize("rows, cols", [(40, 50), (200, 300), (300, 200), (200, 304)])
def test_orthogonalize_reads_no_argument_of_a_step(dev, rows, cols):
    """Rates, momentum and the device scalars of args are a step's: NaN behind the pointers changes no byte."""
    import torch
    x, nan = gradient(dev, rows, cols, 1), torch.full((4,), float("nan"), device=dev)
    want = pkg.orthogonalize([x])[0]
    got = torch.empty_like(want)
    items = (pkg.MuonMatrix * 1)(pkg.MuonMatrix(got.data_ptr(), None, x.data_ptr(), None, rows, cols, 0.0, 0.0, 1, 0))
    a, b, c = pkg.POLYNOMIAL
    args = pkg.MuonArgs(lr=float("nan"), momentum=float("nan"), update_rms=-1.0, a=a, b=b, c=c, eps=1e-7, lr_dev=nan.data_ptr(),
                        grad_scale=nan.data_ptr() + 4, iterations=5, nesterov=7)
    ws = torch.empty(pkg.rlk_muon_workspace_bytes(items), dtype=torch.uint8, device=dev)
    pkg.rlk_orthogonalize(items, args, ws)
    pkg.rlk_joint_attn_check_status()
    assert Hh.bits_equal(want, got)


@pytest.mark.parametrize("rows, cols", [(40, 50), (16, 1160), (300, 40), (200, 304), (301, 200)])
def test_small_norms_with_any_eps(dev, rows, cols):
    """Zero stays zero and nothing becomes infinite for the smallest eps; a norm above 2^-56 is the formula's, one below
    counts as 2^-56: X is then no more than |u| 2^56 and its growth, 3.4445^5."""
    import torch
    x = gradient(dev, rows, cols, 2)
    zero = torch.zeros_like(x)
    for eps in (2.0 ** -126, 1e-30, 1e-7):
        assert bool((pkg.orthogonalize([zero], eps=eps)[0] == 0).all()), eps
        for size in (2.0 ** -60, 2.0 ** -70, 2.0 ** -90):  # (entries of about 2^-9 times this)
            u = x * (size / float(x.double().norm()))
            top = float(u.double().norm()) * 2.0 ** 56 * 3.45 ** 5
            got = pkg.orthogonalize([u], eps=eps)[0]
            assert bool(torch.isfinite(got).all()) and float(got.double().norm()) <= top + 2.0 ** -20, (eps, size)
        u = x * (2.0 ** -50 / float(x.double().norm()))
        if eps < 1e-7:
            assert_orthogonal(pkg.orthogonalize([u], eps=eps)[0], f64(u), (rows, cols, eps), eps=eps)
    pkg.rlk_joint_attn_check_status()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("lr", [0.01, 2.0 ** -9, 1e-4])
def test_device_rate_gives_the_numbers_bytes(dev, bf16, lr):
    """One step from a rate on the device and from the same number: every byte of p, its master and m. The rates' products
    with unlike scales and decays are no powers of two, so that another order or rounding of them shows; and both are the
    formula's: p's error is X's, three roundings of the step, two of the decay and one of p."""
    import torch
    shapes = [(100, 40), (40, 96), (300, 200), (129, 1001), (700, 20), (150, 150)]
    decay, share = [0.1, 0.3, 0.7, 0.9, 0.0, 1.1], [0.3, 1.0, 1.7, 0.9, 1.3, 0.7]
    on_device = torch.tensor([lr], device=dev)
    number, runs = float(on_device), []
    for rate in (number, on_device):
        params, masters, m, grads = state(dev, shapes, 9, bf16)
        p0, m0 = [f64(t) for t in (masters or params)], [f64(t) for t in m]
        opt = pkg.Muon(params, masters=masters, m=m, grads=grads, weight_decay=decay, lr_scale=share, lr=5.0, momentum=0.9)
        opt.step(lr=rate)
        pkg.rlk_joint_attn_check_status()
        runs.append([*params, *(masters or ()), *m])
        for i, (s, w) in enumerate(zip(shapes, masters or params)):
            want, _, x = O.muon(p0[i], m0[i], f64(grads[i]), number * share[i], 0.9, True, decay[i], 0.2)
            step, norm = number * share[i] * 0.2 * np.sqrt(max(s)), np.linalg.norm
            tol = step * (2.0 ** -9 + 3 * 2.0 ** -24) * norm(x) + 2.0 ** -24 * (2 + 2 * number * share[i] * decay[i]) * norm(p0[i])
            assert norm(f64(w) - want) <= tol, (i, s)
    assert all(Hh.bits_equal(a, b) for a, b in zip(*runs))


def test_device_rate_scales_the_decay(dev):
    """A zero update: p -= rate decay p alone, which a decay without the rate, or twice the rate, misses."""
    import torch
    for shape in ((30, 70), (200, 304), (301, 150)):
        for rate in (0.25, torch.tensor([0.25], device=dev)):
            p = torch.randn(shape, device=dev)
            want = p.double() * (1 - 0.25 * 0.5 * 0.125)
            zero = torch.zeros_like(p)
            pkg.Muon([p], lr=9.0, lr_scale=0.5, weight_decay=0.125, grads=[zero]).step(lr=rate)
            assert bool(((p.double() - want).abs() <= 2.0 ** -23 * want.abs()).all()), shape


def test_codes_in_the_workspace(dev):
    """Sizes whose codes of X's rounding lie in the workspace beside ones whose do not: steps on two streams at once, a
    captured step and a list turned over give the bytes of steps one by one, whatever the workspace held; a factor that is
    not finite changes nothing."""
    import torch
    shapes = [(64, 4000), (4001, 50), (100, 4001), (33, 9000), (64, 2567), (300, 130), (128, 2600), (20, 30)]

    def make(seed, order=1):
        params, masters, m, grads = state(dev, shapes, seed)
        opt = pkg.Muon(params[::order], masters=masters[::order], m=m[::order], grads=grads[::order], lr=0.02)
        return opt, [*params, *masters, *m]
    want = []
    for seed in (1, 2):
        opt, tensors = make(seed)
        for _ in range(2):
            opt.step()
        want.append([t.clone() for t in tensors])
    both, streams = [make(1), make(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(2):
        for (opt, _), s in zip(both, streams):
            opt.step(stream=s)
    torch.cuda.synchronize()
    for (_, tensors), w in zip(both, want):
        assert all(Hh.bits_equal(a, b) for a, b in zip(tensors, w))
    for order in (1, -1):
        opt, tensors = make(1, order)
        first = [t.clone() for t in tensors]
        opt.step()
        opt.workspace.fill_(0xff)  # (NaN codes)
        for t, k in zip(tensors, first):
            t.copy_(k)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            opt.step()
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert all(Hh.bits_equal(a, b) for a, b in zip(tensors, want[0]))
        opt.step(grad_scale=torch.tensor([float("nan")], device=dev))
        assert all(Hh.bits_equal(a, b) for a, b in zip(tensors, want[0]))
    pkg.rlk_joint_attn_check_status()
