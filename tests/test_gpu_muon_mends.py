"""Calls of Muon and of the orthogonal update that the operators' first tests do not make."""

import pytest

import invariant_mmdit_joint_gb300 as pkg
from tests import _helpers as Hh
from tests.test_gpu_muon import assert_orthogonal, f64, gradient

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
