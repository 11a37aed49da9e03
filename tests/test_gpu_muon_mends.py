"""Calls of Muon and of the orthogonal update that the operators' first tests do not make."""

import pytest

import invariant_mmdit_joint_gb300 as pkg
from tests import _helpers as Hh
from tests.test_gpu_muon import gradient

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
