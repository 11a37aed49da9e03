"""CPU tests of the 8-bit projections and of Muon beside test_projection_host.py: what the header says of their limits
and of what a call reads, held against the library and its sources."""

import math
import os
import re

import pytest

import invariant_mmdit_joint_gb300 as pkg
from tests.test_projection_host import P, L, args, gemm, matrices, no_gpu, product, quant, quantize, step  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "invariant_mmdit_joint_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_kernels_that_start_early_read_by_ordinary_loads():
    """A kernel behind griddepcontrol.wait is alive while the one before it writes its inputs: the language allows
    read-only loads (__ldg, ld.global.nc, const __restrict__) only for memory that nobody writes meanwhile, and the wait
    orders ordinary loads. Files with such kernels hold no read-only load."""
    early = [f for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh")) and "griddepcontrol.wait" in source(f)]
    assert {"k_fp8.cu", "k_muon.cu"} <= set(early)
    for f in early:
        found = re.findall(r"__ldg\w*|ld\.global\.nc|__restrict__|__ldcs|__ldca", source(f))
        assert not found, (f, found)


def test_orthogonalize_takes_no_argument_of_a_step(L):  # noqa: F811
    """Rates, momentum and device scalars are not refused (a step refuses each), and every pointer that the kernels'
    arguments take from args is a step's alone: one that the contract does not read may be no address at all."""
    t = matrices(master=None, m=None)
    t[0].master = t[0].m = None
    for over in (dict(lr=-1.0), dict(lr=math.nan), dict(momentum=1.0), dict(update_rms=-1.0), dict(nesterov=2), dict(lr_dev=P + 2),
                 dict(grad_scale=P + 1)):
        assert step(L, a=args(**over)) != 0
        if no_gpu():
            assert step(L, t, name="rlk_orthogonalize", a=args(**over)) == 5, over
    taken = re.findall(r"=\s*([^;=]*\bq\.(?:lr_dev|grad_scale))\b([^;]*);", source("k_muon.cu"))
    taken = [(a, b) for a, b in taken if "!=" not in a + b]  # (the host's rate looks whether there is a pointer)
    assert len(taken) == 4 and all(a.startswith("step ? ") and b == " : nullptr" for a, b in taken), taken


def test_the_headers_limits_are_the_librarys(L):  # noqa: F811
    """Rows, tokens and sums of the 8-bit calls: the last size that the header allows passes, the next one is refused."""
    with open(os.path.join(ROOT, "include", "rlk_joint_attn.h")) as f:
        text = f.read()
    rows = (1 << 31) - int(re.search(r"0 <= rows < 2\^31 - (\d+)", text).group(1))
    both = (1 << 31) - int(re.search(r"0 <= m, n < 2\^31 - (\d+)", text).group(1))
    k = (1 << 31) - int(re.search(r"1 <= k < 2\^31 - (\d+)", text).group(1))
    assert both % 8 == 0  # (n's last multiple of 8 is 8 below)
    far = lambda i: P + i * (1 << 44)  # noqa: E731
    assert pkg.rlk_fp8_quant_workspace_bytes(rows - 1, 8) > 0 and pkg.rlk_fp8_quant_workspace_bytes(rows, 8) == 0
    q = dict(x=far(0), q=far(1), q_scale=far(2), qt=far(3), qt_scale=far(4), col_sum=far(5), workspace=far(6), cols=8, x_stride=8)
    p = dict(a=far(0), a_scale=far(1), b=far(2), b_scale=far(3), bias=far(4), d=far(5), m=8, n=8, k=128, d_stride=8)
    assert quantize(L, quant(**q, rows=rows)) == 1
    for over in (dict(m=both), dict(n=both, d_stride=both), dict(k=k)):
        assert gemm(L, product(**{**p, **over})) == 1, over
    if no_gpu():  # (what is right goes on to the device)
        assert quantize(L, quant(**q, rows=rows - 1)) == 5
        for over in (dict(m=both - 1), dict(n=both - 8, d_stride=both - 8), dict(k=k - 1)):
            assert gemm(L, product(**{**p, **over})) == 5, over
    torch = pytest.importorskip("torch")
    make = lambda t: pkg.Fp8Projection(1, 0, t, 8, 8, device="cpu", dw_dtype=torch.float32)  # noqa: E731
    make(rows - 1)
    with pytest.raises(pkg.RlkError):
        make(rows)
