"""CPU tests of the 8-bit projections and of Muon: the C entries refuse bad
arguments before any device work, the binding refuses tensors that the library
could not read, and the 64-bit definitions the GPU tests compare with agree with
their formats and with what they are for."""

import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import invariant_mmdit_joint_gb300 as pkg
from oracle import projection_ops as O

P = 1 << 32  # an aligned address that nothing reads: validation stops first
STEP = 1 << 30  # buffers this far apart
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(pkg.library_path()):
        from invariant_mmdit_joint_gb300 import _build
        _build.build()
    return pkg.lib()


def no_gpu():
    import torch
    return not torch.cuda.is_available()


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_struct_layouts_match_the_header(tmp_path):
    import shutil
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    pairs = (("rlk_fp8_quant", pkg.Fp8Quant), ("rlk_fp8_product", pkg.Fp8Product), ("rlk_muon_matrix", pkg.MuonMatrix),
             ("rlk_muon_args", pkg.MuonArgs))
    lines = "".join(f'printf("%zu\\n", sizeof({c}));' +
                    "".join(f'printf("%zu\\n", offsetof({c}, {f}));' for f, _ in s._fields_) for c, s in pairs)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "rlk_joint_attn.h"\n'
                   'int main(void) {' + lines + 'return 0; }\n')
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True).stdout.split()]
    want = [v for _, s in pairs for v in [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]]
    assert got == want


# ------------------------------------------------------------------ codes
def test_sizes(L):
    assert [pkg.rlk_fp8_row_bytes(k) for k in (-1, 0, 1, 16, 17, 2600)] == [0, 0, 16, 16, 32, 2608]
    assert [pkg.rlk_fp8_scale_row_bytes(k) for k in (0, 1, 512, 513, 2600)] == [0, 4, 4, 8, 24]
    assert pkg.rlk_fp8_quant_workspace_bytes(129, 64) == 2 * 64 * 4 and pkg.rlk_fp8_quant_workspace_bytes(0, 8) == 32
    for bad in ((-1, 8), (4, 0), (4, 12), (4, (1 << 20) + 8), (1 << 31, 8)):
        assert pkg.rlk_fp8_quant_workspace_bytes(*bad) == 0


def quant(**over):
    d = dict(x=P, q=P + STEP, q_scale=P + 2 * STEP, qt=P + 3 * STEP, qt_scale=P + 4 * STEP, col_sum=P + 5 * STEP,
             workspace=P + 6 * STEP, rows=300, cols=264, x_stride=264, x_dtype=0, format=0, square=0, reserved=0)
    return pkg.Fp8Quant(**{**d, **over})


def quantize(L, *items, n=None):
    a = (pkg.Fp8Quant * max(1, len(items)))(*items)
    return L.rlk_fp8_quantize(a, len(items) if n is None else n, None)


@pytest.mark.parametrize("over, code", [
    (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(cols=0), 1), (dict(cols=260), 1), (dict(cols=(1 << 20) + 8), 1),
    (dict(x_stride=256), 1), (dict(x_dtype=2), 1), (dict(format=2), 1), (dict(square=2), 1), (dict(reserved=1), 1),
    (dict(x=None), 1), (dict(q=None), 1), (dict(q_scale=None), 1), (dict(qt=None), 1), (dict(qt_scale=None), 1),
    (dict(q=None, q_scale=None, qt=None, qt_scale=None), 1), (dict(workspace=None), 1), (dict(col_sum=None), 1),
    (dict(x_stride=268), 3), (dict(x_dtype=1, x_stride=266), 3), (dict(x=P + 8), 3), (dict(q=P + STEP + 4), 3),
    (dict(qt=P + 3 * STEP + 8), 3), (dict(q_scale=P + 2 * STEP + 2), 3), (dict(qt_scale=P + 4 * STEP + 1), 3),
    (dict(col_sum=P + 5 * STEP + 4), 3), (dict(workspace=P + 6 * STEP + 8), 3),
    (dict(q=P + 16), 1), (dict(q=P + 3 * STEP), 1), (dict(qt_scale=P + 2 * STEP), 1), (dict(col_sum=P + 6 * STEP + 16), 1)])
def test_quantize_fails_closed(L, over, code):
    assert quantize(L, quant(**over)) == code


def test_quantize_lists(L):
    assert quantize(L, quant(), n=0) == 1 and quantize(L, *[quant()] * 9) == 1 and L.rlk_fp8_quantize(None, 1, None) == 1
    assert quantize(L, quant(), quant(x=P)) == 1  # the second writes where the first does
    far = quant(**{k: P + (8 + i) * STEP for i, k in enumerate(("q", "q_scale", "qt", "qt_scale", "col_sum", "workspace"))})
    if no_gpu():  # (what is right goes on to the device)
        assert quantize(L, quant()) == 5 and quantize(L, quant(), far) == 5  # inputs may be shared
        assert quantize(L, quant(rows=0, x=None)) == 5
        assert quantize(L, quant(q=None, q_scale=None, col_sum=None, workspace=None)) == 5


def product(**over):
    d = dict(a=P, a_scale=P + STEP, b=P + 2 * STEP, b_scale=P + 3 * STEP, bias=P + 4 * STEP, d=P + 5 * STEP, m=300, n=264, k=1000,
             d_stride=264, a_format=0, b_format=1, d_dtype=0, accumulate=0)
    return pkg.Fp8Product(**{**d, **over})


def gemm(L, *items, n=None):
    a = (pkg.Fp8Product * max(1, len(items)))(*items)
    return L.rlk_fp8_gemm(a, len(items) if n is None else n, None)


@pytest.mark.parametrize("over, code", [
    (dict(m=-1), 1), (dict(m=1 << 31), 1), (dict(n=-8), 1), (dict(n=260), 1), (dict(k=0), 1), (dict(k=1 << 31), 1),
    (dict(d_stride=256), 1), (dict(a_format=2), 1), (dict(b_format=-1), 1), (dict(d_dtype=2), 1), (dict(accumulate=1), 1),
    (dict(accumulate=2, d_dtype=1), 1), (dict(a=None), 1), (dict(a_scale=None), 1), (dict(b=None), 1), (dict(b_scale=None), 1),
    (dict(d=None), 1), (dict(d_stride=268), 3), (dict(a=P + 8), 3), (dict(b=P + 2 * STEP + 8), 3), (dict(d=P + 5 * STEP + 8), 3),
    (dict(bias=P + 4 * STEP + 2), 3), (dict(a_scale=P + STEP + 2), 3), (dict(b_scale=P + 3 * STEP + 1), 3),
    (dict(d=P), 1), (dict(d=P + 3 * STEP - 1024), 1), (dict(d=P + 4 * STEP), 1), (dict(reserved=1), 1), (dict(a_rows=2), 1),
    (dict(a_rows=1, m=17, a_scale=None), 1), (dict(a_rows=1, m=16, k=12296, a_scale=None), 1),
    (dict(a_rows=1, m=16, k=100, a_scale=None), 1), (dict(a_rows=1, m=16), 1),
    (dict(a_rows=1, m=16, a_scale=None, d=P + 16 * 1000 * 2 - 16), 1)])
def test_product_fails_closed(L, over, code):
    assert gemm(L, product(**over)) == code


def test_product_lists(L):
    assert gemm(L, product(), n=0) == 1 and gemm(L, *[product()] * 9) == 1 and L.rlk_fp8_gemm(None, 1, None) == 1
    assert gemm(L, product(), product()) == 1 and gemm(L, product(), product(d=P + 2 * STEP)) == 1
    if no_gpu():
        assert gemm(L, product()) == 5 and gemm(L, product(bias=None, d_dtype=1, accumulate=1)) == 5
        assert gemm(L, product(), product(d=P + 6 * STEP)) == 5  # operands may be shared
        assert gemm(L, product(m=0, a=None, d=None)) == 5
        few = dict(a_rows=1, m=16, a_scale=None)
        assert gemm(L, product(**few)) == 5 and gemm(L, product(**few, k=12288), product(**few, d=P + 6 * STEP)) == 5
    assert gemm(L, product(a_rows=1, m=16, a_scale=None), product(d=P + 6 * STEP)) == 1  # in every product or in none


# ------------------------------------------------------------------ Muon
def args(**over):
    d = dict(lr=0.01, momentum=0.9, update_rms=0.2, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, iterations=5, nesterov=1)
    return pkg.MuonArgs(**{**d, **over})


def matrices(**over):
    t = (pkg.MuonMatrix * 2)()
    for i in (0, 1):
        d = dict(p=P, master=P + STEP, g=P + 2 * STEP, m=P + 3 * STEP, rows=30, cols=50, lr_scale=1.0, weight_decay=0.1, g_dtype=0)
        for k in ("p", "master", "g", "m"):
            d[k] += i * 4 * STEP
        if i == 1:
            d.update(over)
        t[i] = pkg.MuonMatrix(**d)
    return t


def step(L, t=None, n=2, a=None, ws=P - STEP, size=1 << 29, name="rlk_muon_step"):
    return getattr(L, name)(matrices() if t is None else t, n, ref(args() if a is None else a), ws, size, None)


@pytest.mark.parametrize("over, code", [
    (dict(rows=-1), 1), (dict(cols=(1 << 16) + 1), 1), (dict(rows=1 << 16, cols=1 << 16), 1), (dict(g_dtype=2), 1),
    (dict(reserved=3), 1), (dict(lr_scale=-1.0), 1), (dict(lr_scale=math.nan), 1), (dict(weight_decay=math.inf), 1),
    (dict(lr_scale=1e39), 1), (dict(weight_decay=1e39), 1), (dict(p=None), 1), (dict(g=None), 1), (dict(m=None), 1),
    (dict(p=P + 4 * STEP + 8), 3), (dict(g=P + 6 * STEP + 2), 3), (dict(m=P + 7 * STEP + 4), 3), (dict(master=P + 5 * STEP + 4), 3),
    (dict(p=P), 1), (dict(m=P + 2 * STEP), 1), (dict(g=P + 3 * STEP + 16), 1), (dict(master=P - STEP), 1)])
def test_muon_matrices_fail_closed(L, over, code):
    assert step(L, matrices(**over)) == code


@pytest.mark.parametrize("over, code", [
    (dict(lr=-1.0), 1), (dict(lr=math.nan), 1), (dict(momentum=1.0), 1), (dict(momentum=-0.1), 1), (dict(update_rms=-1.0), 1),
    (dict(a=math.inf), 1), (dict(b=math.nan), 1), (dict(c=1e7), 1), (dict(eps=0.0), 1), (dict(eps=2.0), 1),
    (dict(iterations=0), 1), (dict(iterations=33), 1), (dict(nesterov=2), 1), (dict(lr=1e39), 1), (dict(lr_dev=P + 2), 3),
    (dict(grad_scale=P + 1), 3)])
def test_muon_arguments_fail_closed(L, over, code):
    assert step(L, a=args(**over)) == code


def test_muon_lists_and_workspace(L):
    need = pkg.rlk_muon_workspace_bytes(matrices())
    assert need > 0 and pkg.rlk_muon_workspace_bytes(matrices(rows=-1)) == 0
    big = matrices(rows=1000, cols=2000)
    # X twice, A and B in fp16, partial sums; small matrices need none
    assert 2 * (2 * 1000 * 2000 + 2 * 1000 * 1000) <= pkg.rlk_muon_workspace_bytes(big) <= 2 * (2 * 1000 * 2000 + 2 * 1000 * 1000) + 8192
    assert step(L, n=-1) == 1 and L.rlk_muon_step(None, 2, ref(args()), P, 1 << 20, None) == 1
    assert L.rlk_muon_step(matrices(), 2, None, P, 1 << 20, None) == 1
    assert step(L, ws=None) == 1 and step(L, ws=P - STEP + 8) == 3 and step(L, t=big, size=1000) == 4
    assert step(L, n=0) == 0  # nothing to do
    assert step(L, name="rlk_orthogonalize") == 1  # these take neither master nor momentum
    if no_gpu():
        assert step(L) == 5 and step(L, a=args(lr_dev=P + 4, grad_scale=P + 8)) == 5
        assert step(L, matrices(rows=0, p=None, g=None, m=None, master=None)) == 5
        t = matrices(master=None, m=None)
        t[0].master = t[0].m = None
        assert step(L, t, name="rlk_orthogonalize", a=args(lr=-1.0)) == 5


# ------------------------------------------------------------------ binding
def test_projection_binding_refuses_unfit_tensors(L):
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    op = pkg.Fp8Projection(2, 3, 5, 64, 48, device="cpu")
    x = (torch.zeros(2, 3, 64, dtype=bf), torch.zeros(2, 5, 64, dtype=bf))
    dy = (torch.zeros(2, 3, 48, dtype=bf), torch.zeros(2, 5, 48, dtype=bf))
    w = (torch.zeros(48, 64, dtype=bf),) * 2
    b = (torch.zeros(48, dtype=bf),) * 2
    for bad in ((w[0],), (w[0], None), (w[0], w[1].float()), (w[0].half(), w[1].half()), (w[0], torch.zeros(64, 48, dtype=bf)),
                (None, None)):
        with pytest.raises(ValueError):
            op.set_weights(bad)
    with pytest.raises(ValueError, match="CUDA"):
        op.set_weights(w)
    for bad in (dict(x=(x[0],)), dict(x=(x[0], None)), dict(x=(x[0].float(), x[1])), dict(x=(x[0], x[1][:, :4])),
                dict(bias=(b[0].float(), b[1])), dict(bias=(b[0], torch.zeros(47, dtype=bf))), dict(out={"y": x}),
                dict(out={"z": dy})):
        with pytest.raises(ValueError):
            op.forward(**{**dict(x=x, bias=b), **bad})
    with pytest.raises(ValueError, match="weights"):
        op.forward(x, b)
    op._set = True
    with pytest.raises(ValueError, match="CUDA"):
        op.forward(x, b)
    for bad in (dict(saved=None), dict(saved={"y": dy}), dict(want=()), dict(want=("dx",), accumulate=True), dict(accumulate=True),
                dict(dy=x), dict(saved={"xt": x, "xt_scale": x})):
        with pytest.raises(ValueError):
            op.backward(**{**dict(dy=dy, saved=None), **bad})
    for bad in (dict(n_in=60), dict(n_out=0), dict(B=0), dict(T_txt=-1), dict(T_txt=0, T_img=0), dict(B=1 << 20, T_img=1 << 12)):
        with pytest.raises(pkg.RlkError):
            pkg.Fp8Projection(**{**dict(B=2, T_txt=3, T_img=5, n_in=64, n_out=48, device="cpu"), **bad})
    with pytest.raises(ValueError):
        pkg.Fp8Projection(2, 3, 5, 64, 48, grad_format="e3m4", device="cpu")
    with pytest.raises(ValueError):
        pkg.Fp8Projection(2, 3, 5, 64, 48, out_dtype=torch.float16, device="cpu")
    one = pkg.Fp8Projection(1, 0, 5, 64, 48, device="cpu")
    with pytest.raises(ValueError):
        one.forward((x[0], x[1][:1]))


def test_muon_binding_refuses_unfit_tensors(L):
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    p = [torch.zeros(6, 8, dtype=bf), torch.zeros(5, 7)]
    g = [torch.zeros(6, 8), torch.zeros(5, 7, dtype=bf)]
    for bad in (dict(params=[]), dict(params=[torch.zeros(6), p[1]]), dict(params=[p[0].half(), p[1]]), dict(params=[p[0].t(), p[1]]),
                dict(masters=[None, torch.zeros(5, 7)]), dict(masters=[torch.zeros(8, 6), None]), dict(m=[torch.zeros(6, 8)]),
                dict(m=[torch.zeros(6, 8, dtype=bf), None]), dict(lr_scale=[1.0]), dict(grads=g[:1]),
                dict(grads=[g[0].t().contiguous(), g[1]]), dict(grads=[g[0].half(), g[1]])):
        with pytest.raises(ValueError):
            pkg.Muon(**{**dict(params=p), **bad})
    opt = pkg.Muon(p)
    assert opt.masters[0].dtype == torch.float32 and opt.masters[1] is None and opt.m[1].shape == (5, 7)
    with pytest.raises(ValueError, match="no gradients"):
        opt.step()
    with pytest.raises(ValueError, match="CUDA"):
        opt.step(grads=g)
    for t in (p[1], opt.m[0], opt.masters[0], opt.grads[0]):
        old = t.data
        t.data = t.data.clone()
        with pytest.raises(ValueError, match="replaced"):
            opt.step()
        t.data = old
    with pytest.raises(ValueError, match="CUDA"):
        opt.step()


def test_orthogonalize_refuses_unfit_tensors(L):
    torch = pytest.importorskip("torch")
    assert pkg.orthogonalize([]) == []
    for bad in ([torch.zeros(4)], [torch.zeros(4, 5, dtype=torch.float64)], [torch.zeros(4, 5).t()], [torch.zeros(4, 5, 6)]):
        with pytest.raises(ValueError):
            pkg.orthogonalize(bad)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.orthogonalize([torch.zeros(4, 5)])


# ------------------------------------------------------------------ the definitions
@pytest.mark.parametrize("fmt, torch_name", [("e4m3", "float8_e4m3fn"), ("e5m2", "float8_e5m2")])
def test_codes_are_the_formats(fmt, torch_name):
    torch = pytest.importorskip("torch")
    dtype = getattr(torch, torch_name)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 300)) * np.exp(4 * rng.standard_normal((1, 300)))
    x[0, :128], x[1, 5] = 0.0, 448.0 * 2.0 ** 20
    v, e = O.quantize(x, 1, 128, fmt)
    top = O.FORMATS[fmt][2]
    for i in range(5):
        for j in range(3):
            part, most = v[i, 128 * j:128 * j + 128], np.abs(x[i, 128 * j:128 * j + 128]).max()
            assert most <= top * 2.0 ** e[i, j] and (e[i, j] == -126 or most > top * 2.0 ** (e[i, j] - 1))
            codes = torch.from_numpy(part * 2.0 ** -float(e[i, j]))
            assert bool((codes.to(dtype).double() == codes).all())  # on the format's grid
            near = torch.from_numpy(x[i, 128 * j:128 * j + 128] * 2.0 ** -float(e[i, j]))
            # and no other value of the grid is nearer
            grid = torch.arange(256, dtype=torch.uint8).view(dtype).double()
            grid = grid[torch.isfinite(grid)]
            best = (near[:, None] - grid[None]).abs().amin(1)
            assert bool(((near - codes).abs() <= best).all())


def test_orthogonal_update():
    """Singular values go to about 1 (the polynomial swings between 0.68 and 1.14), directions stay; turned inputs give
    turned outputs; storage in fp16 changes it by less than 2^-8."""
    rng = np.random.default_rng(0)
    u = rng.standard_normal((30, 80))
    x = O.orthogonal(u)
    s = np.linalg.svd(x, compute_uv=False)
    assert 0.6 < s.min() and s.max() < 1.25
    left, _, right = np.linalg.svd(u, full_matrices=False)
    core = left.T @ x @ right.T
    assert np.abs(core - np.diag(np.diag(core))).max() < 1e-9
    assert np.allclose(O.orthogonal(u.T), x.T, atol=1e-12)
    assert np.linalg.norm(O.orthogonal(u, stored=True) - x) < 2.0 ** -8 * np.linalg.norm(x)
    p, m, o = O.muon(np.zeros((30, 80)), np.zeros((30, 80)), u, 0.1, 0.9, True, 0.0, 0.2)
    assert np.allclose(o, O.orthogonal(1.9 * u)) and np.allclose(m, u)
    assert abs(np.sqrt((p * p).mean()) - 0.1 * 0.2) < 0.2 * 0.1 * 0.2  # the update's root mean square


def test_product_bound_is_not_met_by_fewer_bits():
    """The bound the GPU's products are held to tells an accumulator of 14 bits from one of 24."""
    rng = np.random.default_rng(1)
    a, _ = O.quantize(rng.standard_normal((4, 512)), 1, 128)
    b, _ = O.quantize(rng.standard_normal((4, 512)), 1, 128)
    exact = a @ b.T

    def summed(bits):
        s = np.zeros((4, 4))
        for k in range(0, 512, 32):
            s = s + a[:, k:k + 32] @ b[:, k:k + 32].T
            m, e = np.frexp(s)
            s = np.ldexp(np.trunc(m * 2.0 ** bits) / 2.0 ** bits, e)
        return np.abs(s - exact)
    bound = O.product_bound(a, b)
    assert np.all(summed(24) <= bound) and np.any(summed(13) > bound)
