"""CPU tests of the adaln operators, the gradient norm and AdamW: the C
entries refuse bad arguments before any device work, the binding refuses
tensors that the library could not read, and the 64-bit definitions the GPU
tests compare with agree with differences and with their format."""

import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import invariant_mmdit_joint_gb300 as pkg
from oracle import block_ops as O

P = 1 << 20  # an aligned address that nothing reads: validation stops first
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


# ------------------------------------------------------------------ adaln
def call(L, name, sh, io=(None, None), grad=None, ws=P, ws_bytes=1 << 40):
    f = getattr(L, "rlk_adaln_" + name)
    args = [ref(sh), ref(io[0]), ref(io[1])]
    if name.endswith("bwd"):
        args += [ref(grad[0]), ref(grad[1]), ws, ws_bytes]
    return f(*args, None)


IO = dict(x=P, h=P, gate=P, scale=P, shift=P, w=P, w_post=P, r=P, y=P, stats=P, post_stats=P)
GRAD = dict(dy=P, dr=P, dx=P, dh=P, dgate=P, dscale=P, dshift=P, dw=P, dw_post=P)


def io(**over):
    return pkg.AdalnIo(**{**IO, **over})


def grad(**over):
    return pkg.AdalnGrad(**{**GRAD, **over})


@pytest.mark.parametrize("over, code", [
    (dict(B=0), 1), (dict(B=65536), 1), (dict(T_txt=-1), 1), (dict(T_img=-4), 1), (dict(T_txt=0, T_img=0), 1),
    (dict(C=0), 1), (dict(C=12), 1), (dict(C=8200), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1),
    (dict(alpha=float("inf")), 1), (dict(mod_stride=56), 1), (dict(dmod_stride=60), 1),
    (dict(T_img=(1 << 20) + 1), 1), (dict(B=65535, T_img=1 << 15), 1),
    (dict(y_fp32=True), 2), (dict(mod_stride=68), 3), (dict(mod_fp32=True, mod_stride=66), 3), (dict(dmod_stride=66), 3)])
def test_adaln_shapes_fail_closed(L, over, code):
    sh = pkg.AdalnShape.make(**{**dict(B=2, T_txt=3, T_img=5, C=64, post="rms"), **over})
    assert pkg.rlk_adaln_workspace_bytes(sh) == 0
    for name in ("modulation_fwd", "gate_residual_fwd", "modulation_bwd", "gate_residual_bwd"):
        assert call(L, name, sh, (io(), io()), (grad(), grad())) == code


def test_adaln_norm_kinds_and_null_shape(L):
    assert call(L, "modulation_fwd", None, (io(), io())) == 1
    for field, value in (("norm", 0), ("norm", 3), ("post", 3), ("post", -1), ("x_dtype", 2), ("mod_dtype", -1)):
        sh = pkg.AdalnShape.make(2, 3, 5, 64)
        setattr(sh, field, value)
        assert call(L, "modulation_fwd", sh, (io(), io())) == 1, field


def test_adaln_pointers_fail_closed(L):
    sh = pkg.AdalnShape.make(2, 3, 5, 64, post="rms")

    def fwd(name, **over):
        return call(L, name, sh, (io(), io(**over)))

    def bwd(name, i=None, **over):
        return call(L, name, sh, (io(), io(**(i or {}))), (grad(), grad(**over)))
    for k in ("x", "y"):
        assert fwd("modulation_fwd", **{k: None}) == 1, k
    for k in ("x", "h", "r"):
        assert fwd("gate_residual_fwd", **{k: None}) == 1, k
    for k in ("x", "y", "scale", "shift", "w", "stats"):
        assert fwd("modulation_fwd", **{k: P + 8}) == 3, k
    for k in ("x", "h", "r", "y", "gate", "scale", "w_post", "post_stats"):
        assert fwd("gate_residual_fwd", **{k: P + 4}) == 3, k
    assert call(L, "modulation_fwd", sh, (None, io())) == 1            # the text has tokens
    assert call(L, "modulation_fwd", sh, (io(), None)) == 1
    assert bwd("modulation_bwd", dy=None) == 1                         # dy is required
    assert bwd("modulation_bwd", dx=None) == 1
    assert bwd("modulation_bwd", i=dict(stats=None)) == 1
    assert bwd("modulation_bwd", i=dict(x=None)) == 1
    nothing = grad(dy=None, dr=None, dscale=None, dshift=None, dw=None)
    assert call(L, "gate_residual_bwd", sh, (io(), io()), (nothing, nothing)) == 1
    assert call(L, "gate_residual_bwd", sh, (io(), io()), (grad(dy=None), grad(dy=None))) == 1  # sums that dy feeds
    assert bwd("gate_residual_bwd", dh=None) == 1
    assert bwd("gate_residual_bwd", dr=None) == 1                      # for one stream alone
    assert bwd("modulation_bwd", dr=None) == 1
    assert bwd("gate_residual_bwd", i=dict(r=None)) == 1
    assert bwd("gate_residual_bwd", i=dict(post_stats=None)) == 1
    assert bwd("gate_residual_bwd", dgate=P + 4) == 3
    assert bwd("gate_residual_bwd", dh=P + 8) == 3
    assert call(L, "modulation_bwd", sh, (io(), io()), (grad(), None)) == 1
    plain = pkg.AdalnShape.make(2, 3, 5, 64)                           # no norm after the sublayer
    assert call(L, "gate_residual_fwd", plain, (io(), io())) == 1      # w_post without one
    g = grad()
    assert call(L, "gate_residual_bwd", plain, (io(w_post=None), io(w_post=None)), (g, g)) == 1  # dw_post without one
    need = pkg.rlk_adaln_workspace_bytes(sh)
    assert need > 0
    gg = (grad(), grad())
    assert call(L, "modulation_bwd", sh, (io(), io()), gg, ws=None) == 1
    assert call(L, "modulation_bwd", sh, (io(), io()), gg, ws=P + 4) == 3
    assert call(L, "modulation_bwd", sh, (io(), io()), gg, ws_bytes=need - 1) == 4
    if no_gpu():  # well-formed calls reach the device check
        assert call(L, "modulation_bwd", sh, (io(), io()), gg, ws_bytes=need) == 5
        assert fwd("modulation_fwd", scale=None, shift=None, w=None, stats=None) == 5
        assert fwd("gate_residual_fwd", y=None, gate=None) == 5
        alone = tuple(grad(dy=None, dscale=None, dshift=None, dw=None) for _ in range(2))
        assert call(L, "gate_residual_bwd", sh, (io(), io()), alone) == 5
        only = pkg.AdalnShape.make(2, 0, 5, 64)
        assert call(L, "modulation_fwd", only, (None, io())) == 5


def test_adaln_calls_are_traced(L):
    sh = pkg.AdalnShape.make(2, 3, 5, 64)
    with pkg.op_trace() as t:
        call(L, "modulation_fwd", sh, (None, io()))
        call(L, "gate_residual_bwd", sh, (io(), io()), (grad(), grad()))
        call(L, "modulation_fwd", None)
        L.rlk_adamw_step(None, 1, None, None)
        L.rlk_grad_norm(None, 1, 1.0, 1.0, P, P, 64, None)
    got = [(r["entry_point"], r["status"], r["n_kernels"], r["B"], r["T_txt"], r["grid_w"]) for r in t.records]
    assert got == [("rlk_adaln_modulation_fwd", 1, 0, 2, 3, 5), ("rlk_adaln_gate_residual_bwd", 1, 0, 2, 3, 5),
                   ("rlk_adaln_modulation_fwd", 1, 0, 0, 0, 0), ("rlk_adamw_step", 1, 0, 0, 0, 0),
                   ("rlk_grad_norm", 1, 0, 0, 0, 0)]
    assert all(r["fallback"] == 0 and r["atomics"] == 0 and r["reduction_order"] and r["arithmetic_policy"]
               for r in t.records)


def test_the_trace_states_the_orders_of_the_sums_in_full(L):
    """The trees that the GPU tests follow bit by bit, none of them cut off."""
    sh = pkg.AdalnShape.make(2, 3, 5, 64)
    with pkg.op_trace() as t:
        call(L, "modulation_fwd", sh, (None, io()))
        call(L, "modulation_bwd", sh, (None, io()), (grad(), grad()))
        L.rlk_grad_norm(None, 1, 1.0, 1.0, P, P, 64, None)
    for r, words in zip(t.records, (("16 above C = 1024", "xor 16..1", "warps", "xor 8..1"),
                                    ("warps xor 8..1", "rows of a chunk", "32nd chunk", "runs ascending", "b ascending"),
                                    ("16384 elements", "warps ascending", "1024th", "xor 16..1 twice"))):
        assert all(w in r["reduction_order"] for w in words), r["reduction_order"]
        assert len(r["reduction_order"]) < 159


# ------------------------------------------------------------------ optimiser
def entries(count=2, **over):
    base = dict(p=P, master=None, g=P, m=P, v=P, m_scale=None, v_scale=None, n=64, lr_scale=1.0, weight_decay=0.0,
                g_dtype=1, state_bits=32, key=0, reserved=0)
    t = (pkg.AdamwTensor * count)()
    for i in range(count):
        # every buffer of its own, a megabyte apart
        at = {k: P * (1 + 8 * i + j) for j, k in enumerate(("p", "g", "m", "v"))}
        for k, v in {**base, **at, **(over if i == count - 1 else {})}.items():
            setattr(t[i], k, v)
    return t


def args(**over):
    return pkg.AdamwArgs(**{**dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1), **over})


@pytest.mark.parametrize("over, code", [
    (dict(p=None), 1), (dict(g=None), 1), (dict(m=None), 1), (dict(v=None), 1), (dict(n=-1), 1),
    (dict(n=(1 << 40) + 1), 1), (dict(g_dtype=2), 1), (dict(state_bits=16), 1), (dict(state_bits=8), 1),
    (dict(reserved=1), 1), (dict(lr_scale=-1.0), 1), (dict(weight_decay=float("nan")), 1),
    (dict(p=P + 8), 3), (dict(g=P + 2), 3), (dict(m=P + 4), 3), (dict(master=P * 15 + 4), 3),
    (dict(state_bits=8, m_scale=P * 14 + 1, v_scale=P * 15), 3),
    (dict(p=P * 3), 1),             # another tensor's m
    (dict(v=P * 11 + 64 * 4 - 16), 1),  # the end of its own m
    (dict(m=P * 10), 1),            # its own gradient
    (dict(master=P * 12 + 128), 1)])
def test_adamw_tensors_fail_closed(L, over, code):
    assert L.rlk_adamw_step(entries(**over), 2, ref(args()), None) == code


@pytest.mark.parametrize("over, code", [
    (dict(lr=-1.0), 1), (dict(lr=float("nan")), 1), (dict(beta1=1.0), 1), (dict(beta2=-0.1), 1), (dict(eps=0.0), 1),
    (dict(eps=1e-16), 1), (dict(eps=2.0), 1),
    (dict(step=0), 1), (dict(step=1 << 31), 1), (dict(reserved=3), 1), (dict(lr_dev=P + 2), 3), (dict(step_dev=P + 4), 3),
    (dict(grad_scale=P + 1), 3)])
def test_adamw_arguments_fail_closed(L, over, code):
    assert L.rlk_adamw_step(entries(), 2, ref(args(**over)), None) == code


@pytest.mark.parametrize("a, e, code", [
    (dict(lr=1e39), {}, 1), ({}, dict(lr_scale=1e39), 1), ({}, dict(weight_decay=1e39), 1),
    (dict(lr=1e20), dict(lr_scale=1e20), 1), (dict(lr=1e20), dict(weight_decay=1e20), 1),
    (dict(lr=1e20), dict(lr_scale=1e10, weight_decay=1e5), 5)])
def test_adamw_rates_past_fp32_are_refused(L, a, e, code):
    """The kernel holds them in fp32: an infinite rate makes NaN of elements without an update."""
    if code == 1 or no_gpu():
        assert L.rlk_adamw_step(entries(**e), 2, ref(args(**a)), None) == code


def test_adamw_list_limits(L):
    assert L.rlk_adamw_step(entries(), -1, ref(args()), None) == 1
    assert L.rlk_adamw_step(None, 2, ref(args()), None) == 1
    assert L.rlk_adamw_step(entries(), 2, None, None) == 1
    if no_gpu():
        assert L.rlk_adamw_step(entries(), 2, ref(args()), None) == 5
        assert L.rlk_adamw_step(entries(g=2 * P), 2, ref(args(grad_scale=P + 4, step=0, step_dev=P)), None) == 5
        # tensors of no elements have no buffers; gradients may be shared
        assert L.rlk_adamw_step(entries(n=0, p=None, g=None, m=None, v=None), 2, ref(args()), None) == 5


def test_overlaps_are_found_in_any_order(L):
    """Lists of buffers in random places and orders against the rule itself: no
    written range meets another one; read ones (gradients) may meet."""
    if not no_gpu():
        pytest.skip("addresses of no memory: for machines without a GPU")
    rng = np.random.default_rng(12)
    seen = set()
    for trial in range(600):
        count = int(rng.integers(1, 40))
        t = (pkg.AdamwTensor * count)()
        # distinct slots: each kind's buffers in a run, tensor by tensor, or shuffled; some with a collision
        slots = np.arange(7 * count)
        flat = trial % 3 == 0
        if flat:
            slots = slots.reshape(7, count).T.reshape(-1)
        elif trial % 3 == 1:
            rng.shuffle(slots)
        ranges = []
        for i in range(count):
            bits, copy, n = int(rng.choice([8, 32])), bool(rng.integers(2)), int(rng.integers(0, 4096))
            copy = copy if not flat else trial % 2 == 0 or i < count // 2
            fields = {"g": (4, False), "p": (2 if copy else 4, True), "m": (bits // 8, True), "v": (bits // 8, True)}
            if copy:
                fields["master"] = (4, True)
            if bits == 8:
                fields.update(m_scale=(1 / 32, True), v_scale=(1 / 32, True))
            t[i].n, t[i].state_bits, t[i].g_dtype, t[i].lr_scale = n, bits, 1, 1.0
            for k, (size, written) in fields.items():
                at = P + 16384 * int(slots[7 * i + ("g", "p", "master", "m", "v", "m_scale", "v_scale").index(k)])
                if trial % 4 > 1 and rng.random() < 0.02:
                    at += int(rng.integers(-8192, 8192)) // 16 * 16  # perhaps into a neighbour
                if k == "g" and rng.random() < 0.2:
                    at = P + 16384 * 7 * count  # one shared by several
                setattr(t[i], k, at)
                if n:
                    ranges.append((at, at + int(np.ceil(n * size)), written))
        bad = any((a[2] or b[2]) and a[0] < b[1] and b[0] < a[1] for i, a in enumerate(ranges) for b in ranges[:i])
        assert L.rlk_adamw_step(t, count, ref(args()), None) == (1 if bad else 5), trial
        seen.add((flat, bad))
    assert len(seen) == 4


def test_grad_norm_fails_closed(L):
    t = entries()
    need = pkg.rlk_grad_norm_workspace_bytes(t, 2)
    assert need == 8

    def norm(t=t, n=2, pre=1.0, most=1.0, out=P + 4, ws=P, ws_bytes=need):
        return L.rlk_grad_norm(t, n, pre, most, out, ws, ws_bytes, None)
    assert norm(t=None) == 1 and norm(n=-1) == 1 and norm(pre=0.0) == 1 and norm(pre=math.inf) == 1
    assert norm(most=0.0) == 1 and norm(most=math.nan) == 1 and norm(out=None) == 1 and norm(ws=None) == 1
    assert norm(out=P + 2) == 3 and norm(ws=P + 8) == 3 and norm(ws_bytes=need - 1) == 4
    assert norm(t=entries(g=P + 8)) == 3 and norm(t=entries(g=None)) == 1 and norm(t=entries(g_dtype=5)) == 1
    assert pkg.rlk_grad_norm_workspace_bytes(entries(n=-3), 2) == 0
    if no_gpu():
        assert norm() == 5 and norm(most=math.inf) == 5


def test_struct_layouts_match_the_header(tmp_path):
    import shutil
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    pairs = (("rlk_adaln_shape", pkg.AdalnShape), ("rlk_adaln_io", pkg.AdalnIo), ("rlk_adaln_grad", pkg.AdalnGrad),
             ("rlk_adamw_tensor", pkg.AdamwTensor), ("rlk_adamw_args", pkg.AdamwArgs))
    lines = "".join(f'printf("%zu\\n", sizeof({c}));' +
                    "".join(f'printf("%zu\\n", offsetof({c}, {f}));' for f, _ in s._fields_) for c, s in pairs)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "rlk_joint_attn.h"\n'
                   'int main(void) {' + lines + 'return 0; }\n')
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True).stdout.split()]
    want = [v for _, s in pairs for v in [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]]
    assert got == want


# ------------------------------------------------------------------ binding
def test_adaln_binding_refuses_unfit_tensors(L):
    torch = pytest.importorskip("torch")
    op = pkg.AdaLN(2, 3, 5, 64, device="cpu")
    bf = torch.bfloat16
    x = (torch.zeros(2, 3, 64, dtype=bf), torch.zeros(2, 5, 64, dtype=bf))
    mod = torch.zeros(2, 6 * 64, dtype=bf)
    s = (mod[:, :64], mod[:, 64:128])
    bad = [
        dict(x=(x[0], None)), dict(x=(x[0],)), dict(x=(x[0], x[1].float())), dict(x=(x[0], torch.zeros(2, 5, 72, dtype=bf))),
        dict(x=(x[0], torch.zeros(2, 64, 5, dtype=bf).transpose(1, 2))), dict(scale=(s[0], s[1].float())),
        dict(scale=(s[0], mod[:, ::6])), dict(scale=(s[0], torch.zeros(2, 64, dtype=bf))),  # two sample strides
        dict(shift=(s[0], mod[:1, :64])), dict(w=(torch.zeros(64, dtype=bf), None)), dict(w=(torch.zeros(63), None)),
        dict(out={"y": x}), dict(out={"y": (x[0], x[0]), "stats": (None, None)})]
    good = dict(x=x, scale=s, shift=s)
    for over in bad:
        with pytest.raises(ValueError):
            op.modulation(**{**good, **over})
    one_row = (mod[:1, :64].expand(2, 64),) * 2
    with pytest.raises(ValueError, match="every sample"):
        op.modulation(x=x, scale=one_row, shift=one_row)
    with pytest.raises(ValueError, match="CUDA"):
        op.modulation(**good)
    with pytest.raises(ValueError):
        op.gate_residual_bwd(x, x, s, s, None, None)
    with pytest.raises(ValueError):
        pkg.AdaLN(2, 3, 5, 64, x_dtype=torch.float16, device="cpu")
    with pytest.raises(pkg.RlkError):
        pkg.AdaLN(2, 3, 5, 60, device="cpu")
    one = pkg.AdaLN(2, 0, 5, 64, device="cpu")
    with pytest.raises(ValueError):
        one.modulation((x[0], x[1]), s, s)  # a text without tokens


def test_adaln_results_passed_back_are_looked_at(L):
    torch = pytest.importorskip("torch")
    op, names = pkg.AdaLN(2, 3, 5, 64, device="cpu"), ("y", "stats")
    out, p = op._outputs(None, names, None)
    assert op._outputs(out, names, None) == (out, p) and out["y"][1].data_ptr() == p["y"][1]
    held = out["y"]
    out["y"] = (held[0], torch.zeros_like(held[1]))  # another buffer: taken as such
    assert op._outputs(out, names, None)[1]["y"] == tuple(t.data_ptr() for t in out["y"])
    out["y"] = held
    held[1].data = torch.zeros_like(held[1])  # the same tensor over other memory
    assert op._outputs(out, names, None)[1]["y"][1] == held[1].data_ptr()
    held[1].data = torch.zeros(5, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="y.1."):
        op._outputs(out, names, None)
    held[1].data = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    for other in (pkg.AdaLN(2, 3, 4, 64, device="cpu"), pkg.AdaLN(2, 3, 5, 64, y_dtype=torch.float32, x_dtype=torch.float32, device="cpu")):
        with pytest.raises(ValueError):
            other._outputs(out, names, None)
    with pytest.raises(ValueError, match="must hold"):
        op._outputs(out, ("y", "stats", "r"), None)
    out.pop("stats")
    with pytest.raises(ValueError, match="must hold"):
        op._outputs(out, names, None)


def test_adaln_results_hold_their_memory(L):
    """A result whose data was replaced twice must not come to its old address with fewer elements behind it."""
    torch = pytest.importorskip("torch")
    op, names = pkg.AdaLN(2, 3, 5, 64, device="cpu"), ("y", "stats")
    for _ in range(40):
        out, p = op._outputs(None, names, None)
        t, old = out["y"][1], out["y"][1].data_ptr()
        t.data = torch.empty(0, dtype=t.dtype)
        t.data = torch.zeros(2, 5, 63, dtype=t.dtype)
        assert t.data_ptr() != old
        with pytest.raises(ValueError, match="y.1."):
            op._outputs(out, names, None)


def test_adaln_workspace_is_taken_for_what_it_is(L, monkeypatch):
    """A workspace that someone put in place of the object's own: its own size goes to the library, not the needed one."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(pkg, "_require_current", lambda device: None)
    monkeypatch.setattr(pkg, "_raw_stream", lambda stream, index: 0)
    op = pkg.AdaLN(2, 3, 5, 64, device="cpu")
    x = (torch.zeros(2, 3, 64, dtype=torch.bfloat16), torch.zeros(2, 5, 64, dtype=torch.bfloat16))
    stats = (torch.zeros(2, 3, 2), torch.zeros(2, 5, 2))
    op.workspace = torch.zeros(pkg.rlk_adaln_workspace_bytes(op.shape) - 1, dtype=torch.uint8)
    for call in (lambda: op.modulation_bwd(x, None, stats, x),
                 lambda: op.gate_residual_bwd(x, x, None, None, stats, x)):
        with pytest.raises(pkg.RlkError) as e:
            call()
        assert e.value.code == 4


def test_adamw_binding_refuses_unfit_tensors(L):
    torch = pytest.importorskip("torch")
    p = [torch.zeros(5, 7), torch.zeros(33, dtype=torch.bfloat16)]
    opt = pkg.AdamW(p, state_bits=8)
    assert opt.masters[0] is None and opt.masters[1].dtype == torch.float32
    assert [m.dtype for m in opt.m] == [torch.float8_e4m3fn] * 2 and [s.numel() for s in opt.m_scale] == [2, 2]
    g = [torch.zeros(5, 7), torch.zeros(33)]
    for bad in ([g[0]], [g[0], torch.zeros(32)], [g[0].half(), g[1]], [torch.zeros(7, 5).t(), g[1]],
                [torch.zeros(7, 5), g[1]]):
        with pytest.raises(ValueError):
            opt.step(1, grads=bad)
    with pytest.raises(ValueError):
        opt.step(1)  # no gradients
    with pytest.raises(ValueError, match="CUDA"):
        opt.step(1, grads=g)
    with pytest.raises(ValueError, match="CUDA"):
        opt.grad_norm(1.0)
    for bad in (dict(params=[]), dict(params=[p[0].half()]), dict(params=p, state_bits=4), dict(params=p, m=[p[0]]),
                dict(params=p, masters=[p[0], None]), dict(params=p, weight_decay=[0.1]), dict(params=[p[0].t()]),
                dict(params=p, v=[torch.zeros(35), torch.zeros(34)]), dict(params=p, keys=[1]),
                dict(params=p, keys=[0, 2 ** 32]), dict(params=p, seed=-1)):
        with pytest.raises(ValueError):
            pkg.AdamW(**bad)


def test_adamw_keeps_to_its_tensors(L):
    torch = pytest.importorskip("torch")
    p = [torch.zeros(5, 7), torch.zeros(33, dtype=torch.bfloat16)]
    opt = pkg.AdamW(p, state_bits=8, grads=[torch.zeros(35), torch.zeros(33)])
    for held in (opt.params, opt.grads, opt.masters, opt.m, opt.v, opt.m_scale, opt.v_scale):
        with pytest.raises(TypeError):  # the call's list holds the addresses of those that are there
            held[0] = torch.zeros(35)
    p[0].data = torch.zeros(5, 7)
    with pytest.raises(ValueError, match="replaced"):
        opt.step(1)


def test_adamw_looks_at_the_memory_its_list_points_to(L):
    """Every tensor that someone else can hold: one whose data was replaced is
    refused by the calls that would read or write its old memory, and that stays
    allocated, so that no other tensor can come to its address."""
    torch = pytest.importorskip("torch")
    names = {"params": "p", "grads": "g", "masters": "master", "m": "m", "v": "v", "m_scale": "m_scale",
             "v_scale": "v_scale"}

    def make(given):
        p = [torch.zeros(5, 7), torch.zeros(33, dtype=torch.bfloat16)]
        state = dict(masters=[None, torch.zeros(33)])
        for k in ("m", "v"):
            state[k] = [torch.zeros(n, dtype=torch.float8_e4m3fn) for n in (35, 33)]
            state[k + "_scale"] = [torch.zeros(2, dtype=torch.uint8) for _ in p]
        return pkg.AdamW(p, state_bits=8, grads=[torch.zeros(35), torch.zeros(33)], **(state if given else {})), state
    for given in (False, True):
        for name, field in names.items():
            opt, _ = make(given)
            t, old = getattr(opt, name)[1], getattr(opt._list[1], field)
            assert t.data_ptr() == old
            t.data = torch.empty(0, dtype=t.dtype)
            fresh = [torch.zeros(n, dtype=t.dtype) for n in (2, 33, 33) for _ in range(40)]
            assert all(f.data_ptr() != old for f in fresh), name
            for t.data in (fresh[0], fresh[50]):
                with pytest.raises(ValueError, match="replaced"):
                    opt.step(1)
                if name == "grads":
                    with pytest.raises(ValueError, match="replaced"):
                        opt.grad_norm(1.0)
                    with pytest.raises(ValueError, match="CUDA"):  # given anew they are taken
                        opt.step(1, grads=[torch.zeros(35), torch.zeros(33)])
                    opt, _ = make(given)
                    t = opt.grads[1]
        opt, _ = make(given)
        opt.m[0].untyped_storage().resize_(0)
        with pytest.raises(ValueError, match="replaced"):
            opt.step(1)
        for name in names:
            with pytest.raises(AttributeError):
                setattr(opt, name, getattr(opt, name))
    # what a caller gave stays the object's memory, whatever the caller's own tensor is over
    opt, state = make(True)
    state["m"][0].data = torch.zeros(35, dtype=torch.float8_e4m3fn)
    assert opt.m[0].data_ptr() == opt._list[0].m != state["m"][0].data_ptr()
    with pytest.raises(ValueError, match="CUDA"):
        opt.step(1)


# ------------------------------------------------------------------ definitions
def _loss(d, c):
    r = d["x"]
    if c["gate"]:
        r, _, _ = O.residual(d["x"], d["h"], d["gate"], d["w_post"], c["post"], c["alpha"], 1e-6)
    y = O.modulation(r, d["scale"], d["shift"], d["w"], c["norm"], 1e-6)[0]
    return float((y * d["dy"]).sum() + (r * d["dr"]).sum())


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("gate, post", [(False, "none"), (True, "none"), (True, "rms"), (True, "layer")])
def test_definition_gradients_against_differences(norm, gate, post):
    rng = np.random.default_rng(5)
    B, T, C = 2, 3, 16
    c = dict(gate=gate, post=post, norm=norm, alpha=0.7)
    d = {k: rng.standard_normal((B, T, C)) for k in ("x", "h", "dy", "dr")}
    d.update({k: 0.5 * rng.standard_normal((B, C)) for k in ("gate", "scale", "shift")})
    d.update(w=1 + 0.3 * rng.standard_normal(C), w_post=1 + 0.3 * rng.standard_normal(C))
    if gate:
        r, _, st = O.residual(d["x"], d["h"], d["gate"], d["w_post"], post, c["alpha"], 1e-6)
        mean, rstd, _, _ = O.stats(r, norm, 1e-6)
        got = O.gate_residual_backward(r, d["h"], d["gate"], d["scale"], d["w"], d["w_post"], mean, rstd,
                                       None if st is None else st[0], d["dy"], d["dr"], norm, post, c["alpha"])
    else:
        mean, rstd, _, _ = O.stats(d["x"], norm, 1e-6)
        got = O.modulation_backward(d["x"], d["scale"], d["w"], mean, rstd, d["dy"], d["dr"], norm)
    names = {"dx": "x", "dscale": "scale", "dshift": "shift", "dw": "w"}
    if gate:
        names.update(dh="h", dgate="gate")
        if post != "none":
            names["dw_post"] = "w_post"
    step = 1e-5
    for out, inp in names.items():
        value = got[out][0]
        assert value.shape == d[inp].shape
        for at in [tuple(rng.integers(0, n) for n in value.shape) for _ in range(6)]:
            both = []
            for sign in (1, -1):
                e = dict(d, **{inp: d[inp].copy()})
                e[inp][at] += sign * step
                both.append(_loss(e, c))
            diff = (both[0] - both[1]) / (2 * step)
            # truncation step^2 * f''' / 6 (f''' of order 10 here) and cancellation 2^-52 * |loss| / step
            assert abs(diff - value[at]) <= 1e-7 * max(1.0, abs(diff)), (out, at, diff, value[at])


def test_eight_bit_format():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().double().numpy()
    np.testing.assert_array_equal(O.E4M3, want)
    rng = np.random.default_rng(3)
    x = (rng.standard_normal(64 * 32) * np.repeat(10.0 ** rng.integers(-12, 4, 64), 32)).astype(np.float32)
    x[:32] = 0.0
    up = down = 0
    for k in range(40):
        bits = rng.integers(0, 65536, x.size)
        q, s = O.encode(x, bits, False)
        v = O.decode(q, s)
        top = np.abs(x.reshape(-1, 32)).max(1)
        # a code is off by less than one step: 2^-3 of its power of two, or 2^-9 of the scale
        step = np.maximum(np.abs(x) * 2.0 ** -3, np.repeat(2.0 ** (s.astype(float) - 127 - 9), 32))
        assert np.all(np.abs(v - x) < step + 1e-300)
        codes = np.abs(O.E4M3[q]).reshape(-1, 32).max(1)
        assert np.all((codes[top > 0] >= 224) & (codes[top > 0] <= 448))
        up, down = up + (v > x).sum(), down + (v < x).sum()
    assert abs(up / (up + down) - 0.5) < 0.02  # rounded both ways alike
    # the mean over the random bits is the value: 2^16 draws cover every one of them
    for value in (0.3, 1.0625, 0.001):
        block = np.zeros(32, np.float32)
        block[0], block[1] = 1.7, value
        mean = np.mean([O.decode(*O.encode(block, np.full(32, b), False))[1] for b in range(0, 65536, 257)])
        assert abs(mean - np.float32(value)) < 2.0 ** -3 * value / 100 + 1e-5
    q, s = O.encode(np.array([1.0] + [1e-30] * 31), np.zeros(32, int), True)
    assert q[1] == 1  # a positive second moment keeps the smallest code
    q, s = O.encode(np.array([np.inf] + [1.0] * 31), np.zeros(32, int), True)
    assert s[0] == 255 and np.isnan(O.decode(q, s)).all()
