"""One training step of a block's attention half as a user runs it: modulation,
QKV projection, joint attention, output projection, gate and residual with the
next modulation; backward through gate, norm and attention; clipped AdamW on
the gains, norm weights and modulation."""

import numpy as np
import pytest

import invariant_mmdit_joint_gb300 as pkg
from invariant_mmdit_joint_gb300 import workloads as W
from oracle import block_ops as O
from oracle import joint_attn as J
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


def f64(t):
    return t.detach().double().cpu().numpy()


def test_block_step(dev):
    import torch
    w = Hh.workload("block", 2, 3, 24, 5, 9, (24, 13))
    B, H, T, C = w.B, w.H, (w.T_txt, w.T_img), w.H * 128
    d = W.make_qkv_inputs(w, 3)
    x = tuple(Hh.to_dev(d["x_" + s], dev) for s in ("txt", "img"))
    wq = tuple(Hh.to_dev(d["w_" + s], dev) for s in ("txt", "img"))
    bq = tuple(Hh.to_dev(d["b_" + s], dev) for s in ("txt", "img"))
    wo = tuple(t[:C].contiguous() for t in wq)
    bo = tuple(t[:C].contiguous() for t in bq)
    gains = torch.from_numpy(W.gains(3)).to(dev)
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    mod = tuple((0.3 * torch.randn((B, 6 * C), generator=g, device=dev)).bfloat16() for _ in T)
    col = lambda k: tuple(m[:, k * C:(k + 1) * C] for m in mod)  # noqa: E731
    weights = [torch.ones(C, device=dev) for _ in range(4)]
    wn, w2 = tuple(weights[:2]), tuple(weights[2:])
    pre, post = (pkg.AdaLN(B, *T, C, device=dev, eps=EPS) for _ in range(2))
    ja = pkg.JointAttention(B, w.T_txt, w.grid_h, w.grid_w, H, device=dev)
    sh, vl = ja.shape, list(w.valid_len)

    # forward
    n1 = pre.modulation(x, col(0), col(1), w=wn)
    q, k, v = (tuple(torch.empty((B, t, H, 128), dtype=torch.bfloat16, device=dev) for t in T) for _ in range(3))
    pkg.rlk_qkv_bias_gemm(sh, n1["y"], wq, bq, gains, ja.ctx, q, k, v)
    o = tuple(torch.empty_like(t) for t in q)
    lse = torch.empty((B, H, w.S), device=dev)
    pkg.rlk_joint_attn_fwd_ctx(sh, ja.ctx, v, vl, o, lse)
    y = tuple(torch.empty((B, t, C), dtype=torch.bfloat16, device=dev) for t in T)
    pkg.rlk_attn_out_bias_gemm(sh, o, wo, bo, y)
    n2 = post.gate_residual(x, y, col(2), col(3), col(4), w=w2)

    # backward: through the second norm and the gate, the projection (plain), the attention
    dn = tuple(torch.randn((B, t, C), generator=g, device=dev).bfloat16() for t in T)
    dr = tuple(torch.randn((B, t, C), generator=g, device=dev).bfloat16() for t in T)
    b2 = post.gate_residual_bwd(n2["r"], y, col(2), col(3), n2["stats"], dn, dr, w=w2)
    do = tuple((b2["dh"][i].float() @ wo[i].float()).bfloat16().view(B, T[i], H, 128) for i in (0, 1))
    dq, dk, dv, dgp, dg = ja.backward_streams(q, k, v, gains, vl, o, do, lse)
    dx1 = tuple((torch.cat([t[i].reshape(B, T[i], C) for t in (dq, dk, dv)], -1).float() @ wq[i].float()).bfloat16()
                for i in (0, 1))
    b1 = pre.modulation_bwd(x, col(0), n1["stats"], dx1, b2["dx"], w=wn)
    pkg.rlk_joint_attn_check_status()

    # every operator's outputs from the inputs it was given
    for i in (0, 1):
        s = lambda k: f64(col(k)[i])  # noqa: E731
        ref, err, _, _ = O.modulation(f64(x[i]), s(0), s(1), f64(wn[i]), "layer", EPS)
        got = f64(n1["y"][i])
        assert np.all(np.abs(got - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err))
        r, err, _ = O.residual(f64(x[i]), f64(y[i]), s(2), None, "none", 1.0, EPS)
        assert np.all(np.abs(f64(n2["r"][i]) - r) <= err + 2.0 ** -8 * (np.abs(r) + err))
        st = f64(n2["stats"][i])
        ref = O.gate_residual_backward(f64(n2["r"][i]), f64(y[i]), s(2), s(3), f64(w2[i]), None, st[..., 0], st[..., 1],
                                       None, f64(dn[i]), f64(dr[i]), "layer", "none", 1.0)
        st = f64(n1["stats"][i])
        ref1 = O.modulation_backward(f64(x[i]), s(0), f64(wn[i]), st[..., 0], st[..., 1], f64(dx1[i]), f64(b2["dx"][i]),
                                     "layer")
        for have, want in ((b2, ref), (b1, ref1)):
            for name in have:
                value, bound = want[name]
                half = torch.finfo(have[name][i].dtype).eps / 2
                e = np.abs(f64(have[name][i]) - value)
                assert np.all(e <= bound * (1 + 1e-6) + half * (np.abs(value) + bound)), (i, name)
    # the attention between them, from the q, k, v that the projection gave it
    cat = lambda pair: torch.cat(pair, 1)  # noqa: E731
    ro, rl = J.joint_attn_forward(f64(cat(q)), f64(cat(k)), f64(cat(v)), W.gains(3).astype(np.float64), w.T_txt, w.grid_h,
                                  w.grid_w, vl, store_bf16=True)
    Hh.assert_forward_close(f64(cat(o)), f64(lse), ro, rl, scale=float(cat(v).float().std()))

    # the optimiser: gains, norm weights and the modulation's rows
    params = [gains] + weights + [m.float() for m in mod]
    grads = [dg, *b1["dw"], *b2["dw"]]
    for i in (0, 1):
        z = torch.zeros_like(b1["dscale"][i])
        grads.append(torch.cat([b1["dscale"][i], b1["dshift"][i], b2["dgate"][i], b2["dscale"][i], b2["dshift"][i], z], 1))
    for bits in (32, 8):
        mine = [p.clone() for p in params]
        opt = pkg.AdamW(mine, state_bits=bits, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.0)
        n = opt.grad_norm(1.0, grads=grads)
        opt.step(1, grad_scale=n[1:])
        want = np.sqrt(sum((f64(t) ** 2).sum() for t in grads))
        assert abs(f64(n)[0] / want - 1) <= 20 * O.U
        for p0, p1, t in zip(params, mine, grads):
            (ref, _, _), (pe, _, _) = O.adamw(f64(p0), f64(t), 0.0, 0.0, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8,
                                              weight_decay=0.0, step=1, scale=f64(n)[1])
            assert np.all(np.abs(f64(p1) - ref) <= pe)


def test_calls_on_two_streams_at_once(dev):
    """Objects of their own on two streams, their kernels in flight together: the bytes of one stream alone."""
    import torch
    g = torch.Generator(device=dev).manual_seed(5)

    def r(*shape):
        return torch.randn(shape, generator=g, device=dev).bfloat16()
    B, T, C = 2, (40, 1500), 1280
    x, h, dy, dr = (tuple(r(B, t, C) for t in T) for _ in range(4))
    mods = tuple(r(B, 3 * C) for _ in T)
    scale, shift, gate = (tuple(m[:, i * C:(i + 1) * C] for m in mods) for i in range(3))
    grads = [torch.randn(n, generator=g, device=dev) for n in (300_001, 70_000, 33)]

    def job():
        op = pkg.AdaLN(B, *T, C, device=dev)
        opt = pkg.AdamW([torch.zeros_like(d) for d in grads], state_bits=8, grads=grads)

        def run(t):
            f = op.gate_residual(x, h, gate, scale, shift)
            q = op.gate_residual_bwd(f["r"], h, gate, scale, f["stats"], dy, dr)
            n = opt.grad_norm(1.0)
            opt.step(t, grad_scale=n[1:])
            return [t for d in (f, q) for k in sorted(d) for t in d[k]] + [n]
        return run, opt
    results = []
    for streams in ([torch.cuda.current_stream()], [torch.cuda.Stream(), torch.cuda.Stream()]):
        jobs = [job() for _ in streams]
        torch.cuda.synchronize()
        outs = [[] for _ in streams]
        for t in range(1, 9):
            for (run, _), s, o in zip(jobs, streams, outs):
                with torch.cuda.stream(s):
                    o += run(t)
        torch.cuda.synchronize()
        results += [o + list(opt.params + opt.m + opt.v) for o, (_, opt) in zip(outs, jobs)]
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_workspace_waits_for_the_streams_that_use_it(dev):
    """Objects that go while a call on another stream than their workspace's own
    has not run yet: its memory may not come to a tensor of the first stream
    before that."""
    import torch
    g = torch.Generator(device=dev).manual_seed(6)

    def r(*shape):
        return torch.randn(shape, generator=g, device=dev).bfloat16()
    B, T, C = 2, (40, 3000), 1024
    x, dy = (tuple(r(B, t, C) for t in T) for _ in range(2))
    grads = [torch.randn(n, generator=g, device=dev) for n in (3_000_001, 70_000)]
    other = torch.cuda.Stream()
    for by_hand in (False, True):
        op = pkg.AdaLN(B, *T, C, device=dev)
        opt = pkg.AdamW([torch.zeros_like(d) for d in grads], grads=grads)
        stats = op.modulation(x, None, None)["stats"]
        out, norm = op.modulation_bwd(x, None, stats, dy), opt.grad_norm(1.0)
        want = [t.clone() for k in sorted(out) for t in out[k]] + [norm.clone()]
        for t in (*(t for p in out.values() for t in p), norm):
            t.zero_()
        sizes = [op.workspace.numel(), opt.workspace.numel()]
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            torch.cuda._sleep(40_000_000)  # 20 ms ahead of the calls
            if not by_hand:
                op.modulation_bwd(x, None, stats, dy, out=out)
                opt.grad_norm(1.0, out=norm)
        if by_hand:
            op.modulation_bwd(x, None, stats, dy, out=out, stream=other)
            opt.grad_norm(1.0, out=norm, stream=other)
        assert not other.query()
        del op, opt
        junk = [torch.full((n // 4,), float("nan"), device=dev) for n in sizes for _ in range(4)]
        other.synchronize()
        torch.cuda.synchronize()
        got = [t for k in sorted(out) for t in out[k]] + [norm]
        for a, b in zip(got, want):
            assert Hh.bits_equal(a, b)
        del junk
