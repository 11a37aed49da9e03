"""The gradient norm and AdamW on the GPU against their 64-bit definitions,
within the bounds that come with these, and the 8-bit states bit by bit."""

import numpy as np
import pytest

import invariant_mmdit_joint_gb300 as pkg
from oracle import block_ops as O
from tests import _helpers as Hh

pytestmark = pytest.mark.gpu
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8)
SIZES = [1, 7, 8, 31, 32, 33, 255, 2048, 2049, 4096, 4100, 12345, 100_003]


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


def make(dev, sizes, bits, seed=1, **kw):
    """Parameters (every second one bf16 with a master), gradients of both types, and the optimiser."""
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def r(n, s=1.0):
        return torch.randn(n, generator=g, device=dev) * s
    masters = [r(n, 0.05) if i % 2 else None for i, n in enumerate(sizes)]
    params = [m.bfloat16() if m is not None else r(n, 0.05) for m, n in zip(masters, sizes)]
    grads = [r(n, 10.0 ** ((i % 7) - 5)).to(torch.bfloat16 if i % 3 else torch.float32) for i, n in enumerate(sizes)]
    kw = {**dict(lr=HYPER["lr"], betas=(HYPER["beta1"], HYPER["beta2"]), eps=HYPER["eps"],
                 weight_decay=[0.1 * (i % 2) for i in range(len(sizes))],
                 lr_scale=[1.0 + 0.5 * (i % 3) for i in range(len(sizes))], seed=77), **kw}
    return pkg.AdamW(params, masters=masters, state_bits=bits, grads=grads, **kw), grads


def truth(opt, i):
    return opt.params[i] if opt.masters[i] is None else opt.masters[i]


def state(opt, i):
    """m and v of a parameter in 64 bits."""
    import torch
    if opt.state_bits == 32:
        return f64(opt.m[i]), f64(opt.v[i])
    u = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
    return O.decode(u(opt.m[i]), u(opt.m_scale[i])), O.decode(u(opt.v[i]), u(opt.v_scale[i]))


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_against_the_definition(dev, bits):
    import torch
    opt, grads = make(dev, SIZES, bits)
    for step in (1, 2, 3, 500):
        before = [(f64(truth(opt, i)), *state(opt, i)) for i in range(len(SIZES))]
        opt.step(step)
        for i, (p, m, v) in enumerate(before):
            (p1, m1, v1), (pe, me, ve) = O.adamw(
                p, f64(grads[i]), m, v, **{**HYPER, "lr": HYPER["lr"] * (1.0 + 0.5 * (i % 3))},
                weight_decay=0.1 * (i % 2), step=step)
            got = f64(truth(opt, i))
            assert np.all(np.abs(got - p1) <= pe + 1e-37), (bits, step, i, np.max(np.abs(got - p1) / (pe + 1e-37)))
            if opt.masters[i] is not None:
                assert Hh.bits_equal(opt.params[i], opt.masters[i].bfloat16())
            gm, gv = state(opt, i)
            if bits == 32:
                assert np.all(np.abs(gm - m1) <= me + 1e-37) and np.all(np.abs(gv - v1) <= ve + 1e-37), (step, i)
                continue
            # 8 bits: less than a step (2^-3 of the value's power of two, 2^-9 of the scale) around the fp32 value
            for got, value, err, s in ((gm, m1, me, opt.m_scale[i]), (gv, v1, ve, opt.v_scale[i])):
                scale = np.repeat(2.0 ** (s.cpu().numpy().astype(float) - 127), 32)[:value.size]
                gap = np.maximum(np.abs(value) * 2.0 ** -3, scale * 2.0 ** -9) + err
                assert np.all(np.abs(got - value) <= gap), (step, i)
    assert all(bool(torch.isfinite(truth(opt, i)).all()) for i in range(len(SIZES)))


def test_moments_bit_by_bit(dev):
    """Each product and sum rounded by itself, as numpy's float32 does."""
    import torch
    n, f = 1_000_003, np.float32
    g = torch.Generator(device=dev).manual_seed(8)
    p, m, d = (torch.randn(n, generator=g, device=dev) for _ in range(3))
    v = torch.rand(n, generator=g, device=dev)
    m0, v0, d0 = (t.cpu().numpy() for t in (m, v, d))
    pkg.AdamW([p], betas=(0.9, 0.95), m=[m], v=[v], grads=[d]).step(3)
    o1, o2 = f(1 - 0.9), f(1 - 0.95)
    np.testing.assert_array_equal(m.cpu().numpy(), f(0.9) * m0 + o1 * d0)
    np.testing.assert_array_equal(v.cpu().numpy(), f(0.95) * v0 + (o2 * d0) * d0)


def test_eight_bit_states_bit_by_bit(dev):
    """The codes and scales follow from the fp32 moments and the hash's random bits."""
    import torch
    keys = [3 * i + 5 for i in range(len(SIZES))]
    opt, grads = make(dev, SIZES, 8, keys=keys)
    f, b1, b2 = np.float32, np.float32(0.9), np.float32(0.95)
    o1, o2 = f(1 - 0.9), f(1 - 0.95)
    scale = torch.tensor([0.37], device=dev)
    for step in (1, 2, 9):
        before = [state(opt, i) for i in range(len(SIZES))]
        opt.step(step, grad_scale=scale)
        for i, (m, v) in enumerate(before):
            g = grads[i].float().cpu().numpy() * f(0.37)
            m1, v1 = b1 * m.astype(f) + o1 * g, b2 * v.astype(f) + (o2 * g) * g
            assert m1.dtype == f and v1.dtype == f
            rnd = O.random_bits(77, step, keys[i], m.size)
            for name, value, part, positive in (("m", m1, rnd & 0xFFFF, False), ("v", v1, rnd >> 16, True)):
                q, s = O.encode(value, part, positive)
                got = getattr(opt, name)[i].view(torch.uint8).cpu().numpy()
                np.testing.assert_array_equal(getattr(opt, name + "_scale")[i].cpu().numpy(), s)
                np.testing.assert_array_equal(got, q)


def test_the_quotient_over_the_whole_range(dev):
    """p = -m / (sqrt(v) + eps), from v = 0 and subnormal v to v near the type's
    end, for several eps: with beta 0.5 and no gradient m and v halve exactly,
    at step 60 the corrections are 1, and p starts from 0 with a rate of 1.
    Square root and quotient are within one unit in the last place (2u each),
    their operand d = sqrt(v) + eps is rounded once, v below 2^-100 is moved
    by 2^-124 - 40 (at most 2^-82 in its root)."""
    import torch
    rng = np.random.default_rng(8)
    v = np.concatenate([[0.0, 2.0 ** -149, 2.0 ** -148, 2.0 ** -126, 2.0 ** 85, 2.0 ** 86, 2.0 ** 87, 3e38],
                        2.0 ** rng.uniform(-149, 128, 40_000), 2.0 ** rng.uniform(-60, 0, 40_000)])
    v = np.minimum(v, 3e38).astype(np.float32)
    m = (rng.standard_normal(v.size) * np.maximum(np.sqrt(v.astype(np.float64)), 1e-25)).astype(np.float32)
    # halves that are exact: no subnormal operand may lose its last bit
    v, m = np.where(v < 2.0 ** -125, 0.0, v).astype(np.float32), np.where(np.abs(m) < 2.0 ** -125, 0.0, m).astype(np.float32)
    tiny = 2.0 ** -149 * rng.integers(0, 1 << 20, 4096) * 2
    v, m = np.concatenate([v, tiny.astype(np.float32)]), np.concatenate([m, np.full(4096, 1e-25, np.float32)])
    for eps in (2.0 ** -50, 1e-15, 1e-8, 1.0):
        p = torch.zeros(v.size, device=dev)
        opt = pkg.AdamW([p], grads=[torch.zeros(v.size, device=dev)], m=[torch.from_numpy(m).to(dev)],
                        v=[torch.from_numpy(v).to(dev)], lr=1.0, betas=(0.5, 0.5), eps=eps, weight_decay=0.0)
        opt.step(60)
        root = np.sqrt(v.astype(np.float64) / 2)
        eps32 = float(np.float32(eps))
        d = root + eps32
        want = -(m.astype(np.float64) / 2) / d
        bound = np.abs(want) * (2 * O.U * root / d + 2.0 ** -82 / d + 3 * O.U) * 1.001 + 2.0 ** -149
        assert np.all(np.abs(f64(p) - want) <= bound), (eps, np.max(np.abs(f64(p) - want) / bound))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_does_not_depend_on_its_list(dev, bits):
    """One list, and each tensor by itself under the same key: the same bytes; a list past one launch's entries too."""
    sizes = (SIZES * 45)[:560]
    opt, grads = make(dev, sizes, bits, weight_decay=0.01, lr_scale=1.0)
    copies = [(truth(opt, i).clone(), grads[i]) for i in range(len(sizes))]
    for step in (1, 2):
        opt.step(step)
    for i in (0, 5, 12, 254, 255, 256, 257, 511, 512, 559):
        p, g = copies[i]
        one = pkg.AdamW([p], state_bits=bits, lr=HYPER["lr"], betas=(0.9, 0.95), weight_decay=0.01, seed=77, keys=[i],
                        grads=[g])
        for step in (1, 2):
            one.step(step)
        assert Hh.bits_equal(p, truth(opt, i)), i
        for a, b in ((one.m[0], opt.m[i]), (one.v[0], opt.v[i])):
            import torch
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


def test_a_run_resumes_from_its_tensors(dev):
    """Stopped after two steps and taken up by a new object from copies of the tensors: the same bytes."""
    import torch
    for bits in (32, 8):
        a, grads = make(dev, SIZES, bits)
        for step in (1, 2):
            a.step(step)
        copy = lambda ts: [None if t is None else t.clone() for t in ts]  # noqa: E731
        state = dict(m=copy(a.m), v=copy(a.v))
        if bits == 8:
            state.update(m_scale=copy(a.m_scale), v_scale=copy(a.v_scale))
        b = pkg.AdamW(copy(a.params), masters=copy(a.masters), state_bits=bits, lr=HYPER["lr"], betas=(0.9, 0.95),
                      weight_decay=[0.1 * (i % 2) for i in range(len(SIZES))],
                      lr_scale=[1.0 + 0.5 * (i % 3) for i in range(len(SIZES))], seed=77, grads=grads, **state)
        for opt in (a, b):
            opt.step(3)
        for x, y in zip(a.params + a.m + a.v, b.params + b.m + b.v):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), bits


@pytest.mark.parametrize("count", [4, 30])
def test_one_list_of_both_kinds_of_state(dev, count):
    """Tensors with 32-bit and 8-bit states in one call, in short and long lists: the bytes of two calls."""
    import torch
    sizes = (SIZES * 4)[:count]
    pair = [[make(dev, sizes, bits, seed=4)[0] for bits in (32, 8)] for _ in range(2)]
    for opt in pair[0]:
        opt.step(1)
    both = (pkg.AdamwTensor * (2 * count))()
    for i in range(count):  # alternating
        both[2 * i], both[2 * i + 1] = pair[1][0]._list[i], pair[1][1]._list[i]
    args = pkg.AdamwArgs.from_buffer_copy(pair[1][0]._args)
    args.step, args.lr = 1, HYPER["lr"]
    pkg.rlk_adamw_step(both, 2 * count, args)
    for a, b in zip(*pair):
        for x, y in zip(a.params + a.m + a.v, b.params + b.m + b.v):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("sizes", [[1], [5, 0, 4097], SIZES, [3_000_001]], ids=str)
def test_gradient_norm(dev, sizes):
    import torch
    opt, grads = make(dev, sizes, 32)
    want = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
    # a chunk's squares: 16 in a thread, 5 shuffles, 8 warps, in fp32; half of that in the root; three roundings
    tol = (0.5 * (16 + 5 + 8 + 2) + 3) * O.U
    for pre, most in ((1.0, float("inf")), (0.25, want / 10), (1.0, 2 * want)):
        got = f64(opt.grad_norm(most, pre_scale=pre))
        assert abs(got[0] - pre * want) <= tol * pre * want
        factor = pre * min(1.0, most / (pre * want + 1e-6))
        assert abs(got[1] - factor) <= 2 * tol * factor
    again = opt.grad_norm(2.0)
    assert Hh.bits_equal(again, opt.grad_norm(2.0))


def test_a_norm_that_is_not_finite_leaves_everything(dev):
    import torch
    for bits in (32, 8):
        opt, grads = make(dev, SIZES, bits)
        opt.step(1)
        keep = [t.clone() for t in opt.params + opt.masters + opt.m + opt.v if t is not None]
        for bad in (float("nan"), float("inf"), 3e30):  # the last one's square is not finite
            grads[-1][17] = bad
            n = opt.grad_norm(1.0)
            assert not bool(torch.isfinite(n[0])) and bool(torch.isnan(n[1]))
            opt.step(2, grad_scale=n[1:])
            now = [t for t in opt.params + opt.masters + opt.m + opt.v if t is not None]
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(now, keep))


def test_non_finite_gradients_without_a_norm(dev):
    """A NaN stays in its element with 32-bit states; with 8-bit ones its block of 32 reads as NaN from then on."""
    import torch
    for bits in (32, 8):
        p = torch.zeros(100, device=dev)
        g = torch.ones(100, device=dev)
        g[40] = float("nan")
        opt = pkg.AdamW([p], state_bits=bits, grads=[g])
        opt.step(1)
        assert torch.isnan(p).nonzero().flatten().tolist() == [40]
        if bits == 8:
            assert opt.m_scale[0].tolist()[1] == 255 and opt.v_scale[0].tolist()[1] == 255
            opt.step(2)
            assert torch.isnan(p).nonzero().flatten().tolist() == list(range(32, 64))


def test_extreme_values_in_eight_bits(dev):
    import torch
    n = 64
    g = torch.zeros(n, device=dev)
    g[0], g[1], g[2] = 1e-18, -1e-30, 1e-38     # squares that vanish, a subnormal
    g[32], g[33], g[34] = 1e18, 1.0, -1e-4      # a block of one giant
    p = torch.zeros(n, device=dev)
    opt = pkg.AdamW([p], state_bits=8, grads=[g], lr=1e-3, weight_decay=0.0, seed=5)
    opt.step(1)
    assert bool(torch.isfinite(p).all())
    rnd = O.random_bits(5, 1, 0, n)
    x = g.cpu().numpy()
    f = np.float32
    m1, v1 = f(1 - 0.9) * x, (f(1 - 0.999) * x) * x
    for name, value, part, positive in (("m", m1, rnd & 0xFFFF, False), ("v", v1, rnd >> 16, True)):
        q, s = O.encode(value, part, positive)
        np.testing.assert_array_equal(getattr(opt, name + "_scale")[0].cpu().numpy(), s)
        np.testing.assert_array_equal(getattr(opt, name)[0].view(torch.uint8).cpu().numpy(), q)


def test_the_rounding_keeps_slow_moments_moving(dev):
    """With beta2 = 0.999 a second moment moves by a thousandth a step, far
    below half a code. Its mean over many elements still follows the running
    average: 4096 elements from 0 toward g^2 = 1 over 200 steps."""
    import torch
    n = 4096
    g = torch.ones(n, device=dev)
    opt = pkg.AdamW([torch.zeros(n, device=dev)], state_bits=8, grads=[g], betas=(0.9, 0.999), lr=0.0, seed=11)
    for step in range(1, 201):
        opt.step(step)
    _, v = state(opt, 0)
    want = 1 - 0.999 ** 200
    # a step's rounding has a variance of at most (change) * (code step = v / 8): relative standard deviation of one
    # element below sqrt(sum of 0.001 / (8 v_t)) < 0.5, of the mean over 4096 below 0.008; four of those
    assert abs(v.mean() / want - 1) < 0.032, v.mean() / want


def test_captured_steps_follow_their_counter(dev):
    import torch
    for bits in (32, 8):
        a, grads = make(dev, SIZES, bits)
        b, _ = make(dev, SIZES, bits)
        lr = torch.tensor([1e-3], device=dev)
        count = torch.zeros(1, dtype=torch.int64, device=dev)
        out, s, graph = torch.empty(2, device=dev), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        b.grad_norm(1.0, out=out)  # allocates the workspace
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                count.add_(1)
                b.grad_norm(1.0, out=out)
                b.step(count, lr=lr, grad_scale=out[1:])
        torch.cuda.current_stream().wait_stream(s)
        for step in range(1, 6):
            rate = 1e-3 / step
            lr.fill_(rate)
            n = a.grad_norm(1.0)
            a.step(step, lr=float(np.float32(rate)), grad_scale=n[1:])
            graph.replay()
            torch.cuda.synchronize()
            assert Hh.bits_equal(n, out)
            for x, y in zip(a.params + a.m + a.v, b.params + b.m + b.v):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (bits, step)


def test_elements_behind_the_tensors_stay(dev):
    import torch
    for bits in (32, 8):
        for n in (1, 9, 33, 2047, 4099):
            bufs = {}

            def view(name, dtype, size, fill=0):
                bufs[name] = torch.full((size + 256,), 1, dtype=torch.float32, device=dev).to(dtype)
                t = bufs[name][:size]
                t.copy_(torch.full((size,), fill, dtype=torch.float32, device=dev).to(dtype))
                return t
            code = torch.float8_e4m3fn if bits == 8 else torch.float32
            kw = dict(m=[view("m", code, n)], v=[view("v", code, n)])
            if bits == 8:
                kw.update(m_scale=[view("ms", torch.uint8, -(-n // 32))], v_scale=[view("vs", torch.uint8, -(-n // 32))])
            opt = pkg.AdamW([view("p", torch.bfloat16, n, 0.5)], masters=[view("w", torch.float32, n, 0.5)],
                            state_bits=bits, grads=[view("g", torch.bfloat16, n, 0.25)], **kw)
            opt.step(1, grad_scale=opt.grad_norm(1.0)[1:])
            torch.cuda.synchronize()
            for name, b in bufs.items():
                size = -(-n // 32) if name in ("ms", "vs") else n
                assert bool((b[size:].float() == 1).all()), (bits, n, name)


def test_a_tensor_past_32_bits(dev):
    """More than 2^32 elements with 8-bit states: the last ones are updated like the first."""
    import torch
    n = 2 ** 32 + 4097
    p = torch.zeros(n, device=dev)
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=dev)
    g[-1] = -2.0
    opt = pkg.AdamW([p], state_bits=8, grads=[g], lr=1e-2, weight_decay=0.0)
    norm = f64(opt.grad_norm(float("inf")))[0]
    assert abs(norm / np.sqrt((n - 1) * 0.25 + 4.0) - 1) < 40 * O.U
    opt.step(1)
    assert torch.equal(p[:4096], p[2 ** 32:2 ** 32 + 4096])
    # the first step is lr * |g| / (|g| + eps): 1 - 2e-8 of lr for |g| = 0.5, 1 - 5e-9 for |g| = 2, each with the
    # definition's 8u of roundings, so the two sizes are not equal but at most 1.5e-8 + 16u apart
    assert float(p[0]) < 0 and abs(float(p[-1]) / -float(p[0]) - 1) <= 1.5e-8 + 16 * O.U
    # the hash repeats after 2^32 elements
    assert torch.equal(opt.m[0].view(torch.uint8)[:4096], opt.m[0].view(torch.uint8)[2 ** 32:2 ** 32 + 4096])


def test_a_nan_stays_in_its_block_in_long_chunks(dev):
    """A block that reads as NaN must not reach the tensor's last block, 2048
    elements on: a list long enough for chunks of two passes, a last block of
    less than 25 elements (threads past the end share its exchanges), and the
    bytes of the tensor stepped alone, in chunks of one pass."""
    import torch
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    g = torch.Generator(device=dev).manual_seed(6)
    for n in (2048 + 32 + 1, 2048 + 32 + 8, 2048 + 64 + 24, 4096 + 13):
        grad = torch.randn(n, generator=g, device=dev)
        grad[n - n % 32 - 2048 + 9] = float("nan")
        grads = [grad, torch.randn(8 * sms * 4096 + 5, generator=g, device=dev)]
        opts = [pkg.AdamW([torch.zeros_like(t) for t in grads[:k]], state_bits=8, grads=grads[:k], seed=3) for k in (1, 2)]
        for step in (1, 2, 3):
            for opt in opts:
                opt.step(step)
        for name in ("params", "m", "v", "m_scale", "v_scale"):
            a, b = (getattr(opt, name)[0] for opt in opts)
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (n, name)
        assert opts[1].m_scale[0][-1] != 255 and bool(torch.isfinite(opts[1].params[0][-(n % 32):]).all()), n


def test_a_counter_out_of_range_leaves_everything(dev):
    """A device counter that was not advanced before the first step, or has run over."""
    import torch
    for bits in (32, 8):
        opt, _ = make(dev, SIZES, bits)
        opt.step(1)
        tensors = [t for t in opt.params + opt.masters + opt.m + opt.v + opt.m_scale + opt.v_scale if t is not None]
        keep = [t.clone() for t in tensors]
        for t in (0, -1, 2 ** 31, -2 ** 63, 2 ** 32 + 5):
            opt.step(torch.tensor([t], device=dev))
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(tensors, keep)), t
        opt.step(torch.tensor([2 ** 31 - 1], device=dev))
        assert not torch.equal(opt.params[-1], keep[len(SIZES) - 1])


@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.5, 0.99999), (1 - 2.0 ** -12, 1 - 2.0 ** -20), (0.0, 0.3)], ids=str)
def test_a_step_number_on_the_device_gives_the_bytes_of_an_ordinary_one(dev, betas):
    """The corrections 1 - beta^t are the same numbers wherever they are computed."""
    import torch
    rng = np.random.default_rng(2)
    steps = [*range(1, 1500), *(int(t) for t in np.unique((2 ** rng.uniform(11, 31, 1500)).astype(np.int64))), 2 ** 31 - 1]
    steps = [t for t in steps if t < 2 ** 31]
    grads = [torch.tensor([1.0, -0.3], device=dev)]
    opts = [pkg.AdamW([torch.zeros(2, device=dev)], grads=grads, betas=betas, lr=1e-2) for _ in range(2)]
    device = torch.tensor(steps, device=dev)
    out = torch.empty(2, len(steps), 2, device=dev)
    for i, t in enumerate(steps):
        for k, opt in enumerate(opts):
            for s in (opt.params[0], opt.m[0], opt.v[0]):
                s.zero_()
            opt.step(device[i] if k else t)
            out[k, i] = opt.params[0]
    same = (out[0].view(torch.int32) == out[1].view(torch.int32)).all(1)
    assert bool(same.all()), [steps[i] for i in (~same).nonzero().flatten().tolist()][:10]


@pytest.mark.parametrize("t, bit", [(1, 24), (3, 20), (7, 15), (1, 10)])
def test_the_quotient_under_large_corrections(dev, t, bit):
    """beta2 = 1 - 2^-bit in its first steps: 1 / sqrt(1 - beta2^t) far above 1,
    second moments of 0 and near it, the smallest eps."""
    import torch
    beta2 = 1 - 2.0 ** -bit
    rng = np.random.default_rng(9)
    v = np.concatenate([np.zeros(512), 2.0 ** rng.uniform(-125, -60, 4096)]).astype(np.float32)
    m = (rng.standard_normal(v.size) * 1e-20).astype(np.float32)
    for eps in (2.0 ** -50, 2.0 ** -40, 1e-8):
        p, mm, vv = (torch.from_numpy(a).to(dev) for a in (np.zeros_like(m), m, v))
        pkg.AdamW([p], grads=[torch.zeros_like(p)], m=[mm], v=[vv], lr=1.0, betas=(0.5, beta2), eps=eps,
                  weight_decay=0.0).step(t)
        c1, c = 1 - 0.5 ** t, 1 / np.sqrt(-np.expm1(t * np.log1p(-2.0 ** -bit)))
        root = np.sqrt(f64(vv)) * c  # of the moments that the step left
        d = root + float(np.float32(eps))
        want = -f64(mm) / c1 / d
        # root 2u, c and d u, the quotient 2u, rate / c1 (c1 is exact) and its product u each
        bound = np.abs(want) * (3 * O.U * root / d + 2.0 ** -27 + 5 * O.U) * 1.001 + 2.0 ** -149
        assert np.all(np.abs(f64(p) - want) <= bound), (eps, np.max(np.abs(f64(p) - want) / bound))


def test_the_quotient_of_the_smallest_moments(dev):
    """|m| about the smallest normal value, where the residual m - d q of the
    quotient's correction falls below the type's last bit. With an estimate of
    1 / d within 2u, q is within 3u and the residual at most 3u |m|; its rounding
    adds 2^-150, at most u |m| of a normal m, so the quotient is within 2u; of a
    subnormal m it adds at most the residual itself, 4u in all."""
    import torch
    rng = np.random.default_rng(10)
    normal = 2.0 ** rng.uniform(-124.9, -95, 20_000)
    tiny = 2.0 ** -148 * rng.integers(1, 1 << 22, 20_000)  # halves that are exact
    m = (np.concatenate([normal, tiny]) * rng.choice([-1, 1], 40_000)).astype(np.float32)
    v = (2.0 ** rng.uniform(-100, 10, m.size)).astype(np.float32)
    p = torch.zeros(m.size, device=dev)
    pkg.AdamW([p], grads=[torch.zeros_like(p)], m=[torch.from_numpy(m).to(dev)], v=[torch.from_numpy(v).to(dev)],
              lr=2.0 ** 40, betas=(0.5, 0.5), eps=2.0 ** -50, weight_decay=0.0).step(60)
    half = m.astype(np.float64) / 2
    root = np.sqrt(v.astype(np.float64) / 2)
    d = root + 2.0 ** -50
    want = -half / d * 2.0 ** 40
    # d is rounded once; two roundings of q below the type's last bit, 2^40 of rate times
    units = np.where(np.abs(half) >= 2.0 ** -126, 2, 4) + 1
    bound = np.abs(want) * (2 * O.U * root / d + units * O.U) * 1.001 + 2.0 ** -109
    assert np.all(np.abs(f64(p) - want) <= bound), np.max(np.abs(f64(p) - want) / bound)


def test_the_norm_sums_in_the_stated_order(dev):
    """out[0] bit by bit, of bfloat16 gradients (whose squares fp32 holds): the
    squares of a thread's eight elements of each pass in order, exchanges, warps
    ascending; in 64 bits every 1024th chunk of the list, exchanges twice."""
    import torch
    f = np.float32
    sizes = [5, 16384, 16385, 40_000, 1040 * 16384 + 77]
    g = torch.Generator(device=dev).manual_seed(13)
    grads = [(torch.randn(n, generator=g, device=dev) * 10.0 ** -i).bfloat16() for i, n in enumerate(sizes)]
    opt = pkg.AdamW([torch.zeros(n, device=dev) for n in sizes], grads=grads)
    got = opt.grad_norm(1.0).cpu().numpy()[0]

    def fold(x, lanes):
        while lanes > 1:
            lanes //= 2
            x = x + x[..., np.arange(x.shape[-1]) ^ lanes]
        return x[..., 0]
    chunks = []
    for d in grads:
        x = d.float().cpu().numpy()
        x = np.pad(x, (0, -x.size % 16384)).reshape(-1, 8, 256, 8)  # chunk, pass, thread, element
        s = np.zeros((x.shape[0], 256), f)
        for j in range(8):
            for i in range(8):
                s = s + x[:, j, :, i] ** 2
        s = fold(s.reshape(-1, 8, 32), 32)
        total = s[:, 0]
        for w in range(1, 8):
            total = total + s[:, w]
        assert total.dtype == f
        chunks.append(total)
    part = np.concatenate(chunks).astype(np.float64)
    lanes = np.zeros(1024)
    for i in range(0, part.size, 1024):
        row = part[i:i + 1024]
        lanes[:row.size] = lanes[:row.size] + row
    total = fold(fold(lanes.reshape(32, 32), 32)[None], 32)[0]
    assert got == np.sqrt(f(total))


def test_long_chunks_step_like_short_ones(dev):
    """Chunks of two, four and eight passes, whose copies ahead go round their
    stages several times: the bytes of each tensor stepped alone in chunks of
    one pass, from states of a step before, gradients and parameters of both types."""
    import torch
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    for passes in (2, 4, 8):
        count = 6
        share = 8 * sms * 2048 * passes // count
        sizes = [share + 16385 * passes + 321 * i for i in range(count)]  # chunks that do not come out even
        if passes == 8:  # each still below the length from which a tensor alone takes two passes
            sizes = [min(n, 8 * sms * 4096 - 4097 + 31 * i) for i, n in enumerate(sizes)]
        assert sum(n // (2048 * passes) for n in sizes) >= 8 * sms and all(-(-n // 4096) < 8 * sms for n in sizes)
        opt, grads = make(dev, sizes, 8, weight_decay=0.01, lr_scale=1.0)
        copies = [truth(opt, i).clone() for i in range(count)]
        for step in (1, 2):
            opt.step(step)
        for i in range(count):
            p = copies[i].bfloat16() if opt.masters[i] is not None else copies[i]
            one = pkg.AdamW([p], masters=[copies[i]] if opt.masters[i] is not None else None, state_bits=8,
                            lr=HYPER["lr"], betas=(0.9, 0.95), weight_decay=0.01, seed=77, keys=[i], grads=[grads[i]])
            for step in (1, 2):
                one.step(step)
            for a, b in ((truth(one, 0), truth(opt, i)), (p, opt.params[i]), (one.m[0], opt.m[i]), (one.v[0], opt.v[i]),
                         (one.m_scale[0], opt.m_scale[i]), (one.v_scale[0], opt.v_scale[i])):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (passes, i)


def test_the_functions_give_the_bytes_of_the_class(dev):
    """rlk_grad_norm and rlk_adamw_step on a list of the caller's own, tensors and sizes in hand."""
    import torch
    (a, _), (b, _) = (make(dev, SIZES, 8, seed=6) for _ in range(2))
    n = len(SIZES)
    ws = torch.empty(pkg.rlk_grad_norm_workspace_bytes(b._list, n), dtype=torch.uint8, device=dev)
    out = torch.empty(2, device=dev)
    args = pkg.AdamwArgs.from_buffer_copy(b._args)
    args.step, args.grad_scale, args.lr = 4, out[1:].data_ptr(), HYPER["lr"]
    pkg.rlk_grad_norm(b._list, n, 0.5, 3.0, out, ws)
    pkg.rlk_adamw_step(b._list, n, args)
    want = a.grad_norm(3.0, pre_scale=0.5)
    a.step(4, grad_scale=want[1:])
    assert Hh.bits_equal(out, want)
    for name in ("params", "m", "v", "m_scale", "v_scale"):
        for x, y in zip(getattr(a, name), getattr(b, name)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name
    with pytest.raises(pkg.RlkError):
        pkg.rlk_grad_norm(b._list, n, 0.5, 3.0, out, ws[:-1])
