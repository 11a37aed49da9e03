"""How far X is from the formula's, against the figures that the header states, with the default polynomial and five
iterations: 2^-9 of its norm for dense matrices of 16 rows and columns or more, also where a few directions lead the
others by 100 times; 2^-6 for any other.

X is read without a rounding of its own: a Muon step with momentum 0, update_rms 1 and rate 1 on weights of 0 leaves
-sqrt(max(rows, columns)) X in fp32, off by 2^-23 at most. Where the figures come from: the kernels keep X in fp16, the
first three with codes of what that leaves, about five bits more. A rounding to fp16 is off by 2^-11 / sqrt(12) of a
power of two above the value in the mean square, 1.4e-4 to 2e-4 of X's norm in all directions alike, and two iterations
on from the first X without more bits a small singular value has grown 3.4445^2 = 11.9 times: 2.4e-3 of the norm for
what is lost in the small directions; where these hold a hundredth of the norm and more, they stop growing before the
end, since their values come near 1: half of it. A and B add 3e-4 to 8e-4 (less than 2^-10, as the tests of independent
entries hold), and the rests, which B X does not take, are taken with a coefficient that is off by no more than b s of 4.775 / 3.4445
where s is A's mean: twice that rounding once more for a few rows. 2^-7 = 7.8e-3 holds all of it
where there are enough entries for the roundings' mean square; a few of them may all be half a place off, 2^-11 for
2^-11 / sqrt(12) of a power of two: 2^-6."""

import numpy as np
import pytest

import invariant_mmdit_joint_gb300 as pkg
from oracle import projection_ops as O
from tests.test_gpu_muon import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def spectrum(dev, rows, cols, kind):
    """fp32. (rank, lead): independent entries and ``rank`` directions ``lead`` times as strong an entry; "1/i": singular
    values 1, 1/2, 1/3 ..; "steps": from 1 to 10^-4 in equal ratios; "rank 3": nothing beside three directions."""
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(rows * 7 + cols)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.float64)  # noqa: E731
    r = min(rows, cols)
    if kind in ("1/i", "steps"):
        s = 1.0 / torch.arange(1, r + 1, device=dev) if kind == "1/i" else torch.logspace(0, -4, r, device=dev)
        x = torch.linalg.qr(rnd(rows, r))[0] * s.double() @ torch.linalg.qr(rnd(cols, r))[0].T
    elif kind == "rank 3":
        x = rnd(rows, 3) @ rnd(3, cols)
    else:
        x = rnd(rows, cols) + kind[1] * rnd(rows, kind[0]) @ rnd(kind[0], cols)
    return (1e-3 * x).float()


def update_of(x):
    import torch
    p = torch.zeros_like(x, dtype=torch.float32)
    pkg.Muon([p], lr=1.0, momentum=0.0, nesterov=False, weight_decay=0.0, update_rms=1.0, grads=[x]).step()
    pkg.rlk_joint_attn_check_status()
    return -f64(p) / np.sqrt(max(x.shape))


# one kernel's (one CTA, a few, eight; 64 and 128 rows; odd and aligned rows, tall and wide), and the large ones
SIZES = [(16, 1160), (1160, 16), (64, 700), (701, 63), (64, 2567), (64, 4000), (4001, 50), (33, 9000), (32, 33), (128, 1000),
         (1000, 127), (100, 4001), (130, 300), (300, 1000), (1000, 300), (301, 999), (999, 301), (512, 512), (768, 1536)]
KINDS = [(0, 0), (4, 1), (4, 10), (4, 30), (1, 100), "1/i"]


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("rows, cols", SIZES)
def test_documented_error(dev, rows, cols, kind):
    x = spectrum(dev, rows, cols, kind)
    exact, norm = O.orthogonal(f64(x)), np.linalg.norm
    err = norm(update_of(x) - exact) / norm(exact)
    print(f"{rows} x {cols} {kind}: {err:.2e}")
    assert err <= 2.0 ** -9, err
    # what goes to bf16: no more than its rounding beside it
    got = f64(pkg.orthogonalize([x])[0])
    assert norm(got - exact) <= (2.0 ** -9 + 2.0 ** -8) * norm(exact)


@pytest.mark.parametrize("kind", [(1, 10000), "steps", "rank 3"], ids=str)
@pytest.mark.parametrize("rows, cols", SIZES)
def test_documented_error_of_far_leading_directions(dev, rows, cols, kind):
    x = spectrum(dev, rows, cols, kind)
    exact, norm = O.orthogonal(f64(x)), np.linalg.norm
    err = norm(update_of(x) - exact) / norm(exact)
    print(f"{rows} x {cols} {kind}: {err:.2e}")
    assert err <= 2.0 ** -7, err


def test_documented_error_of_few_rows_and_entries(dev):
    """One list of many: up to 15 rows, from one column to 1200, each kind of spectrum; one entry a row."""
    import torch
    rng = np.random.default_rng(3)
    xs = []
    for i in range(400):
        r, k = int(rng.integers(1, 16)), int(np.exp(rng.uniform(0, 7.1)))
        x = spectrum(dev, r, k, [*KINDS, (1, 1000), (1, 10000), "steps", "rank 3"][i % 10])
        xs.append(x if i % 3 else x.T.contiguous())
    for r, k in ((16, 16), (40, 50), (109, 20), (200, 200), (300, 140)):
        x = torch.zeros((r, k), device=dev)
        x[range(min(r, k)), range(min(r, k))] = torch.from_numpy(np.exp(rng.standard_normal(min(r, k)))).float().to(dev)
        xs.append(x)
    ps = [torch.zeros_like(x) for x in xs]
    pkg.Muon(ps, lr=1.0, momentum=0.0, nesterov=False, weight_decay=0.0, update_rms=1.0, grads=xs).step()
    pkg.rlk_joint_attn_check_status()
    worst = 0.0
    for x, p in zip(xs, ps):
        exact, norm = O.orthogonal(f64(x)), np.linalg.norm
        err = norm(-f64(p) / np.sqrt(max(x.shape)) - exact) / norm(exact)
        worst = max(worst, err)
        # (one row: three X's are rounded whole, 2^-11 each, and grow 1.3 times an iteration: 2e-3; D's roundings as much)
        assert err <= (2.0 ** -6 if min(x.shape) > 1 else 2.0 ** -8), (tuple(x.shape), err)
    print(f"worst {worst:.2e}")


@pytest.mark.parametrize("kind", [(0, 0), (4, 10), (4, 30), (1, 100), "1/i"], ids=str)
@pytest.mark.parametrize("rows, cols", [(16, 1160), (700, 64), (100, 1000), (300, 1000), (1000, 301)])
def test_no_further_off_than_the_stated_roundings(dev, rows, cols, kind):
    """The kernels' form with exact sums is d away from the formula's. The kernels are another draw of the same roundings
    (halfway cases and fp32 sums that fall on the other side): 2 d. d is the largest of a few draws, since a matrix of a
    few rows has few roundings to it."""
    x = spectrum(dev, rows, cols, kind)
    u, norm = f64(x), np.linalg.norm
    exact = O.orthogonal(u)
    d = max(norm(O.orthogonal_as_kept(u, lead=f) - exact) for f in (1.0, 1.23, 1.52, 1.83))
    assert norm(update_of(x) - exact) <= 2 * d
