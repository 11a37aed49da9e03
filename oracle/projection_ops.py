"""64-bit definitions of the 8-bit projections and of Muon's orthogonal update
(numpy), which the tests compare the kernels with.

``quantize`` rounds to codes with a power-of-two scale a block; ``orthogonal``
runs the Newton-Schulz products, exactly or with X, A and B rounded whole to fp16;
``orthogonal_as_kept`` has the kernels' own form and roundings."""

from __future__ import annotations

import numpy as np

# significant bits after the first, smallest normal exponent, largest value, exponent of the largest
FORMATS = {"e4m3": (3, -6, 448.0, 8), "e5m2": (2, -14, 57344.0, 15)}
BLOCK = 128
POLYNOMIAL = (3.4445, -4.7750, 2.0315)


def quantize(x, tall, wide, fmt="e4m3"):
    """(values, exponents): x [rows, cols] on the grid of its codes, and each
    block's scale exponent [ceil(rows / tall), ceil(cols / wide)]. An infinity or
    NaN becomes NaN and takes no part in its block's scale."""
    x = np.asarray(x, np.float64)
    digits, low, top, _ = FORMATS[fmt]
    out = np.empty_like(x)
    rows, cols = x.shape
    exps = np.empty((-(-rows // tall), -(-cols // wide)), np.int64)
    for i in range(exps.shape[0]):
        for j in range(exps.shape[1]):
            part = np.s_[i * tall:(i + 1) * tall, j * wide:(j + 1) * wide]
            v = x[part]
            live = np.isfinite(v)
            most = np.max(np.abs(v[live]), initial=0.0)
            e = -126
            while most > top * 2.0 ** e:  # the smallest e with most <= top 2^e
                e += 1
            exps[i, j] = e
            v = np.where(live, v, 0.0) * 2.0 ** -e
            _, k = np.frexp(v)
            step = np.exp2(np.maximum(k - 1, low) - digits)
            out[part] = np.where(live, np.rint(v / step) * step * 2.0 ** e, np.nan)
    return out, exps


def product_bound(a, b, bias=None):
    """Largest error of a computed a b^T (+ bias), per element, before the output's rounding: a matrix instruction
    (32 terms) cuts its sum to no fewer bits than 2^-22 of the terms' magnitudes, 16 of them share a chunk's
    accumulator: 2^-18; K / 512 chunks added in fp32, 2^-24 of the sums so far each; the bias the same."""
    terms = np.abs(a) @ np.abs(b).T
    if bias is not None:
        terms = terms + np.abs(bias)
    return terms * (2.0 ** -18 + (a.shape[1] / 512 + 2) * 2.0 ** -24)


def _half(x):
    return x.astype(np.float16).astype(np.float64)


def orthogonal(u, iterations=5, coefficients=POLYNOMIAL, eps=1e-7, stored=False, lead=1.0):
    """X of u; stored: X, A and B rounded to fp16, X at the start with a power of two near the root of its shorter side
    times ``lead`` (another one draws other roundings), for matrices of up to 128 rows B in two fp16 numbers a value.
    The kernels' own form (orthogonal_as_kept) rounds no more than that."""
    u = np.asarray(u, np.float64)
    if u.shape[0] > u.shape[1]:
        return orthogonal(u.T, iterations, coefficients, eps, stored, lead).T
    rnd = _half if stored else (lambda x: x)
    two = (lambda x: _half(x) + _half(x - _half(x))) if stored and u.shape[0] <= 128 else rnd
    start = 2.0 ** np.floor(0.5 * np.log2(u.shape[0])) * lead if stored else 1.0
    x = rnd(u * (start / (np.sqrt((u * u).sum()) + eps)))
    a, b, c = coefficients
    for _ in range(iterations):
        gram = rnd(x @ x.T / start ** 2)
        poly = two(b * gram + c * (gram @ gram))
        x = rnd((a * x + poly @ x) / start)
        start = 1.0
    return x


def muon(p, m, g, lr, momentum, nesterov, weight_decay, update_rms, **kw):
    """(p, m, X) after a step."""
    m = momentum * m + g
    x = orthogonal(g + momentum * m if nesterov else m, **kw)
    return p - lr * weight_decay * p - lr * update_rms * np.sqrt(max(p.shape)) * x, m, x


def kept(x, scale):
    """x as the kernels keep it: (fp16, and what that leaves as an e4m3 code of ``scale`` times it; scale 0: none)."""
    h = _half(x)
    if scale == 0:
        return h, np.zeros_like(h)
    y = np.clip((x - h) * scale, -448.0, 448.0)
    _, e = np.frexp(y)
    step = np.exp2(np.maximum(e - 1, -6) - 3)
    return h, np.rint(y / step) * step / scale


def orthogonal_as_kept(u, iterations=5, coefficients=POLYNOMIAL, eps=1e-7, rests=3, lead=1.0, alone=None):
    """X of u with the kernels' own roundings and exact sums. A = D + s I is kept as D, so that X = of_x X + B X with
    of_x = a + b s + c s^2 and B = (b + 2 c s) D + c D D; X, D and B are fp16, the first ``rests`` X's with codes of
    their rests, which enter X alone: with a (``alone``: a + b t + c t^2, t a
    quarter of s; 2 or 3 rows none, one row all of it), the last of them with of_x. s is the mean of A's diagonal (1 / r at first) for the
    matrices that one kernel takes (``alone``), else what the polynomial makes of 0.35 / r, 1 at most. ``lead``: another
    factor at the start draws other roundings."""
    u = np.asarray(u, np.float64)
    if u.shape[0] > u.shape[1]:
        return orthogonal_as_kept(u.T, iterations, coefficients, eps, rests, lead, alone).T
    r, k = u.shape
    if alone is None:
        alone = r <= 128 and k <= (12288 if r <= 64 else 4096)
    a, b, c = coefficients
    start = 2.0 ** np.floor(0.5 * np.log2(r)) * lead
    x, low = kept(u * (start / (np.sqrt((u * u).sum()) + eps)), 2.0 ** 20 / start if rests > 0 else 0)
    scale, square = 1.0 / start, 0.35 / r
    for n in range(iterations):
        s = (1.0 / r if n == 0 else (x * x).sum() / r) if alone else min(square, 1.0)
        square *= (a + b * square + c * square * square) ** 2
        of_x = a + b * s + c * s * s
        d = _half(x @ x.T * scale ** 2 - s * np.eye(r))
        poly = _half((b + 2 * c * s) * d + c * (d @ d))
        t = s * (1.0 if r == 1 else 0.0 if r < 4 else 0.25) if alone else 0.0
        of_rest = a + b * t + c * t * t if n + 1 < rests else of_x
        x, low = kept(scale * (of_x * x + of_rest * low + poly @ x), 2.0 ** 20 if n + 1 < rests else 0)
        scale = 1.0
    return x
