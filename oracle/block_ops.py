"""Float64 definitions of the operators around the block's projections
(adaln_modulation, adaln_gate_residual, gradient norm, AdamW), each value
together with a bound of the error that fp32 arithmetic may make in it.

The bounds are running error bounds: u = 2^-24 is the unit roundoff of fp32;
a sum of n terms in any order is off by at most n * u times the sum of the
magnitudes (the kernels' trees are far shallower, so ``depth`` bounds the
longest chain: 16 values of a thread, 5 shuffle steps, 16 warps, and the few
operations that form a term); every other operation adds its operands'
errors and u times its result."""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24
ROW_DEPTH = 16 + 5 + 16 + 3


def stats(x, kind, eps):
    """(mean, rstd) of rows and the bounds of their errors. The variance sums
    squares about the mean, each with relative error 3u at most."""
    C = x.shape[-1]
    mean = x.sum(-1) / C if kind == "layer" else np.zeros(x.shape[:-1])
    mean_err = (ROW_DEPTH * U * np.abs(x).sum(-1) / C) if kind == "layer" else np.zeros(x.shape[:-1])
    var = ((x - mean[..., None]) ** 2).sum(-1) / C
    rstd = 1.0 / np.sqrt(var + eps)
    # var: (depth + 4) u var and the mean's error squared; rstd: half of that, and three roundings
    var_err = (ROW_DEPTH + 4) * U * var + mean_err ** 2
    rstd_err = rstd * (0.5 * var_err / (var + eps) + 4 * U)
    return mean, rstd, mean_err, rstd_err


def hat(x, mean, rstd, mean_err=0.0, rstd_err=0.0):
    mean, rstd = mean[..., None], rstd[..., None]
    mean_err, rstd_err = (np.asarray(e)[..., None] if np.ndim(e) else e for e in (mean_err, rstd_err))
    z = x - mean
    h = z * rstd
    err = rstd * (mean_err + U * np.abs(z)) + np.abs(z) * rstd_err + 2 * U * np.abs(h)
    return h, err


def modulation(x, scale, shift, w, kind, eps):
    """y and its bound, (mean, rstd) and theirs; scale, shift [B, C], w [C]."""
    mean, rstd, me, re = stats(x, kind, eps)
    h, he = hat(x, mean, rstd, me, re)
    k = w * (1.0 + scale)[:, None, :]
    y = h * k + shift[:, None, :]
    err = np.abs(k) * (he + 4 * U * np.abs(h)) + 2 * U * (np.abs(h * k) + np.abs(y))
    return y, err, (mean, rstd), (me, re)


def residual(x, h, gate, w_post, post, alpha, eps):
    """r before its rounding and its bound; (mean, rstd) of h and theirs, or None."""
    u, ue, st = h, np.zeros_like(h), None
    if post != "none":
        mean, rstd, me, re = stats(h, post, eps)
        z, ze = hat(h, mean, rstd, me, re)
        u, ue, st = z * w_post, np.abs(w_post) * (ze + 2 * U * np.abs(z)), ((mean, rstd), (me, re))
    k = alpha * gate[:, None, :]
    r = x + k * u
    err = np.abs(k) * (ue + 4 * U * np.abs(u)) + 2 * U * np.abs(r)
    return r, err, st


def _norm_backward(e, ee, z, ze, rstd, kind):
    """rstd * (e - mean(e) - z * mean(e z)) and its bound."""
    C = e.shape[-1]
    c2 = (e * z).sum(-1, keepdims=True) / C
    c2e = ((np.abs(e) * ze + ee * np.abs(z)).sum(-1, keepdims=True) + ROW_DEPTH * U * np.abs(e * z).sum(-1, keepdims=True)) / C
    c1 = c1e = 0.0
    if kind == "layer":
        c1 = e.sum(-1, keepdims=True) / C
        c1e = (ee.sum(-1, keepdims=True) + ROW_DEPTH * U * np.abs(e).sum(-1, keepdims=True)) / C
    out = rstd[..., None] * (e - c1 - z * c2)
    size = np.abs(e) + np.abs(c1) + np.abs(z * c2)
    err = rstd[..., None] * (ee + c1e + np.abs(z) * c2e + ze * np.abs(c2) + 5 * U * size)
    return out, err


def _column_sum(terms, errs):
    """Over the tokens of a sample [B, T, C] -> [B, C]."""
    T = terms.shape[1]
    return terms.sum(1), errs.sum(1) + (T + 8) * U * np.abs(terms).sum(1)


def _sample_sum(k, a, ae):
    t = k * a
    return t.sum(0), (np.abs(k) * ae).sum(0) + (t.shape[0] + 4) * U * np.abs(t).sum(0)


def modulation_backward(x, scale, w, mean, rstd, dy, dr, kind):
    """{name: (value, bound)} of dx, dscale, dshift, dw from given statistics."""
    z, ze = hat(x, mean, rstd)
    k = w * (1.0 + scale)[:, None, :]
    e, ee = dy * k, 4 * U * np.abs(dy * k)
    t, te = _norm_backward(e, ee, z, ze, rstd, kind)
    dx = dr + t
    a, ae = _column_sum(dy * z, np.abs(dy) * ze + U * np.abs(dy * z))
    s, se = _column_sum(dy, np.zeros_like(dy))
    return {"dx": (dx, te + 2 * U * (np.abs(dx) + np.abs(t))), "dscale": (w * a, np.abs(w) * (ae + 2 * U * np.abs(a))),
            "dshift": (s, se), "dw": _sample_sum(1.0 + scale, a, ae + 2 * U * np.abs(a))}


def gate_residual_backward(r, h, gate, scale, w, w_post, mean, rstd, post_stats, dy, dr, kind, post, alpha):
    """The same with dh, dgate, dw_post; dy None: y was not used."""
    if dy is None:
        out = {"dx": (dr, np.zeros_like(dr))}
    else:
        out = modulation_backward(r, scale, w, mean, rstd, dy, dr, kind)
    d, de = out["dx"]
    k = alpha * gate[:, None, :]
    f, fe = d * k, np.abs(k) * (de + 4 * U * np.abs(d))
    if post == "none":
        z, ze, share = h, np.zeros_like(h), np.ones(h.shape[-1])
        dh, dhe = f, fe
    else:
        z, ze = hat(h, *post_stats)
        share = w_post
        dh, dhe = _norm_backward(f * w_post, np.abs(w_post) * (fe + 2 * U * np.abs(f)), z, ze, post_stats[1], post)
    g, ge = _column_sum(d * z, np.abs(d) * ze + de * np.abs(z) + U * np.abs(d * z))
    out["dh"] = (dh, dhe)
    out["dgate"] = (alpha * share * g, np.abs(alpha * share) * (ge + 4 * U * np.abs(g)))
    out["dw_post"] = _sample_sum(alpha * gate, g, ge + 4 * U * np.abs(g))
    return out


# ------------------------------------------------------------------ optimiser
def adamw(p, g, m, v, *, lr, beta1, beta2, eps, weight_decay, step, scale=1.0):
    """(p, m, v) after one step and the bounds of their errors."""
    g = g * scale
    m1, v1 = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    me = 4 * U * (np.abs(beta1 * m) + np.abs((1 - beta1) * g))
    ve = 6 * U * v1
    c1, c2 = 1 - beta1 ** step, 1 - beta2 ** step
    den = np.sqrt(v1 / c2) + eps
    den_err = 8 * U * den  # half of v's, the square root, 1 / sqrt(c2), one fma
    up = lr / c1 * m1 / den
    up_err = np.abs(lr / c1) * (me / den + np.abs(m1) * den_err / den ** 2) + 8 * U * np.abs(up)
    p1 = p - lr * weight_decay * p - up
    pe = up_err + 6 * U * np.abs(lr * weight_decay * p) + 2 * U * np.abs(p1)
    return (p1, m1, v1), (pe, me, ve)


def hash32(x):
    """The 32-bit integer hash "lowbias32" of Wellons' prospector search."""
    x = np.asarray(x, dtype=np.uint32).copy()
    x ^= x >> np.uint32(16)
    x *= np.uint32(0x7FEB352D)
    x ^= x >> np.uint32(15)
    x *= np.uint32(0x846CA68B)
    x ^= x >> np.uint32(16)
    return x


def random_bits(seed, step, key, n):
    """The 32 random bits of each of a tensor's n elements."""
    with np.errstate(over="ignore"):
        base = hash32(hash32(hash32(np.uint32(seed)) ^ np.uint32(step)) ^ np.uint32(key))
        return hash32(np.arange(n, dtype=np.uint64).astype(np.uint32) * np.uint32(0x9E3779B9) + base)


E4M3 = np.array([(-1.0 if c & 128 else 1.0) *
                 ((c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10))
                 for c in range(256)])
E4M3[[127, 255]] = np.nan


def decode(codes, scales):
    """The values that 8-bit states stand for (uint8 codes and scales)."""
    n = codes.size
    s = np.where(scales == 0, 0.0, np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127)))
    return E4M3[codes] * np.repeat(s, 32)[:n]


def encode(x, bits16, positive):
    """fp32 values as codes and scales, with 16 random bits each: from the
    format's definition, in exact (float64) arithmetic."""
    x = np.asarray(x, dtype=np.float64)
    n = x.size
    pad = -n % 32
    b, r = np.pad(x, (0, pad)).reshape(-1, 32), np.pad(bits16.astype(np.float64), (0, pad)).reshape(-1, 32)
    codes, scales = np.zeros(b.shape, np.uint8), np.zeros(b.shape[0], np.uint8)
    magnitudes = E4M3[:127]
    for i, row in enumerate(b):
        if not np.isfinite(row).all():
            scales[i] = 255
            continue
        top = np.abs(row).max()
        e = -1000 if top == 0 else int(np.floor(np.log2(top)))
        if top > 1.75 * 2.0 ** e:
            e += 1
        e = max(e, 32 - 127)
        y = np.abs(row) * 2.0 ** (8 - e)
        low = np.searchsorted(magnitudes, y, side="right") - 1
        gap = np.where(low < 126, magnitudes[np.minimum(low + 1, 126)] - magnitudes[low], 1.0)
        # the 20 bits below a code's last one, and the random ones added to them
        rest = np.floor((y - magnitudes[low]) / gap * 2.0 ** 20)
        c = low + (rest + r[i] * 16 + 8 >= 2.0 ** 20)
        if positive:
            c = np.where(row > 0, np.maximum(c, 1), c)
        else:
            c = c | np.where(np.signbit(row), 128, 0)
        codes[i], scales[i] = c, e + 127 - 8
    return codes.reshape(-1)[:n], scales
