"""The norm, few-row products and experts of a few tokens in 64 bits (numpy), with error bounds.

Magnitudes that come with a result bound what fp32 sums of its terms can be off by.
"""
import numpy as np

import mx_reference as M

# E4M3's finite magnitudes by code
E4M3 = np.array([m / 512 for m in range(8)] + [(8 + m) * 2.0 ** (x - 10) for x in range(1, 16) for m in range(8)][:-1])


def decode8(codes, scales):
    """fp64 values [..., K] of E4M3 bytes and scale bytes."""
    mag = codes & 127
    v = np.where(mag == 127, np.nan, E4M3[np.minimum(mag, 126)]) * np.where(codes & 128, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def quantize8(n):
    """(codes, scale bytes) of rows [R, K]: nearest, ties to the even code, no magnitude above 256."""
    R, K = n.shape
    b = np.asarray(n, np.float64).reshape(R, K // 32, 32)
    amax = np.abs(b).max(2)
    bad = ~np.isfinite(amax)
    e = np.frexp(np.where(bad, 1.0, amax))[1] - 1 - 7
    e = np.where(amax == 0, -127, np.maximum(e, -127))
    with np.errstate(invalid="ignore"):
        a = np.where(bad[..., None], 0.0, np.abs(b)) / np.ldexp(1.0, np.where(bad, 0, e))[..., None]
    hi = np.searchsorted(E4M3, a).clip(1, len(E4M3) - 1)
    lo = hi - 1
    up = (E4M3[hi] - a < a - E4M3[lo]) | ((E4M3[hi] - a == a - E4M3[lo]) & (hi % 2 == 0))
    code = np.where(up, hi, lo) + 128 * (np.signbit(b) & ~bad[..., None])
    return code.astype(np.uint8).reshape(R, K), np.where(bad, 255, e + 127).astype(np.uint8)


def rms(total, eps):
    return 1.0 / np.sqrt((total ** 2).mean(-1, keepdims=True) + eps)


def norm(total, gamma, eps):
    return total * rms(total, eps) * gamma


def norm_backward(dn, total, gamma, dtotal, eps):
    """((dx, magnitudes), (dgamma, magnitudes))."""
    r, g = rms(total, eps), dn * gamma
    dx = r * (g - total * r * r * (g * total).mean(-1, keepdims=True)) + (0.0 if dtotal is None else dtotal)
    mx = r * (np.abs(g) + np.abs(total) * r * r * np.abs(g * total).mean(-1, keepdims=True))
    mx = mx + (0.0 if dtotal is None else np.abs(dtotal))
    return (dx, mx), ((dn * total * r).sum(0), np.abs(dn * total * r).sum(0))


def situ(g, u, b1, b2):
    a = b1 * np.tanh(g / b1)
    return a / (1 + np.exp(-a)) * b2 * np.tanh(u / b2)


def block_top(x):
    """Each element's block's largest magnitude."""
    top = np.abs(x).reshape(*x.shape[:-1], -1, 32).max(-1)
    return np.repeat(top, 32, axis=-1)


def product(x, w):
    """(y, bound) of x [R, K] w [N, K]^T: K fp32 additions, and what the blocks' fp16 form drops."""
    return x @ w.T, (x.shape[1] * 2.0 ** -24 * np.abs(x) + 2.0 ** -40 * block_top(x)) @ np.abs(w).T


def experts(x, idx, w, gate, up, out, gamma, eps, b1=4.0, b2=25.0):
    """(y [T, L], bound before the output's rounding) of tokens x [T, L]."""
    T, k = idx.shape
    L = x.shape[1]
    z, dz = np.zeros((T, L)), np.zeros((T, L))
    for t in range(T):
        for i in range(k):
            e = idx[t, i]
            if not 0 <= e < gate.shape[0]:
                continue
            g, dg = product(x[t:t + 1], gate[e])
            u, du = product(x[t:t + 1], up[e])
            a, b = b1 * np.tanh(g / b1), b2 * np.tanh(u / b2)
            act = situ(g, u, b1, b2)
            # |d(a sigmoid(a))/da| <= 1.1, |da/dg|, |db/du| <= 1; the functions themselves to 2^-20 of
            # the value; then one rounding to fp16 (2^-11 covers its half step of 2^-12 twice over)
            da = 1.1 * dg * np.abs(b) + np.abs(a / (1 + np.exp(-a))) * du + (2.0 ** -20 + 2.0 ** -12) * np.abs(act)
            s, ds = product(act, out[e])
            ds = ds + (da + 2.0 ** -40 * block_top(act)) @ np.abs(out[e]).T
            z[t] += w[t, i] * s[0]
            dz[t] += np.abs(w[t, i]) * (ds[0] + (k + 2) * 2.0 ** -24 * np.abs(s[0]))
    if gamma is None:
        return z, dz
    r = rms(z, eps)
    y = z * r * gamma
    dy = r * (dz + np.abs(z) * r * r * (np.abs(z) * dz).mean(-1, keepdims=True)) * np.abs(gamma)
    return y, dy + 2.0 ** -18 * np.abs(y)


def weights(r, *shape):
    """(codes, scales, values) of MXFP4 weights [..., K]."""
    K = shape[-1]
    w = r.standard_normal((int(np.prod(shape[:-1])), K)) / np.sqrt(K)
    c, s, v = M.quantize(w)
    return c.reshape(*shape[:-1], K // 2), s.reshape(*shape[:-1], K // 32), v.reshape(shape)
