"""MXFP4 and router-training formulas in 64 bits (numpy), for the tests."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(packed codes, scale bytes, values) of rows [R, K]: nearest, ties to the even code."""
    R, K = x.shape
    b = np.asarray(x, np.float64).reshape(R, K // 32, 32)
    amax = np.abs(b).max(2)
    bad = ~np.isfinite(amax)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.frexp(np.where(bad, 1.0, amax))[1] - 1 - 2
    e = np.where(amax == 0, -127, np.maximum(e, -127))
    scale = np.ldexp(1.0, np.where(bad, 0, e))
    with np.errstate(invalid="ignore"):
        a = np.where(bad[..., None], 0.0, np.abs(b)) / scale[..., None]
    d = np.abs(a[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)
    odd = np.arange(8) % 2
    code = np.argmin(np.where(near, odd, 2), axis=-1)        # the even one of two nearest codes
    neg = np.signbit(b) & ~bad[..., None]
    v = np.where(neg, -GRID[code], GRID[code]) * scale[..., None]
    v = np.where(bad[..., None], np.nan, v).reshape(R, K)
    code = (code + 8 * neg).reshape(R, K).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8), v


def decode(codes, scales):
    """fp64 values [..., K] of packed codes and scale bytes."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def groups(offsets, R):
    return [(0, R)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def matmul(x, w, offsets):
    """(y, sum of magnitudes) of rows x [R, K] and weights w [E, N, K]."""
    y = np.zeros((x.shape[0], w.shape[1]))
    m = np.zeros_like(y)
    for e, (a, b) in enumerate(groups(offsets, x.shape[0])):
        y[a:b] = x[a:b] @ w[e].T
        m[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, m


def matmul_backward(dy, x, w, offsets):
    """((dx, magnitudes), (dw, magnitudes))."""
    dx, dw = np.zeros(x.shape), np.zeros(w.shape)
    mx, mw = np.zeros_like(dx), np.zeros_like(dw)
    for e, (a, b) in enumerate(groups(offsets, x.shape[0])):
        dx[a:b], mx[a:b] = dy[a:b] @ w[e], np.abs(dy[a:b]) @ np.abs(w[e])
        dw[e], mw[e] = dy[a:b].T @ x[a:b], np.abs(dy[a:b]).T @ np.abs(x[a:b])
    return (dx, mx), (dw, mw)


def scores(logits):
    return 1.0 / (1.0 + np.exp(-np.clip(np.asarray(logits, np.float64), -80, 80)))


def balance(logits, idx, offsets=None, mask=None):
    """(loss [S], counts, probs, tokens) of each sequence's valid tokens."""
    T, n = logits.shape
    k = idx.shape[1]
    s = scores(logits)
    p = s / s.sum(1, keepdims=True)
    mask = np.ones(T, bool) if mask is None else mask.astype(bool)
    out = []
    for a, b in groups(offsets, T):
        t = [i for i in range(a, b) if mask[i]]
        c = np.bincount([j for i in t for j in idx[i] if 0 <= j < n], minlength=n)
        m = p[t].mean(0) if t else np.zeros(n)
        out.append((n / (k * max(1, len(t))) * (c * m).sum(), c, m, len(t)))
    return tuple(np.array(v) for v in zip(*out))


def objective(logits, idx, dw, dloss, counts, tokens, offsets=None, mask=None):
    """What the router's gradient differentiates: the routes are constants."""
    T, n = logits.shape
    k = idx.shape[1]
    s = scores(logits)
    p = s / s.sum(1, keepdims=True)
    mask = np.ones(T, bool) if mask is None else mask.astype(bool)
    total = 0.0
    for q, (a, b) in enumerate(groups(offsets, T)):
        for t in range(a, b):
            if not mask[t]:
                continue
            if dw is not None:
                sk = np.array([s[t, j] if 0 <= j < n else 0.0 for j in idx[t]])
                total += (dw[t] * sk).sum() / sk.sum() if sk.sum() > 0 else 0.0
            if dloss is not None:
                total += dloss[q] * n / (k * max(1, tokens[q]) ** 2) * (counts[q] * p[t]).sum()
    return total


def router_grad(logits, idx, dw, dloss, counts, tokens, offsets=None, mask=None):
    T, n = logits.shape
    k = idx.shape[1]
    x = np.asarray(logits, np.float64)
    s = scores(x)
    ds = np.zeros((T, n))
    mask = np.ones(T, bool) if mask is None else mask.astype(bool)
    for q, (a, b) in enumerate(groups(offsets, T)):
        for t in range(a, b):
            if not mask[t]:
                continue
            if dw is not None:
                ok = (idx[t] >= 0) & (idx[t] < n)
                sk, d = s[t, idx[t][ok]], dw[t][ok]
                if ok.any():
                    ds[t, idx[t][ok]] += (d - (d * sk).sum() / sk.sum()) / sk.sum()
            if dloss is not None:
                f = dloss[q] * n / (k * max(1, tokens[q]) ** 2) * counts[q]
                ds[t] += (f - (f * s[t]).sum() / s[t].sum()) / s[t].sum()
    return ds * s * scores(-x) * (np.abs(x) <= 80)
