"""Cases of the operators that serve MXFP4 experts to a few tokens, and of the norm before them.

Four operators of one decode (or training) step of a block with routed experts
in MXFP4 (E2M1 codes, one E8M0 scale per 32 along K):

  norm       the residual's addition and the RMS norm of the sum; rows of the
             input's type, or MXFP8 (E4M3 codes, one E8M0 scale per 32) with
             the values that the codes stand for
  norm_grad  its gradients: of the sum's terms and of the gain
  matvec     few rows (bf16 or MXFP8, not rounded further) times MXFP4 weights;
             one matrix, or one per expert over expert-ordered rows
  experts    the routed experts of a few tokens: gate and up products, SiTU-GLU,
             down product, weighted sum over a token's experts, RMS norm

`run` computes them in elementary torch operations in 32 bits, or, where `own`
is set, with the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 32                    # elements that share an E8M0 scale
EPS = 1e-6
BETA1, BETA2 = 4.0, 25.0      # SiTU softcaps of the gate and up branches


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoded token before the layer: what a call costs when there is next to nothing to do
        dict(name="norm_token", op="norm", T=1, H=7168, x="bfloat16", res="bfloat16", q=True),
        # an odd batch with the residual stream kept in fp32, and rows of an odd number of elements
        dict(name="norm_odd", op="norm", T=999, H=2021, x="bfloat16", res="float32", q=False),
        # the norm before the layer at the prefill batch, rows in 8 bits
        dict(name="norm_prefill", op="norm", T=16384, H=7168, x="bfloat16", res="bfloat16", q=True),
        # a small fine-tuning batch with an fp32 residual stream
        dict(name="norm_grad_small", op="norm_grad", T=77, H=3584, dy="bfloat16", res="float32", dtotal=False),
        # the norm's backward pass at the prefill batch, the residual stream's own gradient added
        dict(name="norm_grad_train", op="norm_grad", T=16384, H=7168, dy="bfloat16", res="bfloat16", dtotal=True),
        # one decoded token through a dense full-width projection
        dict(name="matvec_token", op="matvec", R=1, E=0, N=6144, K=7168, skew=0.0, x="bfloat16", y="bfloat16"),
        # router logits of an odd handful of tokens, from 8-bit rows, in fp32
        dict(name="matvec_logits", op="matvec", R=13, E=0, N=896, K=7168, skew=0.0, x="mxfp8", y="float32"),
        # expert-ordered rows of a small layer: odd sizes, experts without rows
        dict(name="matvec_small", op="matvec", R=61, E=24, N=264, K=544, skew=2.0, x="bfloat16", y="bfloat16"),
        # a decode batch of 256 tokens, 16 experts each: about five rows an expert
        dict(name="matvec_decode", op="matvec", R=4096, E=896, N=1024, K=3584, skew=0.4, x="bfloat16", y="bfloat16"),
        # the routed experts of one decoded token
        dict(name="experts_token", op="experts", T=1, k=16, E=896, L=3584, M=1024, skew=0.4, x="bfloat16", norm=True),
        # a speculative handful of tokens, from 8-bit rows
        dict(name="experts_few", op="experts", T=7, k=16, E=896, L=3584, M=1024, skew=0.4, x="mxfp8", norm=True),
        # the routed experts of a decode batch of 256 tokens
        dict(name="experts_decode", op="experts", T=256, k=16, E=896, L=3584, M=1024, skew=0.4, x="bfloat16", norm=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "matvec", "matvec", "experts", "experts"])
    if op in ("norm", "norm_grad"):
        c = dict(op=op, T=_log_int(rng, 1, 16384))
        if op == "norm":
            c["q"] = rng.choice([False, True])
            c["H"] = BLOCK * _log_int(rng, 1, 224) if c["q"] else _log_int(rng, 1, 7168)
            c["x"] = rng.choice(["bfloat16", "float32"])
        else:
            c["H"] = rng.choice([_log_int(rng, 1, 7168), BLOCK * _log_int(rng, 1, 224)])
            c["dy"] = rng.choice(["bfloat16", "float32"])
            c["dtotal"] = rng.choice([False, True])
        c["res"] = rng.choice(["bfloat16", "float32"])
        c["T"] = min(c["T"], 60_000_000 // c["H"])
        return c
    x = rng.choice(["bfloat16", "mxfp8"])
    if op == "matvec":
        E = rng.choice([0, 0, 1, _log_int(rng, 2, 448)])
        K = BLOCK * _log_int(rng, 1, 320)
        N = 8 * min(_log_int(rng, 1, 800), 1_500_000_000 // (max(1, E) * K * 8))
        R = _log_int(rng, 1, 24 * max(1, E))
        # a strong skew leaves most experts empty; the plain form then pads every expert to the largest
        return dict(op=op, R=R, E=E, N=N, K=K, skew=rng.choice([0.3, 1.0]) if E > 1 else 0.0, x=x,
                    y=rng.choice(["bfloat16", "float32"]))
    E = _log_int(rng, 2, 384)
    k = rng.randint(1, min(16, E))
    return dict(op=op, T=_log_int(rng, 1, 4096 // k // 8), k=k, E=E, L=BLOCK * _log_int(rng, 1, 112),
                M=BLOCK * _log_int(rng, 1, 48), skew=rng.choice([0.0, 0.4, 1.0]), x=x, norm=rng.choice([True, False]))


def _size(t):
    return {"float32": 4, "bfloat16": 2, "mxfp8": 1 + 1 / BLOCK}[t]


def work(case):
    op = case["op"]
    if op == "norm":          # both terms, the sum; the norm (in 8 bits: codes, scales and their values), the gain
        e = case["T"] * case["H"]
        y = 2 + _size("mxfp8") if case["q"] else _size(case["x"])
        return {"bytes": int(e * (_size(case["x"]) + 2 * _size(case["res"]) + y)) + 4 * case["H"], "flops": 5 * e}
    if op == "norm_grad":     # the norm's gradient, the sum and its own gradient; the terms' gradient, the gain's
        e, r = case["T"] * case["H"], _size(case["res"])
        return {"bytes": e * (_size(case["dy"]) + r * (3 if case["dtotal"] else 2)) + 8 * case["H"], "flops": 9 * e}
    packed = lambda e: e // 2 + e // BLOCK  # noqa: E731
    if op == "matvec":        # rows, packed weights of the experts that have rows, products
        R, N, K = case["R"], case["N"], case["K"]
        used = int((_loads(case, 0) > 0).sum()) if case["E"] else 1
        return {"bytes": int(R * K * _size(case["x"])) + used * packed(N * K) + R * N * _size(case["y"]),
                "flops": 2 * R * N * K}
    T, k, L, M = case["T"], case["k"], case["L"], case["M"]
    used = len(np.unique(_routes(case, 0)[0]))
    return {"bytes": int(T * L * _size(case["x"])) + T * k * 8 + used * packed(3 * L * M) + T * L * 2 + 4 * L,
            "flops": 6 * T * k * L * M}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _loads(case, seed):
    """Rows of each expert: log-normal popularity; with a large skew many experts get none."""
    E, R = max(1, case["E"]), case["R"]
    r = np.random.RandomState(1000003 + 7919 * int(seed) % (1 << 31))
    p = np.exp(case["skew"] * r.standard_normal(E))
    return r.multinomial(R, p / p.sum())


def _routes(case, seed):
    """idx [T, k], a token's experts in order of score; w [T, k], the scores renormalised."""
    T, k, E = case["T"], case["k"], case["E"]
    r = np.random.RandomState(2000003 + 104729 * int(seed) % (1 << 31))
    logits = r.standard_normal((T, E)) + case["skew"] * r.standard_normal(E)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    s = 1 / (1 + np.exp(-np.take_along_axis(logits, idx, 1)))
    return idx, (s / s.sum(1, keepdims=True)).astype(np.float32)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _quantize_chunks(make, rows, K, chunk=1 << 17):
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, K // BLOCK), dtype=torch.uint8, device=DEV)
    for a in range(0, rows, chunk):
        b = min(rows, a + chunk)
        codes[a:b], scales[a:b] = _make_mxfp4(make(b - a))
    return codes, scales


def _make_mxfp4(x):
    """Packed E2M1 codes and scale bytes of fp32 rows."""
    R, K = x.shape
    b = x.view(R, K // BLOCK, BLOCK)
    amax = b.abs().amax(2)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 3).clamp(min=-127), -127)
    a = b.abs() * ((127 - e) << 23).view(torch.float32)[:, :, None]
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(b).to(torch.uint8)).view(R, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _rows(g, R, K):
    """Activations: unit normal, each row with a scale of its own, a few large channels."""
    x = _normal(g, R, K) * torch.exp(0.5 * _normal(g, R, 1))
    x[:, :: 97] *= 6.0
    return x


def _weights(st, name, g, lead, N, K):
    codes, scales = _quantize_chunks(lambda r: _normal(g, r, K) / math.sqrt(K), math.prod(lead) * N, K)
    st[name + "_codes"], st[name + "_scales"] = codes.view(*lead, N, K // 2), scales.view(*lead, N, K // BLOCK)


def _input_rows(st, g, kind, R, K):
    x = _rows(g, R, K)
    if kind == "mxfp8":
        values, e = _to_mxfp8(x)
        scale = ((127 - e) << 23).view(torch.float32)
        st["x_codes"] = (values.view(R, K // BLOCK, BLOCK) * scale[:, :, None]).view(R, K).to(torch.float8_e4m3fn)
        st["x_scales"] = (e + 127).to(torch.uint8)
    else:
        st["x"] = x.to(torch.bfloat16)


def prepare(case, seed):
    op = case["op"]
    st = dict(op=op, case=dict(case))
    g = _gen(seed)
    if op in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        st["gamma"] = 1.0 + 0.1 * _normal(g, H)
        stream = (3.0 * _rows(g, T, H)).to(getattr(torch, case["res"]))
        if op == "norm":
            st["x"] = _rows(g, T, H).to(getattr(torch, case["x"]))
            st["residual"] = stream
        else:
            st["total"] = stream
            st["dy"] = (1e-3 * _normal(g, T, H)).to(getattr(torch, case["dy"]))
            st["dtotal"] = (1e-3 * _normal(g, T, H)).to(stream.dtype) if case["dtotal"] else None
    elif op == "matvec":
        R, N, K, E = case["R"], case["N"], case["K"], case["E"]
        _weights(st, "w", g, (E,) if E else (), N, K)
        _input_rows(st, g, case["x"], R, K)
        st["offsets"] = None
        if E:
            loads = _loads(case, seed)
            st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(loads)]).astype(np.int32)).to(DEV)
            st["cap"] = int(loads.max())          # most rows of one expert: the plain form's padding
    else:
        T, E, L, M = case["T"], case["E"], case["L"], case["M"]
        _weights(st, "gate", g, (E,), M, L)
        _weights(st, "up", g, (E,), M, L)
        _weights(st, "down", g, (E,), L, M)
        _input_rows(st, g, case["x"], T, L)
        idx, w = _routes(case, seed)
        st["cap"] = int(np.bincount(idx.ravel()).max())
        st["idx"], st["w"] = torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV)
        st["gamma"] = 1.0 + 0.1 * _normal(g, L) if case["norm"] else None
    if own:
        import quantile_balanced_routing_gb300 as qb
        st["qb"] = qb
        for name in ("w", "gate", "up", "down"):
            if name + "_codes" in st:
                st[name + "4"] = qb.Mxfp4(st[name + "_codes"], st[name + "_scales"])
        if "x_codes" in st:
            st["x"] = qb.Mxfp8(st["x_codes"], st["x_scales"])
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _to_mxfp8(x):
    """Values [R, K] and block exponents [R, K / 32] of the MXFP8 form of fp32 rows."""
    R, K = x.shape
    b = x.view(R, K // BLOCK, BLOCK)
    amax = b.abs().amax(2)
    # the scale's exponent: that of the largest magnitude, less 7, so that no value passes E4M3's largest
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 8).clamp(min=-127), -127)
    a = b.abs() * ((127 - e) << 23).view(torch.float32)[:, :, None]
    # E4M3: three mantissa bits, exponents from -6 on; ties to even
    step = torch.exp2((torch.frexp(a)[1] - 1).clamp(min=-6).float() - 3)
    a = torch.round(a / step) * step
    scale = torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)[:, :, None]
    return (torch.where(torch.signbit(b), -a, a) * scale).view(R, K), e


def _scale(s):
    """fp32 value of E8M0 bytes."""
    e = s.to(torch.int32)
    return torch.where(e > 0, e << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _from_mxfp4(codes, scales):
    """fp32 values of packed codes [..., K / 2] and scale bytes [..., K / 32]."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=codes.device)
    pairs = torch.cartesian_prod(grid, grid).flip(1)      # a byte's two values, the low nibble's first
    v = pairs[codes.to(torch.int32)].flatten(-2)
    return (v.unflatten(-1, (-1, BLOCK)) * _scale(scales)[..., None]).flatten(-2)


def _x_rows(st):
    if "x_codes" not in st:
        return st["x"].float()
    return (st["x_codes"].float().unflatten(-1, (-1, BLOCK)) * _scale(st["x_scales"])[..., None]).flatten(-2)


def _norm(st):
    total = (st["x"].float() + st["residual"].float()).to(st["residual"].dtype)
    v = total.float()
    n = v * (1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)) * st["gamma"]
    if st["case"]["q"]:
        return dict(total=total, y=_to_mxfp8(n)[0].to(torch.bfloat16))
    return dict(total=total, y=n.to(st["x"].dtype))


def _norm_grad(st):
    v, dy = st["total"].float(), st["dy"].float()
    r = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    g = dy * st["gamma"]
    dx = (g - v * ((g * v).mean(1, keepdim=True) * r * r)) * r
    if st["dtotal"] is not None:
        dx = dx + st["dtotal"].float()
    return dict(dx=dx.to(st["total"].dtype), dgamma=(dy * v * r).sum(0))


def _busy(offsets, R):
    """The experts that may have rows, where there are fewer rows than experts; else all of them."""
    if R >= offsets.shape[0] - 1:
        return slice(None)
    return torch.argsort(offsets[1:] - offsets[:-1], descending=True)[:R]


def _padded(rows, offsets, some, cap):
    """Expert-ordered rows [R, C] as [experts, cap, C], padded with zeros; and each place's row, or R."""
    R = rows.shape[0]
    i = offsets[:-1][some][:, None] + torch.arange(cap, device=DEV)
    i = torch.where(i < offsets[1:][some][:, None], i, R).long()
    rows = torch.cat((rows, torch.zeros((1, rows.shape[1]), device=DEV)))
    return rows[i], i


def _ordered(padded, i, R):
    """The rows [R, C] of a padded [experts, cap, C]."""
    out = torch.empty((R + 1, padded.shape[2]), device=DEV)
    out[i.flatten()] = padded.flatten(0, 1)
    return out[:R]


def _matvec(st):
    x = _x_rows(st)
    to = getattr(torch, st["case"]["y"])
    if st["offsets"] is None:
        return dict(y=(x @ _from_mxfp4(st["w_codes"], st["w_scales"]).t()).to(to))
    some = _busy(st["offsets"], x.shape[0])
    w = _from_mxfp4(st["w_codes"][some], st["w_scales"][some])
    xp, i = _padded(x, st["offsets"], some, st["cap"])
    return dict(y=_ordered(torch.bmm(xp, w.transpose(1, 2)), i, x.shape[0]).to(to))


def _experts(st):
    x, idx, w = _x_rows(st), st["idx"], st["w"]
    (T, k), E = idx.shape, st["case"]["E"]
    flat = idx.flatten().long()
    order = torch.argsort(flat, stable=True)              # routes in expert order
    load = torch.zeros(E, device=DEV, dtype=torch.int64).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((load.new_zeros(1), load.cumsum(0)))
    some = _busy(offsets, T * k)
    weights = lambda name: _from_mxfp4(st[name + "_codes"][some], st[name + "_scales"][some]).transpose(1, 2)  # noqa: E731
    xp, i = _padded(x[order // k], offsets, some, st["cap"])
    gate = torch.bmm(xp, weights("gate"))
    up = torch.bmm(xp, weights("up"))
    a = BETA1 * torch.tanh(gate / BETA1)
    act = a / (1.0 + torch.exp(-a)) * (BETA2 * torch.tanh(up / BETA2))
    e = torch.bmm(act, weights("down"))
    rows = torch.empty((T * k, e.shape[2]), device=DEV)
    rows[order] = _ordered(e, i, T * k)
    z = (rows.view(T, k, -1) * w[:, :, None]).sum(1)
    if st["gamma"] is not None:
        z = z * (1.0 / torch.sqrt((z * z).mean(1, keepdim=True) + EPS)) * st["gamma"]
    return dict(y=z.to(torch.bfloat16))


def run(st):
    op = st["op"]
    if not own:
        return {"norm": _norm, "norm_grad": _norm_grad, "matvec": _matvec, "experts": _experts}[op](st)
    qb = st["qb"]
    if op == "norm":
        r = qb.add_rmsnorm(st["x"], st["gamma"], residual=st["residual"], eps=EPS, mxfp8=st["case"]["q"])
        return dict(total=r.total, y=r.y)
    if op == "norm_grad":
        dx, dgamma = qb.add_rmsnorm_backward(st["dy"], st["total"], st["gamma"], dtotal=st["dtotal"], eps=EPS)
        return dict(dx=dx, dgamma=dgamma)
    if op == "matvec":
        return dict(y=qb.mxfp4_matvec(st["x"], st["w4"], offsets=st["offsets"],
                                      out_dtype=getattr(torch, st["case"]["y"])))
    return dict(y=qb.mxfp4_experts(st["x"], st["idx"], st["w"], st["gate4"], st["up4"], st["down4"],
                                   gamma=st["gamma"], eps=EPS, beta1=BETA1, beta2=BETA2))


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_decode(codes, scales):
    grid = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=codes.device)
    v = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=codes.device)
    v[..., 0::2] = grid[(codes % 16).int()]
    v[..., 1::2] = grid[(codes // 16).int()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, dim=-1)


def _exact_rows(st):
    if "x_codes" not in st:
        return st["x"].double()
    return st["x_codes"].double() * torch.exp2(st["x_scales"].double() - 127).repeat_interleave(BLOCK, dim=-1)


def _exact_mxfp8(n):
    """MXFP8 values of 64-bit rows: the nearest of E4M3's magnitudes below 256, ties to the even code."""
    b = n.reshape(n.shape[0], -1, BLOCK)
    amax = b.abs().amax(2, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    e = torch.where(torch.exp2(e) > amax, e - 1, e)          # a logarithm rounded up to the next integer
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    scale = torch.exp2((e - 7).clamp(min=-127))
    a = b.abs() / scale
    # E4M3's magnitudes up to 256 in order: codes 0 to 120, the even ones at even places
    grid = torch.tensor([m / 512 for m in range(8)] + [(8 + m) * 2.0 ** (x - 10) for x in range(1, 15) for m in range(8)]
                        + [256.0], dtype=torch.float64, device=n.device)
    lo = (torch.searchsorted(grid, a, right=True) - 1).clamp(max=len(grid) - 2)
    below, above = a - grid[lo], grid[lo + 1] - a
    at = torch.where((above < below) | ((above == below) & (lo % 2 == 1)), lo + 1, lo)
    return (torch.sign(b) * grid[at] * scale).reshape(n.shape)


def _exact_norm(st):
    # the sum is rounded to the residual's type before its norm is taken: both terms add exactly in 64 bits
    total = (st["x"].double() + st["residual"].double()).to(st["residual"].dtype)
    v = total.double()
    n = v / torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + EPS) * st["gamma"].double()
    return dict(total=total.double(), y=_exact_mxfp8(n) if st["case"]["q"] else n)


def _exact_norm_grad(st):
    v, dy, gamma = st["total"].double(), st["dy"].double(), st["gamma"].double()
    ms = v.square().sum(1, keepdim=True) / v.shape[1] + EPS
    g = dy * gamma
    dx = g / ms.sqrt() - v * (g * v).sum(1, keepdim=True) / (v.shape[1] * ms ** 1.5)
    if st["dtotal"] is not None:
        dx += st["dtotal"].double()
    return dict(dx=dx, dgamma=(dy * (v / ms.sqrt())).sum(0))


def _exact_matvec(st):
    x = _exact_rows(st)
    if st["offsets"] is None:
        return dict(y=x @ _exact_decode(st["w_codes"], st["w_scales"]).t())
    off = st["offsets"].tolist()
    y = torch.zeros((x.shape[0], st["w_codes"].shape[1]), dtype=torch.float64, device=DEV)
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if b > a:
            y[a:b] = x[a:b] @ _exact_decode(st["w_codes"][e], st["w_scales"][e]).t()
    return dict(y=y)


def _exact_experts(st):
    x, idx, w = _exact_rows(st), st["idx"], st["w"].double()
    z = torch.zeros((x.shape[0], st["case"]["L"]), dtype=torch.float64, device=DEV)
    for e in torch.unique(idx).tolist():
        t, i = torch.nonzero(idx == e, as_tuple=True)
        g = x[t] @ _exact_decode(st["gate_codes"][e], st["gate_scales"][e]).t()
        u = x[t] @ _exact_decode(st["up_codes"][e], st["up_scales"][e]).t()
        a = BETA1 * torch.tanh(g / BETA1)
        act = a * torch.sigmoid(a) * (BETA2 * torch.tanh(u / BETA2))
        z.index_add_(0, t, w[t, i][:, None] * (act @ _exact_decode(st["down_codes"][e], st["down_scales"][e]).t()))
    if st["gamma"] is not None:
        z = z / torch.sqrt(z.square().sum(1, keepdim=True) / z.shape[1] + EPS) * st["gamma"].double()
    return dict(y=z)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "matvec": _exact_matvec,
            "experts": _exact_experts}[case["op"]](st)
