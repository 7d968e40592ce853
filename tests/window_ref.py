"""Inputs and plain 64-bit references of the decode-window operators' tests
(4-bit grouped weights, the MoE layer, token log probabilities): numpy only,
nothing of the library."""
import numpy as np


def f64(bits, kind):
    """uint16 bit patterns (f16 / bf16) or float32 values -> float64."""
    if kind == "f32":
        return np.asarray(bits, np.float64)
    if kind == "f16":
        return np.asarray(bits, np.uint16).view(np.float16).astype(np.float64)
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


# relative rounding error of one value stored in a type, and its spacing at zero
ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def gen_w4(shape, group, kind, zeros, seed, sd=0.02):
    """A 4-bit grouped weight [..][k]: packed codes, scale bits of `kind`
    (about the standard deviation sd), zero points or None."""
    import workloads as WL

    rng = np.random.default_rng(seed)
    *lead, k = shape
    q = rng.integers(0, 16, size=(*lead, k), dtype=np.uint8)
    codes = (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)
    scales = WL.to_bits(rng.uniform(0.5, 1.5, size=(*lead, k // group)) * sd / 4.6, kind)
    z = rng.integers(0, 16, size=(*lead, k // group), dtype=np.uint8) if zeros else None
    return codes, scales, z


def w4_parts(w, kind):
    """(codes, scales, zero points) of a 4-bit grouped weight, each [..][k] in 64 bits."""
    codes, scales, zeros = w
    k = 2 * codes.shape[-1]
    q = np.empty((*codes.shape[:-1], k))
    q[..., 0::2] = codes & 15
    q[..., 1::2] = codes >> 4
    g = k // scales.shape[-1]
    s = np.repeat(f64(scales, kind), g, axis=-1)
    z = np.full_like(s, 8.0) if zeros is None else np.repeat(zeros.astype(np.float64), g, axis=-1)
    return q, s, z


def w4_weight(w, kind):
    q, s, z = w4_parts(w, kind)
    return s * (q - z)


def w4_mm(a, w, kind):
    """The product in 64 bits and, per element, the sum of magnitudes that the
    kernel's fp32 sums pass through: |s| * (16 + q + 16 + z) * |a|."""
    q, s, z = w4_parts(w, kind)
    A = f64(a, kind)
    return A @ (s * (q - z)).T, np.abs(A) @ (np.abs(s) * (32.0 + q + z)).T


def _sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def _mm(a, w, kind, mag_w=None):
    """a [m][k] (64 bits) . w [n][k]^T with the magnitudes that fp32 sums pass
    through; w is (codes, scales, zeros) or bits."""
    if isinstance(w, tuple):
        q, s, z = w4_parts(w, kind)
        return a @ (s * (q - z)).T, np.abs(a) @ (np.abs(s) * (32.0 + q + z)).T
    W = f64(w, kind)
    return a @ W.T, np.abs(a) @ np.abs(W).T


def pick(w, e):
    return tuple(None if t is None else t[e] for t in w) if isinstance(w, tuple) else w[e]


EPS = 2.0 ** -24


def _adds(k, w):
    """Additions that follow one another on a path of a sum over k, at most."""
    if isinstance(w, tuple):
        g = 2 * w[0].shape[-1] // w[1].shape[-1]
        return g + k // g + 12
    return k + 16


def _ffn(x, ex, w13, w2, p, ep, kind):
    """p * f(x) of one row in 64 bits, and a bound on the error of the same in
    fp32 sums, given x's error bound ex (0) and p's relative error ep:
    |silu'| <= 1.1; silu, the product and the planes round by at most
    16 * 2^-24 together."""
    d = x.shape[1]
    y, mag = _mm(x, w13, kind)
    ey = _adds(d, w13) * EPS * mag
    n = y.shape[1] // 2
    g, u, eg, eu = y[:, :n], y[:, n:], ey[:, :n], ey[:, n:]
    s = g * _sigmoid(g)
    h = s * u * p
    eh = p * (1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu) + np.abs(h) * (16 * EPS + ep)
    o, _ = _mm(h, w2, kind)
    _, mag = _mm(np.abs(h) + eh, w2, kind)
    _, prop = _mm(eh, w2, kind)
    return o, prop + _adds(n, w2) * EPS * mag, mag


def moe(x, router, w13, w2, topk, renorm, shared, kind, out):
    """(out, bound, ids, weights) of the layer in 64 bits; bound holds per
    element for fp32 sums and the output type's rounding.  Asserts that the
    logits leave no doubt about the top-k (inputs are chosen so)."""
    X = f64(x, kind)
    m, d = X.shape
    lg, mag = _mm(X, router, kind)
    el = (d + 16) * EPS * mag
    experts = lg.shape[1]
    ref = np.zeros((m, d))
    err = np.zeros((m, d))
    tot = np.zeros((m, d))
    ids = np.zeros((m, topk), np.int64)
    wts = np.zeros((m, topk))
    for t in range(m):
        order = sorted(range(experts), key=lambda e: (-lg[t, e], e))
        for a, b in zip(order[:topk], order[1:topk + 1]):
            assert lg[t, a] == lg[t, b] or lg[t, a] - lg[t, b] > 4e-6, "inputs with a doubtful top-k"
        ids[t] = order[:topk]
        p = np.exp(lg[t] - lg[t].max())
        p /= p[ids[t]].sum() if renorm else p.sum()
        wts[t] = p[ids[t]]
        ep = 2 * float(el[t].max()) + (experts + 16) * EPS
        for e in sorted(ids[t]):
            o, eo, mg = _ffn(X[t:t + 1], 0.0, pick(w13, e), pick(w2, e), p[e], ep, kind)
            ref[t] += o[0]
            err[t] += eo[0]
            tot[t] += mg[0]
        if shared is not None:
            s13, s2, sg = shared
            v = float((X[t] * f64(sg, kind)).sum())
            ev = (d + 16) * EPS * float((np.abs(X[t]) * np.abs(f64(sg, kind))).sum())
            o, eo, mg = _ffn(X[t:t + 1], 0.0, s13, s2, _sigmoid(v), ev + 8 * EPS, kind)
            ref[t] += o[0]
            err[t] += eo[0]
            tot[t] += mg[0]
    err = err + (topk + 16) * EPS * tot
    return ref, err * (1 + ULP[out]) + ULP[out] * np.abs(ref) + TINY[out], ids, wts


def logprobs(x, tokens, topk):
    """(logprob, entropy, rank, ids, top logprobs) of rows x [m][V] in 64 bits,
    and error bounds of the fp32 evaluation for the two sums' results and, per
    row, of any log probability x_j - M - ln S at distance |x_j - M|.

    With d = x - M: t = d log2 e is off by 2 * 2^-24 |t|, so a term p = 2^t by
    (2 |d| + 4) * 2^-23 relatively; a thread adds at most V/256 + 64 terms one
    after another, each step rounding three times when its maximum grows."""
    m, V = x.shape
    adds = 4 * (V // 256 + 64) * EPS
    lp = np.zeros(m)
    ent = np.zeros(m)
    rank = np.zeros(m, np.int64)
    ids = np.zeros((m, topk), np.int64)
    top = np.zeros((m, topk))
    blp = np.zeros(m)
    bent = np.zeros(m)
    btop = np.zeros((m, topk))
    for r in range(m):
        v, t = x[r], int(tokens[r])
        order = np.lexsort((np.arange(V), -v))[:topk]
        ids[r] = order
        known = 0 <= t < V
        rank[r] = 1 + np.sum(v > v[t]) + np.sum(v[:t] == v[t]) if known else 0
        M = v.max()
        if M == -np.inf:
            lp[r], ent[r], top[r] = (-np.inf if known else np.nan), 0.0, -np.inf
            continue
        d = v - M
        p = np.exp(d)
        S = p.sum()
        p /= S
        dz = np.where(np.isfinite(d), d, 0.0)
        term = (2 * np.abs(dz) + 4) * 2 * EPS + adds
        rs = float((p * term).sum())  # S's relative error
        lnS = np.log(S)
        ent[r] = lnS - (p * dz).sum()
        mean = abs(float((p * dz).sum()))
        bent[r] = rs + float((p * np.abs(dz) * term).sum()) + mean * rs + 8 * EPS * (lnS + mean + 1)
        lp[r] = d[t] - lnS if known else np.nan
        top[r] = d[order] - lnS
        blp[r] = rs + 8 * EPS * (lnS + 1 + (abs(d[t]) if known and np.isfinite(d[t]) else 0))
        btop[r] = rs + 8 * EPS * (lnS + 1 + np.where(np.isfinite(d[order]), np.abs(d[order]), 0))
    return (lp, ent, rank, ids, top), (blp, bent, btop)
