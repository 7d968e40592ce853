"""Plain 64-bit references of the operators of a batch of requests (residual and
norm, low-rank adapters, logit adjustments) with bounds on the error of the same
in fp32: numpy only, nothing of the library."""
import numpy as np

from window_ref import EPS, TINY, ULP


def rms_norm(x, r, w, eps, group, d_adds):
    """(h, y, scales, y / scales, relative bound of y in fp32) of rows x [m][d] and a
    residual r (or None) in 64 bits.

    fp32: h rounds once; the sum of squares is off by at most `d_adds` additions
    and products that follow one another (relative to itself, all terms being
    positive), of which the square root takes half; mean, + eps, root, reciprocal
    and the two products round by 6 * 2^-24 more."""
    h = x if r is None else x + r
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    if w is not None:
        y = y * w
    m, d = y.shape
    size = group or d
    groups = -(-d // size)
    padded = np.zeros((m, groups * size))
    padded[:, :d] = y
    scales = np.maximum(np.abs(padded).reshape(m, groups, size).max(2) / 448.0, 2.0 ** -126)
    return h, y, scales, y / np.repeat(scales, size, axis=1)[:, :d], (0.5 * (d_adds + 2) + 8) * EPS


def adapters(x, A, B, ids, ranks, scaling, base, out):
    """(out, bound) in 64 bits of rows x [m][k], A [count][rank][k], B [count][n][rank];
    out names the output's type.

    fp32: sums of k (and of the rank) products, each product exact, so every
    addition rounds once: k + 64 of them on a path at the most.  The inner value is
    kept in three bf16 planes (2^-24) and f16 weights in two, without the product
    of the lowest two (2^-16 * 2^-8); the scaled sum and the base's addition round
    once more."""
    m, n = x.shape[0], B.shape[1]
    ref = np.zeros((m, n)) if base is None else base.astype(np.float64).copy()
    err = np.zeros((m, n))
    for t in range(m):
        a = int(ids[t])
        if not 0 <= a < A.shape[0]:
            continue
        r = A.shape[1] if ranks is None else int(ranks[a])
        if not 1 <= r <= A.shape[1]:
            continue
        Aa, Ba = A[a, :r], B[a, :, :r]
        s = 1.0 if scaling is None else float(scaling[a])
        h = Aa @ x[t]
        eh = (x.shape[1] + 64) * EPS * (np.abs(Aa) @ np.abs(x[t])) + 4 * EPS * np.abs(h)
        part = s * (Ba @ h)
        mag = abs(s) * (np.abs(Ba) @ (np.abs(h) + eh))
        err[t] = abs(s) * (np.abs(Ba) @ eh) + (5 * r + 16) * EPS * mag + 2 * EPS * (np.abs(part) + np.abs(ref[t]))
        ref[t] += part
    return ref, err * (1 + ULP[out]) + (ULP[out] * np.abs(ref) if out != "f32" else EPS * np.abs(ref)) + TINY[out]


def adjust(x, history, lengths, prompts, theta, freq, pres, bias_ids, bias_values, mask, mask_rows, out):
    """(out, bound, touched) in 64 bits of rows x [m][vocab]; any rule may be None.

    fp32 rounds the quotient, the product and the sum of the penalty, its
    subtraction, each bias's addition and the last one: each by 2^-24 of its result,
    which none of the magnitudes' sums below is smaller than."""
    m, V = x.shape
    ref = x.astype(np.float64).copy()
    err = np.zeros((m, V))
    touched = np.zeros((m, V), bool)
    for i in range(m):
        if history is not None:
            n = history.shape[1] if lengths is None else min(max(int(lengths[i]), 0), history.shape[1])
            p = 0 if prompts is None else min(max(int(prompts[i]), 0), n)
            toks = history[i, :n].astype(np.int64)
            ok = (toks >= 0) & (toks < V)
            seen = np.zeros(V, bool)
            seen[toks[ok]] = True
            made = toks[p:][ok[p:]]
            c = np.bincount(made, minlength=V).astype(np.float64)
            th = 1.0 if theta is None else float(theta[i])
            v = np.where(ref[i] > 0, ref[i] / th, ref[i] * th)
            ref[i] = np.where(seen, v, ref[i])
            f, q = (0.0 if t is None else float(t[i]) for t in (freq, pres))
            pen = np.where(c > 0, f * c + q, 0.0)
            with np.errstate(invalid="ignore"):
                err[i] += np.where(seen, EPS * (2 * np.abs(ref[i]) + 4 * np.abs(f * c) + 4 * abs(q)), 0.0)
            ref[i] -= pen
            touched[i] |= seen
        if bias_ids is not None:
            for j, b in zip(bias_ids[i].astype(np.int64), bias_values[i].astype(np.float64)):
                if 0 <= j < V:
                    ref[i, j] += b
                    # every addition rounds a sum that is at most the biases' magnitudes
                    err[i, j] += EPS * (bias_ids.shape[1] + 2) * abs(b) + EPS * np.abs(ref[i, j])
                    touched[i, j] = True
        if mask is not None:
            which = i if mask_rows is None else int(mask_rows[i])
            if 0 <= which < mask.shape[0]:
                bits = np.unpackbits(np.ascontiguousarray(mask[which]).view(np.uint8), bitorder="little")[:V]
                ref[i, bits == 0] = -np.inf
                touched[i, bits == 0] = True
    err = np.where(np.isfinite(ref), err, 0.0)
    step = np.where(np.isfinite(ref), ULP[out] * np.abs(ref), 0.0)
    return ref, err * (1 + ULP[out]) + step + TINY[out], touched
