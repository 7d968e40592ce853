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
