"""GPU parity of the residual's addition and norm against 64 bits
(requests_ref.rms_norm, which derives the bounds of the fp32 sums)."""
import numpy as np
import pytest

import requests_ref as Q
from window_ref import EPS, TINY, ULP

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sk = pytest.importorskip("row_gemv_decode_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def store(a, kind):
    t = torch.from_numpy(np.asarray(a, np.float64)).to(DT[kind])
    return t.cuda(), t.double().numpy()


def adds(d):
    """Additions of squares that follow one another: a lane's values (at most 8 of
    every chunk of a thread), the wave's and the workgroup's reductions."""
    return 32 + 8 + 16 + (d + 8191) // 8192 * 9


def inputs(m, d, xk, rk, wk, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (m, d)) * np.exp(rng.normal(0, 1, (m, 1)))
    x[:, :: max(1, d // 3)] *= 30
    X = store(x, xk)
    R = store(rng.normal(0, 2, (m, d)), rk) if rk else (None, None)
    W = store(rng.uniform(0.5, 1.5, d), wk) if wk else (None, None)
    return X, R, W


def check_values(got, x, r, w, kinds, eps, group):
    """kinds: types of residual and out (or None)."""
    rk, ok = kinds
    h, y, scales, quot, rel = Q.rms_norm(x, r, w, eps, group or 0, adds(x.shape[1]))
    if got.residual is not None:
        assert np.all(np.abs(got.residual.double().cpu().numpy() - h) <= (ULP[rk] + 2 * EPS) * np.abs(h) + TINY[rk])
    if got.out is not None:
        o = got.out.double().cpu().numpy()
        assert np.all(np.abs(o - y) <= (rel + ULP[ok] * (1 + rel)) * np.abs(y) + TINY[ok])
    if got.q is not None:
        s = got.scales.double().cpu().numpy()
        assert s.shape == scales.shape
        assert np.all(np.abs(s - scales) <= (rel + 2 * EPS) * scales)
        q = got.q.float().double().cpu().numpy()
        # half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6) from the quotient of
        # rows off by rel, whose scale is off by as much, and its own three roundings
        off = np.abs(quot) * (2 * rel + 8 * EPS)
        assert np.all(np.abs(q - quot) <= np.maximum(2.0 ** -4 * (np.abs(quot) + off), 2.0 ** -10) + off)


def check(m, d, xk="bf16", rk="bf16", wk="bf16", ok="bf16", group=None, eps=1e-6, seed=0):
    print(f"norm m={m} d={d} {xk} {rk} {wk} -> {ok} group={group}", flush=True)
    X, R, W = inputs(m, d, xk, rk, wk, seed + 31 * m + d)
    got = sk.rms_norm(X[0], W[0], eps, residual=R[0], out_dtype=DT[ok] if ok else None, quant=group)
    torch.cuda.synchronize()
    assert (got.out is None) == (ok is None and group is not None) and (got.residual is None) == (rk is None)
    check_values(got, X[1], R[1], W[1], (rk, ok or xk), eps, group)
    return X, R, W, got


LENGTHS = [1, 2, 7, 8, 9, 63, 64, 65, 96, 127, 128, 200, 256, 511, 512, 513, 520, 896, 1016, 1024, 1025, 1032, 2561, 4133, 5120,
           8192, 8193, 8200, 16384, 16392, 20011, 32768, 32769, 32776, 40000]


@pytest.mark.parametrize("d", LENGTHS)
def test_norm_lengths(d):
    """From one value on, at and past a chunk, a group of lanes, a wave, a
    workgroup's registers."""
    check(3, d)
    check(2, d, "f16", None, "f32", None, 0)
    check(2, d, "f32", "f32", None, "f32", 64)


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("d", [1, 31, 64, 96, 130, 250, 896, 1000, 2560, 4133, 9000, 33000])
def test_norm_scales(d, group):
    """A scale per row or per group, the row's last group shorter, rows of less
    than a group."""
    check(5, d, "bf16", "f32", "bf16", None, group)
    check(2, d, "f16", "f16", "f16", "f16", group)


@pytest.mark.parametrize("m,d,group", [(2048, 5120, 0), (2048, 5120, 64), (20000, 512, 32), (250, 40000, 0), (250, 40000, 128)])
def test_norm_codes_are_the_quotients(m, d, group):
    """Every code is y / scale in fp32, rounded to 8 bits: a quotient off by a step in 24
    bits shows as codes on the wrong side of a border, up to tens in ten million."""
    gen = torch.Generator(device="cuda").manual_seed(m + group)
    x = torch.randn((m, d), generator=gen, device="cuda")
    x[:, 7] = -0.0
    w = torch.rand(d, generator=gen, device="cuda") + 0.5
    got = sk.rms_norm(x, w, out_dtype=torch.float32, quant=group)
    y, s = got.out.cpu().numpy(), got.scales.cpu().numpy()
    quot = torch.from_numpy(y / np.repeat(s, group or d, axis=1)[:, :d])
    want = quot.to(torch.float8_e4m3fn).view(torch.uint8)
    assert int((got.q.cpu().view(torch.uint8) != want).sum()) == 0


@pytest.mark.parametrize("d", [64, 5120, 40000])
@pytest.mark.parametrize("group", [0, 32])
def test_norm_codes_beside_an_overflow(d, group):
    """A value past fp32 makes its group's scale infinite: the others' quotients are 0, its own
    NaN; other groups and rows do not notice."""
    x = torch.ones((3, d), device="cuda")
    x[1, 1] = 1e18
    w = torch.ones(d, device="cuda")
    w[1] = 1e25
    got = sk.rms_norm(x, w, out_dtype=torch.float32, quant=group)
    y, s = got.out.cpu().numpy(), got.scales.cpu().numpy()
    assert np.isinf(y[1, 1]) and np.isinf(s[1, 0]) and np.isfinite(s[0]).all()
    with np.errstate(invalid="ignore"):
        want = torch.from_numpy(y / np.repeat(s, group or d, axis=1)[:, :d]).to(torch.float8_e4m3fn).float()
    assert torch.equal(got.q.cpu().float().nan_to_num(nan=1000.0), want.nan_to_num(nan=1000.0))
    assert int(want.isnan().sum()) == 1 and not want[1, 2:group or d].any()


@pytest.mark.parametrize("ok", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("xk,rk,wk", [("f32", "f32", "f32"), ("f32", None, None), ("f16", "f16", "f16"), ("f16", "f32", "f32"),
                                      ("bf16", "bf16", "bf16"), ("bf16", "f32", "bf16"), ("bf16", None, "f32"), ("f32", "bf16", "f16"), ("f32", "f16", "f32"), ("f16", "bf16", "bf16"),
                                      ("bf16", "f16", None)])
def test_norm_types(xk, rk, wk, ok):
    for d in (72, 640, 2560):
        check(4, d, xk, rk, wk, ok)


@pytest.mark.parametrize("m,d", [(1, 64), (31, 64), (33, 72), (1000, 128), (257, 896), (4099, 40), (300, 5120), (70000, 8)])
def test_norm_row_counts(m, d):
    check(m, d, group=32 if d % 64 == 0 else None, ok="bf16")


def test_norm_rows_do_not_depend_on_the_others():
    for d in (128, 896, 5120, 33000):
        X, R, W = inputs(21, d, "bf16", "bf16", "bf16", 5)
        one = [sk.rms_norm(X[0][i:i + 1], W[0], residual=R[0][i:i + 1], out_dtype=torch.bfloat16, quant=64) for i in range(21)]
        for m in (2, 7, 21):
            got = sk.rms_norm(X[0][:m], W[0], residual=R[0][:m], out_dtype=torch.bfloat16, quant=64)
            for i in range(m):
                for a, b in zip(got, one[i]):
                    assert torch.equal(a[i].view(torch.uint8), b[0].view(torch.uint8))


@pytest.mark.parametrize("d", [896, 4104, 5120, 7681, 8192, 9000])
def test_norm_rows_are_the_same_bits_in_a_large_batch(d):
    """Also where a large batch gives a row fewer threads."""
    X, R, W = inputs(600, d, "bf16", "f32", "bf16", 6)
    got = sk.rms_norm(X[0], W[0], residual=R[0], out_dtype=torch.float32, quant=0)
    for m in (1, 37, 511, 512):
        part = sk.rms_norm(X[0][:m], W[0], residual=R[0][:m], out_dtype=torch.float32, quant=0)
        for a, b in zip(got, part):
            assert torch.equal(a[:m].view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("offset", [0, 1, 3, 4, 7])
@pytest.mark.parametrize("d", [40, 896, 2561])
def test_norm_alignment_and_strides(d, offset):
    """Rows that start at every element; what lies between the rows stays."""
    m = 5
    X, R, W = inputs(m, d, "bf16", "f32", "bf16", offset)

    def strided(t, dtype, ld):
        big = torch.full((m * ld + 64,), 3.0, device="cuda").to(dtype)
        view = big[offset:offset + m * ld].view(m, ld)[:, :d]
        if t is not None:
            view.copy_(t)
        return big, view

    _, x = strided(X[0], torch.bfloat16, d + 5)
    _, r = strided(R[0], torch.float32, d + 9)
    w = torch.empty(d + 8, dtype=torch.bfloat16, device="cuda")[offset:offset + d].copy_(W[0])
    bo, out = strided(None, torch.float16, d + 3)
    br, ro = strided(None, torch.float32, d + 1)
    bq, q = strided(None, torch.float8_e4m3fn, d + 7)
    got = sk.rms_norm(x, w, residual=r, residual_out=ro, out=out, quant=32, q=q)
    torch.cuda.synchronize()
    assert got.out is out and got.residual is ro and got.q is q
    check_values(got, X[1], R[1], W[1], ("f32", "f16"), 1e-6, 32)
    for big, ld in ((bo, d + 3), (br, d + 1), (bq, d + 7)):
        rest = torch.ones_like(big, dtype=torch.bool)
        rest[offset:offset + m * ld].view(m, ld)[:, :d] = False
        assert bool((big.float()[rest] == 3.0).all())


@pytest.mark.parametrize("d", [65, 896, 5120, 33001])
def test_norm_in_place(d):
    """residual_out over the residual, out over x."""
    X, R, W = inputs(9, d, "bf16", "bf16", "bf16", 3)
    want = sk.rms_norm(X[0], W[0], residual=R[0], out_dtype=torch.bfloat16, quant=0)
    x, r = X[0].clone(), R[0].clone()
    got = sk.rms_norm(x, W[0], residual=r, residual_out=r, out=x, quant=0)
    assert got.out is x and got.residual is r
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_norm_expanded_rows_are_copied():
    X, R, W = inputs(1, 640, "f16", "f16", "f16", 4)
    got = sk.rms_norm(X[0].expand(6, 640), W[0], residual=R[0].expand(6, 640))
    one = sk.rms_norm(X[0], W[0], residual=R[0])
    assert torch.equal(got.out, one.out.expand(6, 640)) and torch.equal(got.residual, one.residual.expand(6, 640))


@pytest.mark.parametrize("d", [64, 1000, 5120, 33000])
def test_norm_zero_and_small_rows(d):
    """Zeros give zeros (codes 0, the least scale); rows so small that eps decides;
    rows near the type's limits."""
    x = np.zeros((5, d))
    x[1] = 1e-7
    x[2] = 6e4
    x[3, d // 2] = -5e4
    x[4, :] = np.where(np.arange(d) % 2 == 0, 1e-5, -3.0)
    for xk in ("f32", "f16"):
        X = store(x, xk)
        got = sk.rms_norm(X[0], None, 1e-5, out_dtype=torch.float32, quant=0)
        torch.cuda.synchronize()
        check_values(got, X[1], None, None, (None, "f32"), 1e-5, 0)
        assert not got.q[0].float().any() and float(got.scales[0]) == 2.0 ** -126


def test_norm_non_finite_values_stay_in_their_row():
    X, _, W = inputs(6, 896, "bf16", None, "bf16", 8)
    want = sk.rms_norm(X[0], W[0], out_dtype=torch.bfloat16, quant=128)
    x = X[0].clone()
    x[1, 5], x[4, 800] = float("nan"), float("inf")
    got = sk.rms_norm(x, W[0], out_dtype=torch.bfloat16, quant=128)
    for i in (0, 2, 3, 5):
        for a, b in zip((got.out, got.q, got.scales), (want.out, want.q, want.scales)):
            assert torch.equal(a[i].view(torch.uint8), b[i].view(torch.uint8))
    assert bool(got.out[1].isnan().all()) and bool(got.q[1].float().isnan().all())


def test_norm_large_offsets():
    """Rows whose places pass 2^31 elements."""
    d, ld = 64, 1 << 28
    big = torch.empty(9 * ld + d, dtype=torch.float16, device="cuda")
    x = big[:9 * ld].view(9, ld)[:, :d]
    X, _, W = inputs(9, d, "f16", None, "f16", 9)
    x.copy_(X[0])
    got = sk.rms_norm(x, W[0])
    assert torch.equal(got.out, sk.rms_norm(X[0], W[0]).out)
    del big, x
    torch.cuda.empty_cache()


def test_norm_streams_and_graphs():
    """On another stream, and captured: every replay equals the eager result."""
    X, R, W = inputs(17, 2560, "bf16", "bf16", "bf16", 10)
    want = sk.rms_norm(X[0], W[0], residual=R[0], out_dtype=torch.bfloat16, quant=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sk.rms_norm(X[0], W[0], residual=R[0], out_dtype=torch.bfloat16, quant=128, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    x = X[0].clone()
    with torch.cuda.graph(g):
        cap = sk.rms_norm(x, W[0], residual=R[0], out_dtype=torch.bfloat16, quant=128)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for k in range(3):
        x.copy_(X[0] * (1 + k))
        g.replay()
        eager = sk.rms_norm(x, W[0], residual=R[0], out_dtype=torch.bfloat16, quant=128)
        torch.cuda.synchronize()
        for a, b in zip(cap, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_norm_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w, y = torch.ones(64, dtype=torch.bfloat16, device="cuda"), x.clone()
    for kw in (dict(weight=w[:32]), dict(residual=x[:2]), dict(residual_out=x), dict(out=x[:, :32]), dict(q=x), dict(scales=x),
               dict(quant=0, scales=torch.zeros((4, 2), device="cuda")), dict(residual=x.cpu()), dict(weight=w.cpu())):
        with pytest.raises(ValueError):
            sk.rms_norm(x, **kw)
    for kw in (dict(quant=48), dict(quant=-1), dict(weight=w.double()), dict(residual=x.double()), dict(eps=-1.0),
               dict(eps=float("nan")), dict(out_dtype=torch.float64), dict(residual=x.clone(), residual_out=x),
               dict(residual=x.clone(), out=y, residual_out=y)):
        with pytest.raises(sk.SkinnyError):
            sk.rms_norm(x, **kw)
