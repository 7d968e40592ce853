"""GPU parity of the GEMV on 4-bit weights with group scales against a plain
product in 64 bits.

Tolerance: the products (16 + q) * a and 1 * a are exact in fp32, so an error
comes from additions alone.  At most group + k/group + 8 of them follow one
another on a path (a group's sum, the groups of one wave, the waves), each
rounding by at most 2^-24 of what it has added up; with the two roundings of a
group's epilogue that is (group + k/group + 10) * 2^-24 * sum of magnitudes,
plus the output type's own rounding.
"""
import numpy as np
import pytest

import window_ref as R
import workloads as WL
from conftest import to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sk = pytest.importorskip("row_gemv_decode_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev_w4(w, kind):
    codes, scales, zeros = w
    return sk.W4(to_dev(codes, "u8"), to_dev(scales, kind), None if zeros is None else to_dev(zeros, "u8"))


def bound(ref, mag, group, k, out):
    return (group + k // group + 10) * 2.0 ** -24 * mag * (1 + R.ULP[out]) + R.ULP[out] * np.abs(ref) + R.TINY[out]


def check(m, n, k, group, kind, out, zeros, seed):
    print(f"w4 m={m} n={n} k={k} group={group} {kind} -> {out} zeros={zeros}", flush=True)
    a = WL.gen_matrix((m, k), kind, ("normal", 1.0), seed)
    w = R.gen_w4((n, k), group, kind, zeros, seed + 1)
    A, W = to_dev(a, kind), dev_w4(w, kind)
    got = sk.mm_w4(A, W, out_dtype=DT[out])
    torch.cuda.synchronize()
    ref, mag = R.w4_mm(a, w, kind)
    assert got.dtype == DT[out]
    res = got.double().cpu().numpy()
    assert np.all(np.abs(res - ref) <= bound(ref, mag, group, k, out))
    return A, W, got


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 2, 7, 16])
def test_w4_parity(m, group, kind):
    """Every group length and row type over a k of several units, with and
    without zero points, in every output type."""
    for zeros, out in ((True, "f32"), (False, "f32"), (True, kind), (False, "f16" if kind == "bf16" else "bf16")):
        check(m, 200, 1280, group, kind, out, zeros, 100 * m + group)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 33, 4097])
def test_w4_column_tails(n):
    check(3, n, 256, 64, "bf16", "f32", True, 7000 + n)


@pytest.mark.parametrize("k,group", [(32, 32), (64, 32), (96, 32), (160, 32), (64, 64), (192, 64), (1088, 64), (128, 128),
                                     (896, 128), (1056, 32), (9216, 128)])
def test_w4_k_tails(k, group):
    """k below, at and past a unit of 128, and a k whose last unit is partial."""
    for m in (1, 16):
        check(m, 50, k, group, "f16", "f32", True, 7100 + k)


@pytest.mark.parametrize("n", [16 * 1024 - 3, 16 * 8192 + 5])
def test_w4_many_columns(n):
    """Column counts past the steps of the tile choice."""
    check(2, n, 128, 128, "bf16", "f32", False, 7200)


def test_w4_random_shapes():
    rng = np.random.default_rng(7300)
    for i in range(24):
        group = int(rng.choice([32, 64, 128]))
        k = group * int(rng.integers(1, 40))
        kind = str(rng.choice(["bf16", "f16"]))
        check(int(rng.integers(1, 17)), int(rng.integers(1, 1500)), k, group, kind, str(rng.choice(["f32", "f16", "bf16"])),
              bool(rng.integers(2)), 7301 + i)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_w4_rows_do_not_depend_on_the_window(kind):
    """Row i at any m equals the one-row call, bit for bit."""
    for n, k, group in ((100, 1312, 32), (3000, 2560, 128)):
        A, W, full = check(16, n, k, group, kind, "f32", True, 7400)
        for m in (1, 3, 5, 8):
            assert torch.equal(sk.mm_w4(A[:m], W), full[:m])
        for r in (4, 15):
            assert torch.equal(sk.mm_w4(A[r:r + 1], W)[0], full[r])


def test_w4_strided_rows_and_output():
    """lda > k and ldc > n; the columns between stay untouched."""
    m, n, k = 5, 37, 320
    a = WL.gen_matrix((m, 352), "bf16", ("normal", 1.0), 7500)
    w = R.gen_w4((n, k), 64, "bf16", True, 7501)
    buf = torch.full((m, 50), 123.0, device="cuda")
    got = sk.mm_w4(to_dev(a, "bf16")[:, 16:16 + k], dev_w4(w, "bf16"), out=buf[:, 3:3 + n])
    torch.cuda.synchronize()
    ref, mag = R.w4_mm(a[:, 16:16 + k], w, "bf16")
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= bound(ref, mag, 64, k, "f32"))
    assert bool((buf[:, :3] == 123.0).all()) and bool((buf[:, 3 + n:] == 123.0).all())


def test_w4_zero_rows_and_exact_codes():
    """A one-hot row picks single weights out exactly: every code value at
    every position of a byte and unit."""
    k, group = 256, 32
    q = (np.arange(16)[:, None] + np.arange(k)[None, :]).astype(np.uint8) % 16
    codes = (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)
    scales = WL.to_bits(np.full((16, k // group), 0.5), "bf16")
    zeros = (np.arange(16 * (k // group)).reshape(16, -1) % 16).astype(np.uint8)
    W = dev_w4((codes, scales, zeros), "bf16")
    want = 0.5 * (q.astype(np.float64) - np.repeat(zeros, group, axis=1))
    for k0 in range(0, k, 16):
        A = torch.zeros((16, k), dtype=torch.bfloat16, device="cuda")
        A[torch.arange(16), k0 + torch.arange(16)] = 2.0
        A[3] = 0.0
        got = sk.mm_w4(A, W).double().cpu().numpy()
        ref = 2.0 * want[:, k0:k0 + 16].T
        ref[3] = 0.0
        assert np.array_equal(got, ref)


def test_w4_on_another_stream():
    A, W, full = check(4, 700, 1024, 128, "bf16", "f32", True, 7600)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = sk.mm_w4(A, W)
    b = sk.mm_w4(A, W, stream=s)
    s.synchronize()
    assert torch.equal(a, full) and torch.equal(b, full)


def test_w4_graph_replay():
    A, W, full = check(4, 700, 1024, 64, "f16", "f32", True, 7700)
    out = torch.empty_like(full)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sk.mm_w4(A, W, out=out)
    for _ in range(4):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, full)
        torch.cuda.synchronize()


def test_w4_refusals():
    A = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((8, 64), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((8, 2), dtype=torch.bfloat16, device="cuda")
    W = sk.W4(codes, scales)
    with pytest.raises(TypeError):
        sk.mm_w4(A.half(), W)
    with pytest.raises(TypeError):
        sk.mm_w4(A, (codes, scales))
    with pytest.raises(ValueError):
        sk.mm_w4(A[:, :64], W)
    with pytest.raises(ValueError):
        sk.mm_w4(A.t().contiguous().t(), W)
    with pytest.raises(ValueError):
        sk.W4(codes, scales[:, :1].expand(8, 5))
    with pytest.raises(ValueError):
        sk.W4(codes, scales.repeat(1, 8))  # groups of 8
    with pytest.raises(TypeError):
        sk.W4(codes.to(torch.int8), scales)
    with pytest.raises(ValueError):
        sk.W4(codes.cpu(), scales)
    with pytest.raises(sk.SkinnyError):
        sk.mm_w4(torch.zeros((17, 128), dtype=torch.bfloat16, device="cuda"), W)
    with pytest.raises(sk.SkinnyError):
        sk.mm_w4(torch.zeros((2, 130), dtype=torch.bfloat16, device="cuda")[:, :128], W)  # lda % 8
    with pytest.raises(ValueError):
        sk.mm_w4(A, W, out=torch.zeros((2, 9), device="cuda"))


def test_w4_rows_that_share_memory():
    """One row expanded to several, and windows that overlap: as their copies."""
    _, W, _ = check(2, 300, 512, 64, "bf16", "f32", True, 7800)
    one = torch.randn((1, 512), generator=torch.Generator().manual_seed(7801)).to(torch.bfloat16).cuda()
    over = torch.randn(1024, generator=torch.Generator().manual_seed(7802)).to(torch.bfloat16).cuda().as_strided((5, 512), (128, 1))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for a in (one.expand(16, -1), over):
        want = sk.mm_w4(a.contiguous(), W)
        assert torch.equal(sk.mm_w4(a, W), want)
        b = sk.mm_w4(a, W, stream=s)
        s.synchronize()
        assert torch.equal(b, want)
    with pytest.raises(ValueError):
        sk.mm_w4(one, W, out=torch.zeros(300, device="cuda").expand(1, -1)[:, :299])
    with pytest.raises(ValueError):
        sk.mm_w4(one.expand(3, -1), W, out=torch.zeros(300, device="cuda").expand(3, -1))


@pytest.mark.parametrize("n,zeros", [((1 << 27) + 5, True), ((1 << 28) + 1, False), ((1 << 30) + 65, False)])
def test_w4_more_columns_than_a_launch(n, zeros):
    """Column counts past a launch's 2^27, and past 2^32 threads in all.  One-hot
    rows pick exact values, which are compared column by column."""
    print(f"w4 n={n} zeros={zeros}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    codes = torch.randint(0, 256, (n, 16), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(1, 9, (n, 1), dtype=torch.uint8, device="cuda", generator=g).to(torch.float16)
    z = torch.randint(0, 16, (n, 1), dtype=torch.uint8, device="cuda", generator=g) if zeros else None
    W = sk.W4(codes, scales, z)
    A = torch.zeros((1, 32), dtype=torch.float16, device="cuda")
    A[0, 21] = 1.0
    got = sk.mm_w4(A, W, out_dtype=torch.float16)
    for j in range(0, n, 1 << 26):
        q = (codes[j:j + (1 << 26), 10] >> 4).to(torch.float16)
        zz = 8.0 if z is None else z[j:j + (1 << 26), 0].to(torch.float16)
        assert torch.equal(got[0, j:j + (1 << 26)], scales[j:j + (1 << 26), 0] * (q - zz))


@pytest.mark.parametrize("k,group", [(2592, 32), (4096, 32), (8192, 32), (5184, 64), (7680, 64), (10368, 128), (16384, 128)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_w4_several_spans_of_scales(k, group, kind):
    """A k of more than 80 groups, whose scales are staged in several spans (the
    last of them short, the last unit partial): parity and row invariance at a
    column tail, and the same bits in wide weights, whose waves take two and
    four tiles of columns."""
    A, W, got = check(16, 50, k, group, kind, "f32", True, 7900 + k)
    check(3, 50, k, group, kind, "f32", False, 7901 + k)
    for m in (1, 5):
        assert torch.equal(sk.mm_w4(A[:m], W), got[:m])
    for n in (5011, 24603):
        reps = n // 50 + 1
        wide = sk.W4(*(t.repeat(reps, 1)[:n].contiguous() for t in (W.codes, W.scales, W.zeros)))
        full = sk.mm_w4(A[:3], wide)
        assert torch.equal(full, got[:3].repeat(1, reps)[:, :n])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("rows", ["centred", "offset", "outlier"])
@pytest.mark.parametrize("zeros", [True, False])
def test_w4_cancellation(zeros, rows, group, kind):
    """A group's sum is a difference: sum (16 + q) a - (16 + z) sum a, whose
    parts are some 5 times the result for centred rows and more for rows with a
    mean.  At most `group` additions form each part; an addition rounds by at
    most 2^-24 of what it has added up, 1/sqrt(3) of that in root mean square,
    and the sum so far is 1/sqrt(3) of the last one where it grows evenly.  So
    the error's root mean square is at most sqrt(2 group) * 2^-24 / 3 * the
    part's magnitudes, squared and added over the groups, next to the adding up
    of the groups: as much again."""
    m, n, k = 4, 300, 2560
    rng = np.random.default_rng(8000)
    v = rng.normal(0.0, 1.0, size=(m, k))
    if rows == "offset":
        v += 4.0
    if rows == "outlier":
        v[:, 1234] = 1000.0
    a, w = WL.to_bits(v, kind), R.gen_w4((n, k), group, kind, zeros, 8001)
    got = sk.mm_w4(to_dev(a, kind), dev_w4(w, kind)).double().cpu().numpy()
    q, s, z = R.w4_parts(w, kind)
    A = R.f64(a, kind)
    ref = A @ (s * (q - z)).T
    part = (np.abs(A)[:, None, :] * (np.abs(s) * (16.0 + np.maximum(q, z)))[None]).reshape(m, n, k // group, group).sum(-1)
    most = np.sqrt(2 * group) * 2.0 ** -24 / 3 * np.sqrt((part ** 2).sum(-1))
    off = np.sqrt(((got - ref) ** 2).mean())
    plain = (torch.from_numpy(A).float() @ torch.from_numpy(s * (q - z)).float().T).double().numpy()
    off32 = np.sqrt(((plain - ref) ** 2).mean())
    print(f"w4 {rows} group={group} zeros={zeros} {kind}: off {off:.2e}, in fp32 {off32:.2e}, outputs {np.sqrt((ref ** 2).mean()):.2e}", flush=True)
    assert off <= 2 * np.sqrt((most ** 2).mean())


@pytest.mark.parametrize("k,group", [(2048, 128), (2080, 32), (2112, 64), (5152, 32)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_w4_bits_do_not_depend_on_the_tiles(k, group, kind):
    """Column counts on both sides of every step of the tile choice, ends inside
    a workgroup's tiles among them: the columns' bits are those of a narrow call."""
    A, W, got = check(7, 50, k, group, kind, "f32", True, 8100 + k)
    for n in (16 * 256, 16 * 256 + 1, 16 * 512 + 1, 16 * 768, 16 * 768 + 9, 16 * 1639, 16 * 1639 + 1, 26297, 32765, 16 * 2048 + 1):
        reps = n // 50 + 1
        wide = sk.W4(*(t.repeat(reps, 1)[:n].contiguous() for t in (W.codes, W.scales, W.zeros)))
        assert torch.equal(sk.mm_w4(A, wide), got.repeat(1, reps)[:, :n])
