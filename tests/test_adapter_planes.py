"""How many bits of an adapter's inner values reach its output: inner values of 24
significant bits whose sums are exact in fp32, each multiplied by one weight, so that
only the product is left to round.

The kernels hold an inner value as three bf16 numbers, each the rounded remainder of
the last: the second is at most 2^-8 of it, the third 2^-16, and three times 8 bits
with signs hold 24 exactly.  The products are added from the smallest on: the last
addition rounds by at most a step of the result, 2^-23 (half of one where the matrix core
rounds to nearest), the up to three before it by steps of sums that are at most 2^-7 of
it, 3 * 2^-7 * 2^-23.  f16 weights are the exact sum of two bf16 numbers, the second at
most 2^-8 of them; its product with the third plane, at most 2^-24, is left out.
Together (1 + 0.03 + 0.5) * 2^-23."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

BOUND = 1.53 * 2.0 ** -23
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def inputs(m, k, n, count, rank, kind, seed):
    """x [m][k], A [count][rank][k], B [count][n][rank] and the rows' adapters."""
    rng = np.random.default_rng(seed)
    x = rng.integers(128, 256, (m, k)).astype(np.float32)
    A = np.zeros((count, rank, k), np.float32)
    for a in range(count):
        for r in range(rank):
            # 8 bits above 8 above 8
            A[a, r, rng.permutation(k)[:3]] = rng.choice([-1, 1], 3) * np.array([2.0 ** 8, 1, 2.0 ** -8])
    B = np.zeros((count, n, rank), np.float32)
    B[:, np.arange(n), np.arange(n) % rank] = torch.from_numpy(rng.normal(0, 1, (count, n))).to(DT[kind]).float().numpy()
    return x, A, B, rng.integers(0, count, m)


def exact(x, A, B, ids):
    out = np.empty((len(x), B.shape[1]))
    cols = np.arange(B.shape[1])
    for t, a in enumerate(ids):
        h = A[a].astype(np.float64) @ x[t]
        assert np.array_equal(h.astype(np.float32), h)
        out[t] = h[cols % A.shape[1]] * B[a, cols, cols % A.shape[1]]
    return out


def parts(v, count):
    """v as the sum of `count` bf16 numbers and what is left."""
    out = []
    for _ in range(count):
        out.append(torch.from_numpy(v).to(torch.bfloat16).double().numpy())
        v = v - out[-1]
    return out, v


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_bound_holds_with_all_planes_only(kind):
    """In 64 bits, from the planes: one left out, or one of the products with an f16
    weight's second part, passes the bound by far."""
    x, A, B, ids = inputs(4, 64, 200, 3, 16, kind, 1)
    ref, cols = exact(x, A, B, ids), np.arange(200)
    h = np.stack([A[a].astype(np.float64) @ x[t] for t, a in enumerate(ids)])[:, cols % 16]
    w = np.stack([B[a, cols, cols % 16] for a in ids]).astype(np.float64)
    planes, rest = parts(h, 3)
    assert not rest.any()
    weights, rest = parts(w, 1 if kind == "bf16" else 2)
    assert not rest.any()
    products = {(p, q): planes[p] * weights[q] for p in range(3) for q in range(len(weights)) if p + q < 3}
    total = sum(products.values())
    assert np.all(np.abs(total - ref) <= (2.0 ** -24 if kind == "f16" else 0.0) * np.abs(ref))
    for left_out, product in products.items():
        worst = np.max(np.abs(total - product - ref) / np.abs(ref))
        assert worst > 8 * BOUND, left_out


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,k,n,rank", [
    (3, 64, 300, 8), (9, 1000, 300, 16), (40, 520, 300, 32),  # both products in one launch
    (3, 4104, 300, 16), (20, 4104, 130, 32), (3, 520, 300, 40), (16, 520, 300, 64), (250, 520, 300, 64),  # a tile of 16 rows, held
    (3, 520, 600, 72), (20, 520, 600, 256), (300, 264, 600, 200),  # the steps of a long rank one after another
    (300, 264, 90, 24), (300, 264, 90, 64), (900, 128, 17003, 16), (900, 128, 17003, 64),  # 16 rows of a tile of 64, all of it
    (900, 128, 17003, 72), (900, 128, 17003, 128),  # four steps held
])
def test_inner_values_keep_24_bits(m, k, n, rank, kind):
    import row_gemv_decode_amd as sk

    x, A, B, ids = inputs(m, k, n, 5, rank, kind, m + rank)
    dev = [torch.from_numpy(v).to(DT[kind]).cuda() for v in (x, A, B)]
    got = sk.add_adapters(dev[0], sk.Adapters(dev[1], dev[2]), torch.from_numpy(ids).cuda(), out_dtype=torch.float32)
    ref = exact(x, A, B, ids)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= BOUND * np.abs(ref))
