"""GPU parity of the low-rank adapters against 64 bits (requests_ref.adapters, which
derives the bounds of the fp32 sums)."""
import threading

import numpy as np
import pytest

import requests_ref as Q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sk = pytest.importorskip("row_gemv_decode_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def store(a, kind):
    t = torch.from_numpy(np.asarray(a, np.float64)).to(DT[kind])
    return t.cuda(), t.double().numpy()


class Case:
    def __init__(self, m, k, n, count, rank, kind="bf16", base="bf16", ranks=None, scaling=True, ids=None, seed=0):
        print(f"adapters m={m} k={k} n={n} {count} of rank {rank} {kind} base={base}", flush=True)
        rng = np.random.default_rng(seed + m + k + n)
        self.kind, self.base_kind = kind, base
        self.x = store(rng.normal(0, 1, (m, k)), kind)
        self.A = store(rng.normal(0, k ** -0.5, (count, rank, k)), kind)
        self.B = store(rng.normal(0, rank ** -0.5, (count, n, rank)), kind)
        self.scaling = rng.uniform(0.5, 2, count).astype(np.float32) if scaling else None
        self.ranks = None if ranks is None else np.resize(np.asarray(ranks, np.int32), count)
        self.ids = rng.integers(-1, count, m) if ids is None else np.resize(np.asarray(ids), m)
        self.base = store(rng.normal(0, 1, (m, n)), base) if base else (None, None)
        self.pool = sk.Adapters(self.A[0], self.B[0], scaling=None if self.scaling is None else torch.from_numpy(self.scaling).cuda(),
                                ranks=None if self.ranks is None else torch.from_numpy(self.ranks).cuda())
        self.dev_ids = torch.from_numpy(self.ids.astype(np.int32)).cuda()

    def run(self, out_kind=None, **kw):
        return sk.add_adapters(self.x[0], self.pool, self.dev_ids, self.base[0],
                               out_dtype=DT[out_kind] if out_kind else None, **kw)

    def check(self, out_kind=None, got=None):
        got = self.run(out_kind) if got is None else got
        torch.cuda.synchronize()
        kind = out_kind or self.base_kind or self.kind
        ref, bound = Q.adapters(self.x[1], self.A[1], self.B[1], self.ids, self.ranks, self.scaling, self.base[1], kind)
        assert got.dtype == DT[kind]
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= bound)
        return got


@pytest.mark.parametrize("kind,base,out", [("bf16", "bf16", "bf16"), ("f16", "f32", "f32"), ("bf16", "f32", "bf16"),
                                           ("f16", "f16", "f32"), ("bf16", None, "f32"), ("f16", None, None)])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 65, 200, 256, 257, 300])
def test_adapters_row_counts(m, kind, base, out):
    """Across the ways of finding an adapter's rows, and the types."""
    Case(m, 264, 200, 5, 16, kind, base).check(out)


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128, 136, 200, 256])
@pytest.mark.parametrize("m", [3, 270])
def test_adapters_ranks(rank, m):
    Case(m, 320, 136, 3, rank, "bf16").check("f32")
    Case(m, 320, 136, 3, rank, "f16", "f32").check()


@pytest.mark.parametrize("m", [6, 300])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_adapters_of_several_ranks(m, kind):
    """Each adapter's own rank, odd ones too; ranks outside 1 .. rank add nothing; what
    the pool holds past them is not used, even if it is NaN."""
    own = [1, 2, 5, 8, 13, 16, 17, 31, 32, 33, 47, 48, 0, -3, 49]
    c = Case(m, 200, 70, 15, 48, kind, "f32", ranks=own)
    for a, r in enumerate(own):
        r = r if 1 <= r <= 48 else 0
        c.A[0][a, r:] = float("nan")
        c.B[0][a, :, r:] = float("nan")
    c.check()
    c.check(kind)


@pytest.mark.parametrize("k", [8, 16, 24, 32, 40, 56, 64, 72, 248, 256, 264, 512, 1000, 1032, 2560, 5128, 9000])
@pytest.mark.parametrize("m", [2, 260])
def test_adapters_lengths_of_k(k, m):
    Case(m, k, 64, 4, 16, "bf16").check("f32")
    Case(m, k, 40, 3, 40, "f16", "f32").check()


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1000, 1023, 1025, 2053])
@pytest.mark.parametrize("m", [3, 280])
def test_adapters_widths(n, m):
    Case(m, 64, n, 4, 16, "bf16").check()
    Case(m, 64, n, 4, 24, "f16", "f32").check()
    Case(m, 64, n, 4, 8, "bf16", "f32").check("bf16")


@pytest.mark.parametrize("m,count", [(17, 3), (40, 3), (64, 70), (100, 2), (130, 200), (256, 20), (256, 1)])
def test_adapters_middle_batches(m, count):
    """In one launch and in two, by adapter and by row, with several tiles of an adapter."""
    Case(m, 1000, 130, count, 16, "bf16").check()
    Case(m, 4096, 1100, count, 16, "f16", "f32").check()
    Case(m, 520, 300, count, 32, "bf16", "f32").check("bf16")
    Case(m, 2048, 1100, count, 32, "f16", "f16").check()
    Case(m, 1024, 300, count, 8, "f16", "f32", ids=[0]).check()


@pytest.mark.parametrize("rank,kind,base", [(72, "bf16", "f32"), (96, "f16", "f16"), (104, "f16", "f32"), (128, "bf16", "bf16"),
                                            (128, "f16", None)])
def test_adapters_long_ranks_of_many_rows(rank, kind, base):
    """Whole tiles of 64 rows with a long rank."""
    Case(700, 64, 17003, 12, rank, kind, base, ranks=[rank, rank - 3, 33, 64, 7, rank]).check("f32")


@pytest.mark.parametrize("m", [16, 250, 600])
def test_adapters_ids(m):
    """One adapter for all, none at all, runs, every row its own, ids out of range."""
    rng = np.random.default_rng(1)
    for ids in ([2], [-1], [0, 1], np.repeat([3, -1, 0, 2], m // 4 + 1)[:m], rng.permutation(m) % 9, [9, 1 << 30, -(1 << 31), 8, 7],
                np.where(np.arange(m) == m - 1, 5, 0)):
        c = Case(m, 128, 96, 9, 16, "bf16", ids=ids)
        want = c.check()
        c.dev_ids = c.dev_ids.long()
        if 1 << 30 in c.ids:  # past 32 bits as well
            c.dev_ids[0] = 1 << 40
            c.dev_ids[m - 1] = -(1 << 40) + 1
            want = want.clone()
            want[0], want[m - 1] = c.base[0][0], c.base[0][m - 1]
        assert torch.equal(c.run(), want)


def test_adapters_many_and_large():
    """More adapters than rows, and thousands of rows of one."""
    Case(40, 64, 48, 3000, 8, "bf16").check()
    Case(700, 64, 48, 8192, 8, "bf16").check()
    ids = np.sort(np.random.default_rng(2).integers(-1, 3, 5000))
    Case(5000, 72, 80, 3, 16, "f16", "f16", ids=ids).check()


@pytest.mark.parametrize("rank", [8, 16, 24, 32])
@pytest.mark.parametrize("kind,base", [("bf16", "bf16"), ("f16", "f32"), ("bf16", None)])
def test_adapters_bits_are_those_of_the_one_row_call(kind, base, rank):
    """Across the sizes at which a window's rows are one launch's or two's, for k of a
    part of a split, one, several, and an odd end."""
    for k, n in ((72, 5003), (512, 40), (1096, 5003), (2040, 4100), (4096, 2570), (4104, 700)):
        c = Case(16, k, n, 4, rank, kind, base, ids=[0, 1, -1, 3, 3, 2])
        want = c.check()
        for m in (1, 3, 6, 7, 9, 12, 13, 15):
            got = sk.add_adapters(c.x[0][:m], c.pool, c.dev_ids[:m], None if base is None else c.base[0][:m])
            assert torch.equal(got, want[:m])
        for i in (2, 5, 15):
            got = sk.add_adapters(c.x[0][i:i + 1], c.pool, c.dev_ids[i:i + 1], None if base is None else c.base[0][i:i + 1])
            assert torch.equal(got[0], want[i])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_adapters_rows_do_not_depend_on_the_batch(kind):
    """Row i of up to 16 rows is the one-row call's, bit for bit, whichever adapters the
    others use; in larger batches it does not depend on the others' values or order."""
    c = Case(16, 1504, 333, 4, 24, kind, "f32")
    one = [sk.add_adapters(c.x[0][i:i + 1], c.pool, c.dev_ids[i:i + 1], c.base[0][i:i + 1]) for i in range(16)]
    for m in (1, 2, 5, 9, 16):
        got = sk.add_adapters(c.x[0][:m], c.pool, c.dev_ids[:m], c.base[0][:m])
        assert all(torch.equal(got[i], one[i][0]) for i in range(m))
    for m in (100, 500):
        c = Case(m, 520, 100, 4, 24, kind, "f32")
        want = c.run()
        p = torch.from_numpy(np.random.default_rng(3).permutation(m)).cuda()
        got = sk.add_adapters(c.x[0][p], c.pool, c.dev_ids[p], c.base[0][p])
        assert torch.equal(got, want[p])


def test_adapters_rows_without_one_are_not_read():
    """Their x may be anything; their base comes through unchanged."""
    for m in (12, 300):
        c = Case(m, 64, 50, 3, 8, "bf16", ids=[0, -1, 2, 7])
        c.x[0][1::4] = float("nan")
        c.x[0][3::4] = float("inf")
        got = c.run()
        assert torch.equal(got[1::4], c.base[0][1::4]) and torch.equal(got[3::4], c.base[0][3::4])
        c.x[0][1::4] = c.x[0][3::4] = 0.0
        assert torch.equal(got, c.run())


@pytest.mark.parametrize("m", [5, 290])
@pytest.mark.parametrize("kind,base", [("bf16", "bf16"), ("f16", "f32")])
def test_adapters_in_place_and_strides(m, kind, base):
    """Into the base itself: columns of a wider projection's output, beside which
    nothing is written; x with padded rows."""
    c = Case(m, 80, 77, 4, 16, kind, base)
    want = c.check()
    wide = torch.full((m, 200), 5.0, dtype=DT[base], device="cuda")
    for first in (0, 1, 3, 100):
        part = wide[:, first:first + 77]
        part.copy_(c.base[0])
        x = torch.zeros((m, 96), dtype=DT[kind], device="cuda")
        x[:, 8:88] = c.x[0]
        got = sk.add_adapters(x[:, 8:88], c.pool, c.dev_ids, part, out=part)
        assert got is part and torch.equal(part, want)
        assert bool((wide[:, :first] == 5).all()) and bool((wide[:, first + 77:] == 5).all())
        part.fill_(5.0)
    one = c.x[0][:1].expand(m, 80)
    assert torch.equal(sk.add_adapters(one, c.pool, c.dev_ids, c.base[0][:1].expand(m, 77)),
                       sk.add_adapters(one.contiguous(), c.pool, c.dev_ids, c.base[0][:1].expand(m, 77).contiguous()))


def test_adapters_values_from_small_to_large():
    """Inner values far below and above 1: the planes keep 24 bits wherever they lie."""
    for kind, scale in (("bf16", 1e-12), ("bf16", 1e12), ("f16", 1e-3), ("f16", 300.0)):
        c = Case(20, 256, 90, 3, 32, kind, "f32")
        c.x[0].copy_((c.x[0].float() * scale).to(DT[kind]))
        c.x = (c.x[0], c.x[0].double().cpu().numpy())
        c.base = (c.base[0] * scale, (c.base[0] * scale).double().cpu().numpy())
        c.check()


def test_adapters_large_offsets():
    """A pool and rows whose places pass 2^31 elements."""
    count, k, n, rank = 70, 4096, 8192 * 16, 256
    A = torch.zeros((count, rank, k), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros((count, n, rank), dtype=torch.bfloat16, device="cuda")
    A[69, :, :] = 2.0 ** -10
    B[69, :, 255] = 1.0
    x = torch.ones((2, k), dtype=torch.bfloat16, device="cuda")
    out = sk.add_adapters(x, sk.Adapters(A, B), torch.tensor([69, 3], device="cuda"))
    assert bool((out[0] == 4.0).all()) and not bool(out[1].any())
    del A, B
    torch.cuda.empty_cache()


def test_adapters_streams_graphs_and_threads():
    """Each stream has its own workspace and a capture one of its own; threads on one
    stream do not interleave their launches."""
    for m, rank in ((9, 16), (9, 40), (300, 16), (300, 256), (100, 128)):
        c, d = Case(m, 512, 120, 4, rank, "bf16"), Case(m, 512, 120, 4, rank, "bf16", seed=50)
        want, other = c.run(), d.run()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = [c.run(stream=s) for _ in range(3)]
        s.synchronize()
        assert all(torch.equal(g, want) for g in got)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cap = c.run()
        x = c.x[0].clone()
        for k in range(3):
            c.x[0].copy_(x * (k + 1))
            g.replay()
            assert torch.equal(d.run(), other)
            eager = c.run()
            torch.cuda.synchronize()
            assert torch.equal(cap, eager)
        c.x[0].copy_(x)
        bad = []

        def work(case, wanted, bad=bad):
            for _ in range(20):
                if not torch.equal(case.run(), wanted):
                    bad.append(1)

        threads = [threading.Thread(target=work, args=a) for a in ((c, want), (d, other))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not bad


def test_adapters_refusals():
    half = dict(dtype=torch.bfloat16, device="cuda")
    A, B, x = torch.zeros((2, 8, 16), **half), torch.zeros((2, 5, 8), **half), torch.zeros((3, 16), **half)
    f, i = torch.ones(2, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    for a in ((A.float(), B.float()), (A, B.half()), (A[0], B)):
        with pytest.raises(TypeError):
            sk.Adapters(*a)
    for a, kw in (((A, B[:1]), {}), ((A, B.transpose(1, 2)), {}), ((A, B), dict(scaling=i)), ((A, B), dict(ranks=f)),
                  ((A, B), dict(scaling=f[:1])), ((A.transpose(1, 2).contiguous().transpose(1, 2), B), {}), ((A, B.cpu()), {}),
                  ((A, B), dict(ranks=i.cpu()))):
        with pytest.raises(ValueError):
            sk.Adapters(*a, **kw)
    for a in ((torch.zeros((2, 4, 16), **half), torch.zeros((2, 5, 4), **half)), (torch.zeros((2, 264, 16), **half),
              torch.zeros((2, 5, 264), **half)), (torch.zeros((2, 8, 12), **half), B)):
        with pytest.raises(sk.SkinnyError):
            sk.Adapters(*a)
    pool, ids = sk.Adapters(A, B), torch.zeros(3, dtype=torch.int32, device="cuda")
    base = torch.zeros((3, 5), **half)
    for a, kw in (((x[:, :8], pool, ids), {}), ((x, pool, ids[:2]), {}), ((x, pool, ids.float()), {}), ((x, pool, ids.cpu()), {}),
                  ((x, pool, ids, base[:2]), {}), ((x, pool, ids), dict(out=base[:, :4])), ((x, pool, ids, base.cpu()), {})):
        with pytest.raises(ValueError):
            sk.add_adapters(*a, **kw)
    for a in ((x.half(), pool, ids), (x, (A, B), ids)):
        with pytest.raises(TypeError):
            sk.add_adapters(*a)
    wide = torch.zeros((4, 5), **half)
    for a, kw in (((x, pool, ids, base.half()), {}), ((x, pool, ids), dict(out_dtype=torch.float16)),
                  ((x, pool, ids, wide[:3]), dict(out=wide[1:])), ((torch.zeros((3, 20), **half)[:, :16], pool, ids), {}),
                  ((torch.zeros((3, 24), **half)[:, 4:20], pool, ids), {})):
        with pytest.raises(sk.SkinnyError):
            sk.add_adapters(*a, **kw)
