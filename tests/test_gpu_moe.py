"""GPU parity of the whole MoE layer against the layer in 64 bits
(window_ref.moe, which also carries the error bound of fp32 sums through the
layer: the additions of each sum times 2^-24 of the magnitudes added, the
activation's slope, the softmax's dependence on the logits, the output type's
rounding)."""
import threading

import numpy as np
import pytest

import window_ref as R
import workloads as WL
from conftest import to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sk = pytest.importorskip("row_gemv_decode_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Case:
    def __init__(self, m, experts, topk, d, inter, shared=0, group=0, zeros=False, kind="bf16", out="f32", renorm=True,
                 seed=0):
        self.__dict__.update(locals())

        def weight(shape, sd, s):
            if group == 0:
                return WL.gen_matrix(shape, kind, ("normal", sd), s)
            return R.gen_w4(shape, group, kind, zeros, s, sd)

        sd1, sd2 = 1.4 / np.sqrt(d), 1.4 / np.sqrt(inter)
        self.x = WL.gen_matrix((m, d), kind, ("normal", 1.0), seed)
        self.router = WL.gen_matrix((experts, d), kind, ("normal", sd1), seed + 1)
        self.w13 = weight((experts, 2 * inter, d), sd1, seed + 2)
        self.w2 = weight((experts, d, inter), sd2, seed + 3)
        self.sh = None
        if shared:
            self.sh = (weight((2 * shared, d), sd1, seed + 4), weight((d, shared), sd2, seed + 5),
                       WL.gen_matrix((d,), kind, ("normal", sd1), seed + 6))

    def dev(self, w):
        if isinstance(w, tuple):
            return sk.W4(to_dev(w[0], "u8"), to_dev(w[1], self.kind), None if w[2] is None else to_dev(w[2], "u8"))
        return to_dev(w, self.kind)

    def layer(self, max_m=16):
        kw = {}
        if self.sh is not None:
            kw = {"shared13": self.dev(self.sh[0]), "shared2": self.dev(self.sh[1]), "shared_gate": self.dev(self.sh[2])}
        return sk.MoELayer(self.dev(self.router), self.dev(self.w13), self.dev(self.w2), topk=self.topk,
                           renorm=self.renorm, out_dtype=DT[self.out], max_m=max_m, **kw)

    def check(self):
        print(f"moe m={self.m} E={self.experts} top-{self.topk} d={self.d} inter={self.inter} shared={self.shared} "
              f"group={self.group} zeros={self.zeros} {self.kind} -> {self.out} renorm={self.renorm}", flush=True)
        layer, x = self.layer(), self.dev(self.x)
        idx = torch.full((self.m, self.topk), -1, dtype=torch.int32, device="cuda")
        wts = torch.zeros((self.m, self.topk), device="cuda")
        got = layer(x, topk_idx=idx, topk_weight=wts)
        torch.cuda.synchronize()
        ref, bound, ids, weights = R.moe(self.x, self.router, self.w13, self.w2, self.topk, self.renorm, self.sh, self.kind,
                                         self.out)
        assert np.array_equal(idx.cpu().numpy(), ids)
        assert np.allclose(wts.double().cpu().numpy(), weights, rtol=1e-4, atol=0)
        assert got.dtype == DT[self.out]
        off = np.abs(got.double().cpu().numpy() - ref)
        assert np.all(off <= bound)
        assert torch.equal(layer(x), got)
        return layer, x, got


@pytest.mark.parametrize("group,zeros", [(0, False), (32, True), (64, False), (128, True)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 5, 16])
def test_moe_parity(m, kind, group, zeros):
    Case(m, 24, 4, 384, 256, shared=128, group=group, zeros=zeros, kind=kind, seed=8000 + m).check()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_moe_output_types_and_plain_softmax(kind):
    for out in ("f32", "f16", "bf16"):
        Case(3, 40, 6, 256, 128, kind=kind, out=out, renorm=False, seed=8100).check()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [0, 128])
def test_moe_16_bit_output_is_the_fp32_output_rounded(group, kind):
    """The inner values lose no bit under a 16-bit output that they keep under
    fp32: the outputs are those of the fp32 layer, rounded once."""
    kw = dict(shared=128, group=group, zeros=group > 0, kind=kind, seed=8150)
    _, _, wide = Case(16, 24, 4, 768, 256, out="f32", **kw).check()
    for out in ("bf16", "f16"):
        _, _, got = Case(16, 24, 4, 768, 256, out=out, **kw).check()
        assert torch.equal(got, wide.to(DT[out]))


@pytest.mark.parametrize("experts,topk", [(1, 1), (2, 2), (32, 32), (63, 3), (64, 10), (65, 10), (300, 7), (1024, 32)])
def test_moe_expert_counts(experts, topk):
    Case(4, experts, topk, 128, 64, shared=32, seed=8200 + experts).check()


@pytest.mark.parametrize("d,inter,shared", [(32, 32, 0), (96, 160, 64), (160, 96, 224), (2080, 32, 32), (64, 1120, 0)])
def test_moe_odd_lengths(d, inter, shared):
    """Lengths below, at and past a unit of 128 and with a partial last unit."""
    for group in (0, 32):
        Case(6, 9, 3, d, inter, shared=shared, group=group, zeros=True, seed=8300 + d).check()


def test_moe_router_split_across_workgroups():
    """A d past 8192: the router's GEMV needs its own part of the workspace."""
    Case(2, 6, 2, 8320, 32, kind="bf16", seed=8400).check()


def test_moe_equal_tokens_and_equal_experts():
    """All tokens alike: every expert serves all of them; equal router rows
    rank by the lower expert."""
    c = Case(16, 12, 5, 256, 96, shared=32, seed=8500)
    c.x[:] = c.x[0]
    c.router[7] = c.router[2]
    c.router[11] = c.router[2]
    layer, x, got = c.check()
    assert all(torch.equal(got[i], got[0]) for i in range(16))


@pytest.mark.parametrize("group,kind", [(0, "bf16"), (0, "f16"), (32, "bf16"), (128, "f16")])
def test_moe_rows_do_not_depend_on_the_window(group, kind):
    """A token's output is the same bits at every m and beside any others."""
    c = Case(16, 40, 6, 640, 896, shared=256, group=group, zeros=True, kind=kind, seed=8600)
    layer, x, got = c.check()
    for m in (1, 2, 3, 9):
        assert torch.equal(layer(x[:m].contiguous()), got[:m])
    perm = torch.randperm(16, generator=torch.Generator().manual_seed(1)).cuda()
    assert torch.equal(layer(x[perm].contiguous()), got[perm])
    small = c.layer(max_m=4)
    assert torch.equal(small(x[12:].contiguous()), got[12:])


def test_moe_window_after_window():
    """A short window after a long one with other experts: nothing of the
    earlier window's lists or inner values is left over."""
    a = Case(16, 64, 8, 256, 128, shared=64, seed=8700)
    layer = a.layer()
    x = a.dev(a.x)
    alone = [a.layer()(x[i:i + 1].contiguous()) for i in range(16)]
    for _ in range(3):
        layer(x)
        for i in (3, 15, 0):
            assert torch.equal(layer(x[i:i + 1].contiguous()), alone[i])


def test_moe_random_shapes():
    rng = np.random.default_rng(8800)
    for i in range(16):
        group = int(rng.choice([0, 32, 64, 128]))
        unit = max(32, group)
        experts = int(rng.integers(1, 80))
        inter = unit * int(rng.integers(1, 6))
        Case(int(rng.integers(1, 17)), experts, int(rng.integers(1, min(experts, 12) + 1)), unit * int(rng.integers(1, 6)), inter,
             shared=int(rng.choice([0, unit, 2 * unit])), group=group, zeros=bool(rng.integers(2)),
             kind=str(rng.choice(["bf16", "f16"])), out=str(rng.choice(["f32", "f16", "bf16"])),
             renorm=bool(rng.integers(2)), seed=8801 + 10 * i).check()


def test_moe_on_other_streams():
    c = Case(5, 20, 4, 256, 128, shared=32, seed=8900)
    layer, x, got = c.check()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:  # in flight together: each stream has its own workspace
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([layer(x) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, got) for os in outs for o in os)


def test_moe_graph_replay():
    c = Case(7, 20, 4, 256, 128, shared=64, group=64, seed=9000)
    layer, x, got = c.check()
    out = torch.empty_like(got)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(x, out=out)  # allocates the stream's workspace before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer(x, out=out)
    for i in range(4):
        out.zero_()
        eager = layer(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(eager, got)


def test_moe_captured_before_a_run():
    """A capture on a stream that the layer has not run on: the graph carries a
    workspace of its own, and eager runs on that stream get theirs."""
    c = Case(3, 20, 4, 256, 128, shared=64, group=64, seed=9050)
    layer, x, got = c.check()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = layer(x)
    for _ in range(3):
        eager = layer(x, stream=s)
        s.synchronize()
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(eager, got)


def test_moe_refusals():
    c = Case(2, 8, 2, 128, 64, shared=32, seed=9100)
    router, w13, w2 = c.dev(c.router), c.dev(c.w13), c.dev(c.w2)
    layer, x, _ = c.check()
    with pytest.raises(ValueError):
        layer(x[:, :64])
    with pytest.raises(ValueError):
        layer(x.half())
    with pytest.raises(ValueError):
        layer(x.t().contiguous().t())
    with pytest.raises(ValueError):
        layer(x.cpu())
    with pytest.raises(sk.SkinnyError):
        layer(c.dev(WL.gen_matrix((17, 128), "bf16", ("normal", 1.0), 1)))
    with pytest.raises(ValueError):
        layer(x, out=torch.empty((2, 128), device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        layer(x, topk_idx=torch.empty((2, 2), device="cuda", dtype=torch.int64))
    with pytest.raises(TypeError):
        sk.MoELayer(router, w13.half(), w2, topk=2)
    with pytest.raises(ValueError):
        sk.MoELayer(router, w13, w2[:, :, :32].contiguous(), topk=2)
    with pytest.raises(ValueError):
        sk.MoELayer(router, w13, w2, topk=2, shared13=c.dev(c.sh[0]))
    with pytest.raises(sk.SkinnyError):
        sk.MoELayer(router, w13, w2, topk=9)
    with pytest.raises(sk.SkinnyError):
        sk.MoELayer(router, w13, w2, topk=2, max_m=17)


@pytest.mark.parametrize("d", [256, 8320])
def test_moe_graph_beside_eager_runs_on_its_stream(d):
    """A graph captured on a stream that the layer has run on, replayed on
    another stream while the first one runs the layer on other tokens (with d
    past 8192 the router's arrival counters are part of the workspace)."""
    c = Case(6, 20, 4, d, 64, shared=32, seed=9200)
    layer, x, got = c.check()
    y = x.flip(0).contiguous()
    want = layer(y)
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    layer(y, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = layer(x)
    for _ in range(4):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            g.replay()
        eager = [layer(y, stream=s) for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(out, got) and all(torch.equal(e, want) for e in eager)


def test_moe_from_several_threads():
    """Threads that call one layer on one stream get their own tokens' outputs."""
    c = Case(16, 24, 4, 256, 96, shared=32, seed=9300)
    layer, x, _ = c.check()
    xs = [x[i:i + 3].contiguous() for i in range(8)]
    want = [layer(v) for v in xs]
    got = [None] * 8

    def work(i):
        got[i] = [layer(xs[i]) for _ in range(40)]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for g, w in zip(got, want) for o in g)


@pytest.mark.parametrize("kind,group", [("f16", 0), ("f16", 32), ("f16", 128), ("bf16", 0), ("bf16", 64)])
def test_moe_inner_values_of_every_size(kind, group):
    """Up rows times a power of two: the inner values and the outputs scale
    with them, from about 2^-17 (k = -14) to past f16's 65504 (k = 17).  The
    weights are small integers times a power of two, which every k leaves exact.
    The outputs then differ by the sums' rounding alone: over the inner length
    of 128 at most 160 additions of 2^-24 of the magnitudes, which are less than
    16 times the largest output: 2^-12.6.  That is worst case; roundings of
    either sign give its square root's share, and 2^-16 is asserted."""
    rng = np.random.default_rng(9400)
    E, d, n, topk = 6, 256, 128, 3

    def grid(*shape):
        return rng.integers(-7, 8, size=shape) * 2.0 ** -7

    def weight(v, k):  # v * 2^k
        if group == 0:
            return to_dev(WL.to_bits(v * 2.0 ** k, kind), kind)
        q = (v * 2.0 ** 7 + 8).astype(np.uint8)
        codes = (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)
        shape = (*v.shape[:-1], v.shape[-1] // group)
        return sk.W4(to_dev(codes, "u8"), to_dev(WL.to_bits(np.broadcast_to(2.0 ** (k - 7.0), shape), kind), kind))

    def stack(rows, k):  # gate rows as they are, up rows times 2^k
        gate, up = rows[..., :n, :], rows[..., n:, :]
        a, b = weight(gate, 0), weight(up, k)
        if group == 0:
            return torch.cat((a, b), dim=-2)
        return sk.W4(torch.cat((a.codes, b.codes), dim=-2), torch.cat((a.scales, b.scales), dim=-2))

    x = to_dev(WL.gen_matrix((5, d), kind, ("normal", 1.0), 9401), kind)
    router = to_dev(WL.gen_matrix((E, d), kind, ("normal", 0.06), 9402), kind)
    gate = to_dev(WL.gen_matrix((d,), kind, ("normal", 0.06), 9403), kind)
    w13, w2, s13, s2 = grid(E, 2 * n, d), grid(E, d, n), grid(2 * n, d), grid(d, n)

    def run(k):
        layer = sk.MoELayer(router, stack(w13, k), weight(w2, 0), topk=topk, renorm=False, out_dtype=torch.float32,
                            shared13=stack(s13, k), shared2=weight(s2, 0), shared_gate=gate)
        return layer(x).double()

    base = run(0)
    for k in (-14, -10, -6, -2, 5, 11, 17):
        off = (run(k) * 2.0 ** -k - base).abs().max() / base.abs().max()
        print(f"moe {kind} group={group} k={k} off {float(off):.1e}", flush=True)
        assert float(off) <= 2.0 ** -16


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 1e-2, 1e-3])
def test_moe_small_inputs(scale, kind):
    """Inputs of 1e-2 and 1e-3 (the router's weight grows as they shrink, so the
    routing stays the same) under a plain softmax and an fp32 output, in root mean
    square against 64 bits.  A sum of n terms of either sign in fp32 is off by
    about sqrt(n) * 2^-24 of its own size; 2 sqrt(d) + sqrt(inter) + 16 stands for
    gate, up, down and the rest."""
    c = Case(4, 64, 6, 768, 256, shared=128, kind=kind, out="f32", renorm=False, seed=9500)
    c.x = WL.gen_matrix((4, 768), kind, ("normal", scale), 9501)
    c.router = WL.gen_matrix((64, 768), kind, ("normal", 1.4 / np.sqrt(768) / scale), 9502)
    got = c.layer()(c.dev(c.x)).double().cpu().numpy()
    ref, _, _, _ = R.moe(c.x, c.router, c.w13, c.w2, 6, False, c.sh, kind, "f32")
    off = np.sqrt(((got - ref) ** 2).mean() / (ref ** 2).mean())
    assert off <= (2 * np.sqrt(768) + np.sqrt(256) + 16) * 2.0 ** -24


@pytest.mark.parametrize("d,inter,group", [(2592, 64, 32), (5184, 64, 64), (10496, 128, 128), (64, 5152, 32)])
def test_moe_several_spans_of_scales(d, inter, group):
    """Lengths of more than 80 groups: the up product stages its scales in spans."""
    Case(5, 6, 2, d, inter, shared=group, group=group, zeros=True, kind="f16", seed=9600 + d).check()


@pytest.mark.parametrize("group,kind,d,inter", [(32, "f16", 4096, 160), (64, "bf16", 4160, 192), (128, "f16", 4096, 384),
                                                (128, "bf16", 4224, 128)])
def test_moe_bits_do_not_depend_on_the_launch(group, kind, d, inter):
    """Windows that fill the chip, whose down product takes four column tiles per
    wave, against one-token calls, whose takes two."""
    c = Case(16, 24, 12, d, inter, shared=2 * group, group=group, zeros=True, kind=kind, seed=9700)
    layer, x, got = c.check()
    for i in (0, 7, 15):
        assert torch.equal(layer(x[i:i + 1].contiguous())[0], got[i])
    for m in (4, 5, 9):
        assert torch.equal(layer(x[:m].contiguous()), got[:m])
