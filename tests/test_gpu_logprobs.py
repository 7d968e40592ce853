"""GPU parity of the token log probabilities against 64 bits
(window_ref.logprobs, which derives the error bounds of the fp32 sums); ranks
and ids are exact."""
import numpy as np
import pytest

import window_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sk = pytest.importorskip("row_gemv_decode_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LOWEST = {"f32": -float(np.finfo(np.float32).max), "f16": -65504.0, "bf16": -float(0xFF) * 2.0 ** 120}


def store(x, kind):
    """float64 -> (device tensor, the stored values in 64 bits)."""
    t = torch.from_numpy(np.asarray(x, np.float64)).to(DT[kind])
    return t.cuda(), t.double().numpy()


def same(got, want):
    """Equal where not finite."""
    return np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])


def check(x, tokens, topk, kind, ids=True, t64=True, logits=None):
    dev, vals = store(x, kind)
    if logits is not None:  # the same values elsewhere in memory
        logits.copy_(dev)
        dev = logits
    m, V = vals.shape
    print(f"logprobs m={m} V={V} top-{topk} {kind} ld={dev.stride(0)}", flush=True)
    tok = torch.tensor(np.asarray(tokens), dtype=torch.int64 if t64 else torch.int32).cuda()
    got = sk.token_logprobs(dev, tok, topk=topk)
    torch.cuda.synchronize()
    (lp, ent, rank, oid, top), (blp, bent, btop) = R.logprobs(vals, tokens, topk)
    g = [t.cpu().numpy() for t in got]
    assert np.array_equal(g[2], rank)
    assert np.array_equal(g[3], oid)
    for a, want, bound in ((g[0], lp, blp), (g[1], ent, bent), (g[4], top, btop)):
        a = a.astype(np.float64)
        assert same(a, want)
        fin = np.isfinite(want)
        assert np.all(np.abs(a[fin] - want[fin]) <= bound[fin])
    return dev, tok, got


def normal(m, V, seed, sd=3.0):
    rng = np.random.default_rng(seed)
    return rng.normal(0.0, sd, size=(m, V)), rng.integers(0, V, size=m)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 63, 64, 65, 255, 1024, 2047, 2048, 2049, 4099, 16384, 50021])
def test_lp_lengths(V, kind):
    """From one logit on, at and past a vector, a wave, a step, a segment."""
    x, t = normal(3, V, 9200 + V)
    for topk in sorted({0, 1, min(5, V), min(32, V)}):
        check(x, t, topk, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 40, 511, 1023, 1024, 1100])
def test_lp_row_counts(m, kind):
    """Across the choices of how many workgroups a row gets."""
    x, t = normal(m, 4500, 9300 + m)
    check(x, t, 6, kind, t64=m % 2 == 0)


@pytest.mark.parametrize("m,V", [(17, 300007), (31, 270001), (1, 600011)])
def test_lp_long_rows(m, V):
    """More logits than the segments' least length times their number."""
    x, t = normal(m, V, 9290 + m)
    check(x, t, 6, "bf16")


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
def test_lp_alignment_and_strides(offset, kind):
    """Rows that start at every element of a 16-byte vector, and padded rows."""
    x, t = normal(5, 4133, 9400 + offset)
    for ld in (4133 + offset, 4133 + 17):
        big = torch.full((5 * ld + 64,), 77.0, dtype=DT[kind], device="cuda")
        view = big[offset:offset + 5 * ld].view(5, ld)[:, :4133]
        check(x, t, 8, kind, logits=view)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_lp_ties(kind):
    """Few distinct values: ids and ranks go to the lower index."""
    rng = np.random.default_rng(9500)
    for V in (40, 3000, 20011):
        x = rng.integers(0, 4, size=(4, V)).astype(np.float64)
        x[1] = 0.5
        x[2, ::2] = -0.0
        x[2, 1::2] = 0.0
        check(x, rng.integers(0, V, size=4), min(32, V), kind)
        check(x, [0, V - 1, V // 2, V - 1], min(7, V), kind)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_lp_order_of_the_logits(kind):
    """Rising and falling rows: every logit beats all before it, or none does."""
    for V in (3000, 40009):
        up = np.linspace(-30.0, 30.0, V)
        x = np.stack([up, up[::-1], np.roll(up, V // 3)])
        check(x, [0, V // 2, V - 1], 32, kind)
        check(x, [V - 1, 0, 17], 3, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_lp_masks(kind):
    """Masked logits (-inf), rows that keep fewer than topk, one or none of
    them, and rows of the type's lowest value."""
    V = 9001
    rng = np.random.default_rng(9600)
    x, t = normal(8, V, 9601)
    x[0, rng.random(V) < 0.9] = -np.inf
    x[1] = -np.inf                       # nothing left
    x[2] = -np.inf
    x[2, 4000] = -5.0                    # one left
    x[3] = -np.inf
    x[3, [17, 8000, 8999]] = [1.0, 2.0, 1.0]
    x[4] = LOWEST[kind]                  # uniform
    x[5, rng.random(V) < 0.5] = LOWEST[kind]
    x[6, 1:] = LOWEST[kind]
    x[7] = -np.inf
    x[7, 100:103] = LOWEST[kind]
    t[:] = [int(np.argmax(x[0])), 5, 4000, 8999, 8999, 3, 2, 101]
    check(x, t, 10, kind)
    t[:] = [int(np.argmin(x[0])), 0, 3999, 0, 0, 1, 0, 99]
    check(x, t, 1, kind)


def test_lp_large_and_spread_values():
    x, t = normal(4, 6000, 9700)
    x[0] *= 1e3
    x[1] += 1e4
    x[2] *= 1e-3
    x[3] = np.where(np.arange(6000) % 2 == 0, 1e30, -1e30)
    check(x, t, 10, "f32")


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_lp_not_finite(kind):
    """A NaN or +inf in a row gives NaN for that row alone; ids stay in the row."""
    x, t = normal(4, 5003, 9800)
    x[1, 4321] = np.nan
    x[2, 77] = np.inf
    dev, _ = store(x, kind)
    got = sk.token_logprobs(dev, torch.from_numpy(t).cuda(), topk=9)
    clean = sk.token_logprobs(dev[[0, 3]].contiguous(), torch.from_numpy(t[[0, 3]]).cuda(), topk=9)
    torch.cuda.synchronize()
    for g, c in zip(got, clean):
        assert torch.equal(g[[0, 3]], c)
    for r in (1, 2):
        assert bool(torch.isnan(got.logprob[r])) and bool(torch.isnan(got.entropy[r]))
        assert bool(torch.isnan(got.top_logprobs[r]).all())
        assert bool(((got.top_ids[r] >= -1) & (got.top_ids[r] < 5003)).all())


def test_lp_tokens_outside_the_row():
    x, t = normal(5, 3000, 9900)
    bad = np.array([-1, 3000, 2 ** 40, -2 ** 62, 7])
    dev, _, got = check(x, bad, 4, "f32")
    assert bool(torch.isnan(got.logprob[:4]).all()) and not bool(torch.isnan(got.logprob[4]))
    check(x, [-1, 3000, 2 ** 31 - 1, -2 ** 31, 7], 4, "bf16", t64=False)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_lp_rows_do_not_depend_on_the_window(kind):
    x, t = normal(16, 70001, 10000)
    dev, tok, full = check(x, t, 12, kind)
    for m in (1, 2, 7):
        part = sk.token_logprobs(dev[:m], tok[:m], topk=12)
        assert all(torch.equal(a, b[:m]) for a, b in zip(part, full))
    one = sk.token_logprobs(dev[13:14], tok[13:14], topk=12)
    assert all(torch.equal(a[0], b[13]) for a, b in zip(one, full))


def test_lp_runs_share_a_workspace():
    """Runs of several sizes after one another on one stream, and several
    streams at once."""
    cases = [normal(m, V, 10100 + m) for m, V in ((16, 30000), (3, 9000), (400, 5000), (1, 100000))]
    devs = [(store(x, "f32")[0], torch.from_numpy(t).cuda()) for x, t in cases]
    want = [sk.token_logprobs(d, t, topk=5) for d, t in devs]
    for _ in range(3):
        for (d, t), w in zip(devs, want):
            assert all(torch.equal(a, b) for a, b in zip(sk.token_logprobs(d, t, topk=5), w))
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got += [(sk.token_logprobs(d, t, topk=5), w) for d, t, w in ((d, t, w) for (d, t), w in zip(devs, want))]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in got for a, b in zip(g, w))


def test_lp_graph_replay():
    x, t = normal(8, 40000, 10200)
    dev, tok, want = check(x, t, 10, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sk.token_logprobs(dev, tok, topk=10)  # the stream's workspace, before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = sk.token_logprobs(dev, tok, topk=10)
    for _ in range(4):
        for o in out:
            o.zero_()
        eager = sk.token_logprobs(dev, tok, topk=10)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(out, want, eager))


def test_lp_captured_before_a_run():
    """A capture on a stream without a workspace: the graph carries its own, and
    eager runs on that stream get theirs."""
    x, t = normal(2, 50000, 10300)
    dev, tok, want = check(x, t, 7, "f32")
    s = torch.cuda.Stream()
    sk._logprob_ws.pop((dev.get_device(), s.cuda_stream), None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = sk.token_logprobs(dev, tok, topk=7)
    for _ in range(3):
        eager = sk.token_logprobs(dev, tok, topk=7, stream=s)
        s.synchronize()
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(out, want, eager))


def test_lp_refusals():
    x = torch.zeros((2, 100), device="cuda")
    t = torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in (t[:1], t.float(), t.view(1, 2)):
        with pytest.raises(ValueError):
            sk.token_logprobs(x, bad)
    with pytest.raises(ValueError):
        sk.token_logprobs(x, t.cpu())
    with pytest.raises(ValueError):
        sk.token_logprobs(x.t(), torch.zeros(100, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        sk.token_logprobs(x.double(), t)
    for topk in (-1, 33):
        with pytest.raises(sk.SkinnyError):
            sk.token_logprobs(x, t, topk=topk)
    with pytest.raises(sk.SkinnyError):
        sk.token_logprobs(x[:, :4], t, topk=5)
    with pytest.raises(sk.SkinnyError):
        sk.token_logprobs(x[:, :0], t)


@pytest.mark.parametrize("V", [40, 5003, 70001])
def test_lp_several_tokens_of_one_row(V):
    """A row expanded to one row per token: the results of its copies."""
    x, _ = normal(1, V, 10400)
    dev, _ = store(x, "f32")
    tok = torch.arange(16, device="cuda") * (V // 16)
    want = sk.token_logprobs(dev.repeat(16, 1), tok, topk=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [sk.token_logprobs(dev.expand(16, -1), tok, topk=3), sk.token_logprobs(dev.expand(16, -1), tok, topk=3, stream=s)]
    s.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


def test_lp_graph_outlives_the_streams_workspace():
    """A stream's workspace is replaced by a larger one after a capture on that
    stream: the graph's replays neither need the old one nor write to the
    tensors that lie there now, also beside eager calls on the stream."""
    x, t = normal(4, 60000, 10500)
    dev, tok, want = check(x, t, 4, "f32")
    big, bt = store(normal(16, 70000, 10501)[0], "f32")[0], torch.arange(16, device="cuda")
    bwant = sk.token_logprobs(big, bt, topk=32)
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    sk.token_logprobs(dev, tok, topk=4, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = sk.token_logprobs(dev, tok, topk=4)
    sk.token_logprobs(big, bt, topk=32, stream=s)
    with torch.cuda.stream(s):
        near = [torch.full((n,), 1 + n % 100, dtype=torch.uint8, device="cuda") for n in (512, 4096, 8192, 20000, 60000) * 4]
    torch.cuda.synchronize()
    for _ in range(4):
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            g.replay()
        eager = [sk.token_logprobs(big, bt, topk=32, stream=s) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for e in eager for a, b in zip(e, bwant))
        assert all(bool((n == 1 + n.numel() % 100).all()) for n in near)


def test_lp_more_rows_than_a_launch():
    """Row counts at, past and far past a launch's 2^22 (2^24 rows of four waves
    are 2^32 threads, which a grid does not hold): rows of one and of three
    logits, the results by the formula."""
    for m, V, kind in (((1 << 22) + 1, 3, "f16"), ((1 << 24) + 65, 1, "bf16"), ((1 << 23) + 3, 3, "f32")):
        print(f"logprobs m={m} V={V} {kind}", flush=True)
        g = torch.Generator(device="cuda").manual_seed(m)
        x = torch.randint(-2, 3, (m, V), device="cuda", generator=g).to(DT[kind])
        tok = torch.randint(0, V, (m,), device="cuda", generator=g, dtype=torch.int32)
        got = sk.token_logprobs(x, tok, topk=1)
        t = tok.long()[:, None]
        lp = torch.log_softmax(x.double(), dim=1)
        mine, before = x.gather(1, t), torch.arange(V, device="cuda")[None] < t
        assert torch.equal(got.rank, (1 + ((x > mine) | ((x == mine) & before)).sum(1)).int())
        assert torch.equal(got.top_ids[:, 0].long(), (x == x.amax(1, keepdim=True)).int().argmax(1))
        # at most three terms: a few roundings of values below 6
        assert float((got.logprob.double() - lp.gather(1, t)[:, 0]).abs().max()) <= 64 * 2.0 ** -24
        assert float((got.entropy.double() + (lp.exp() * lp).sum(1)).abs().max()) <= 64 * 2.0 ** -24


@pytest.mark.parametrize("m,V", [(255, 98304), (256, 98303), (256, 98304), (300, 100003), (511, 98305), (512, 98305)])
def test_lp_hundreds_of_long_rows(m, V):
    """On both sides of the steps at which a row is cut in three."""
    x, t = normal(m, V, 10600 + m)
    x[3] = -np.inf
    x[4, :] = np.linspace(-5.0, 5.0, V)
    check(x, t, 7, "bf16")
    rows = slice(0, 8)
    check(x[rows], t[rows], 20, "f16")
