"""GPU parity of the logit adjustments against 64 bits (requests_ref.adjust, which
derives the bounds of the fp32 steps); what no rule touches is equal bit for bit."""
import numpy as np
import pytest

import requests_ref as Q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sk = pytest.importorskip("row_gemv_decode_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ARRAYS = ("history", "lengths", "prompt_lengths", "repetition", "frequency", "presence", "bias_ids", "bias_values", "mask",
          "mask_rows")


def pack(allowed):
    """[rows][vocab] truth values -> int32 [rows][words]."""
    rows, V = allowed.shape
    bits = np.zeros((rows, (V + 31) // 32 * 32), np.uint8)
    bits[:, :V] = allowed
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def rules_of(m, V, seed, history=0, biases=0, masks=False, t64=False, double=True):
    rng = np.random.default_rng(seed)
    tok = np.int64 if t64 else np.int32
    a = {}
    if history:
        a["history"] = np.minimum((rng.random((m, history)) ** 4 * V).astype(tok), V - 1)
        a["history"][rng.random((m, history)) < 0.02] = -1
        a["history"][rng.random((m, history)) < 0.02] = V
        a["lengths"] = rng.integers(0, history + 1, m).astype(np.int32)
        a["lengths"][0] = history
        a["prompt_lengths"] = (a["lengths"] * rng.random(m)).astype(np.int32)
        a["repetition"] = rng.uniform(0.8, 1.5, m).astype(np.float32)
        a["frequency"] = rng.uniform(-0.5, 0.5, m).astype(np.float32)
        a["presence"] = rng.uniform(-1, 1, m).astype(np.float32)
    if biases:
        a["bias_ids"] = rng.integers(0, V if not double else max(1, V // 3), (m, biases)).astype(tok)
        if not double:
            for i in range(m):
                a["bias_ids"][i] = rng.permutation(V)[:biases]
        a["bias_ids"][rng.random((m, biases)) < 0.1] = -1
        a["bias_ids"][:, -1] = V - 1
        a["bias_values"] = rng.uniform(-8, 8, (m, biases)).astype(np.float32)
    if masks:
        share = np.array([0.0, 0.004, 0.5, 0.95, 1.0])[np.arange(m) % 5, None]
        a["mask"] = pack(rng.random((m, V)) < share)
        a["mask_rows"] = rng.permutation(m).astype(np.int32)
        a["mask_rows"][rng.random(m) < 0.3] = -1
    return a


def logits_of(m, V, kind, seed):
    x = np.random.default_rng(seed).normal(0, 4, (m, V))
    x[:, :: 7] = np.abs(x[:, :: 7])
    if V > 20:
        x[:, 11] = -np.inf
        x[:, 3] = 0.0
    t = torch.from_numpy(x).to(DT[kind])
    return t.cuda(), t.double().numpy()


def device(a):
    return {k: torch.from_numpy(v).cuda() for k, v in a.items()}


def compare(got, x, a, ok):
    ref, bound, touched = Q.adjust(x, *(a.get(k) for k in ARRAYS), ok)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isneginf(g), np.isneginf(ref))
    fin = np.isfinite(ref)
    assert np.all(np.abs(g[fin] - ref[fin]) <= bound[fin])
    assert np.array_equal(g[~touched], x[~touched])


def check(m, V, kind="f32", ok=None, seed=0, **kw):
    print(f"adjust m={m} V={V} {kind} -> {ok} {kw}", flush=True)
    a = rules_of(m, V, seed + V, **kw)
    X = logits_of(m, V, kind, seed + 1)
    rules = sk.LogitRules(m, V, **device(a))
    out = sk.adjust_logits(X[0], rules, out_dtype=DT[ok] if ok else None)
    torch.cuda.synchronize()
    compare(out, X[1], a, ok or kind)
    if ok is None or ok == kind:
        y = X[0].clone()
        assert sk.adjust_logits(y, rules, out=y) is y
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.uint8), out.view(torch.uint8))
    return a, X, out


@pytest.mark.parametrize("kind,ok", [("f32", None), ("bf16", "f32"), ("f16", None), ("bf16", None), ("f16", "f32")])
@pytest.mark.parametrize("V", [1, 2, 5, 8, 31, 32, 33, 64, 100, 1000, 2047, 2048, 2049, 4099, 33000, 50021])
def test_adjust_lengths(V, kind, ok):
    """From one logit on, at and past a mask's word, a vector, a segment."""
    check(3, V, kind, ok, history=17, biases=min(V, 4), masks=True, t64=V % 2 == 1)
    check(5, V, kind, ok, masks=True)
    check(2, V, kind, ok, history=40)


@pytest.mark.parametrize("m", [1, 2, 16, 130, 700])
def test_adjust_row_counts(m):
    check(m, 9001, "bf16", "f32", history=100, biases=8, masks=True)


@pytest.mark.parametrize("history", [1, 3, 4, 5, 255, 1024, 1025, 5000, 16383, 16384, 20000, 70000])
def test_adjust_history_lengths(history):
    """Past the lengths that a thread, a workgroup and a 16-bit entry take at once."""
    check(2, 5003, "f32", history=history, t64=history % 2 == 1)


@pytest.mark.parametrize("history", [4096, 4097, 16383, 16400])
@pytest.mark.parametrize("biases", [0, 1300])
def test_adjust_long_histories_of_many_rows(history, biases):
    """The longest segments and the largest tables, without and with biases."""
    m, V = 600, 33000
    a = rules_of(m, V, 5, history=history, biases=biases)
    x = torch.randn((m, V), generator=torch.Generator().manual_seed(1))
    got = sk.adjust_logits(x.cuda(), sk.LogitRules(m, V, **device(a)))
    torch.cuda.synchronize()
    for i in (0, 1, 299, 599):
        one = {k: v[i:i + 1] for k, v in a.items()}
        compare(got[i:i + 1], x[i:i + 1].double().numpy(), one, "f32")


@pytest.mark.parametrize("vocab,history", [(40000, 16383), (17, 16383), (40000, 40000), (1, 20000)])
def test_adjust_one_token_over_and_over(vocab, history):
    """A count as long as the history."""
    a = rules_of(2, vocab, 3, history=history)
    a["history"][:] = vocab - 1
    a["prompt_lengths"][:] = [0, 5]
    a["lengths"][:] = history
    X = logits_of(2, vocab, "f32", 4)
    compare(sk.adjust_logits(X[0], sk.LogitRules(2, vocab, **device(a))), X[1], a, "f32")


@pytest.mark.parametrize("biases", [1, 7, 15, 16, 17, 255, 256, 300, 1000, 1023, 1024, 1025, 5000])
@pytest.mark.parametrize("double", [False, True])
def test_adjust_bias_lists(biases, double):
    """Lists longer than a workgroup; the same token several times."""
    check(3, 9973, "bf16", "f32", biases=biases, double=double)
    check(2, 9973, "f32", biases=biases, double=double, history=300, masks=True)


def test_adjust_biases_are_added_in_the_lists_order():
    """1e8 + 1 - 1e8 is 0 in fp32 in this order, and 1 in another."""
    V = 500
    a = {"bias_ids": np.array([[7, 7, 3, 7], [7, 7, 3, 7]], np.int32),
         "bias_values": np.array([[1e8, 1.0, 2.0, -1e8], [1e8, -1e8, 2.0, 1.0]], np.float32)}
    x = torch.zeros((2, V), device="cuda")
    out = sk.adjust_logits(x, sk.LogitRules(2, V, **device(a))).cpu()
    assert out[0, 7] == 0.0 and out[1, 7] == 1.0 and out[0, 3] == 2.0


def far_ids(kind, near, V):
    """Ids outside 0 .. V - 1 that have the low 32 bits of a token's place in some segment,
    or that leave their type's range when a segment's first token is taken from them."""
    if kind == np.int32:
        return [-(1 << 31), (1 << 31) - 1, -1, V, -V, -(1 << 31) + near]
    high = [h << s for s in (32, 33, 40, 62) for h in (1, -1)] + [-(1 << 63)]
    return [h + t for h in high for t in (0, near)] + [(1 << 63) - 1, -1, V, (1 << 31) + near, -(1 << 31) + near]


@pytest.mark.parametrize("m,V", [(2, 500), (2, 9973), (40, 40000)])
@pytest.mark.parametrize("biases", [60, 1100])
@pytest.mark.parametrize("kind", [np.int32, np.int64])
def test_adjust_ids_far_outside_the_vocabulary(kind, biases, m, V):
    """Any id outside the vocabulary fills a list up and does not count in a history,
    however far it lies: tokens 0 and `near` listed beside them, once and (row 1) twice,
    before and behind them, in lists that LDS holds and longer ones."""
    for near in (7, V - 3):
        far = far_ids(kind, near, V)
        a = {"bias_ids": np.resize(np.array(far, kind), (m, biases)),
             "bias_values": np.random.default_rng(V).uniform(1, 8, (m, biases)).astype(np.float32)}
        a["bias_ids"][:, 3], a["bias_ids"][::3, biases - 1] = near, 0
        a["bias_ids"][1, biases // 2], a["bias_ids"][1, biases - 2] = near, 0
        a["bias_ids"][m - 1, 0], a["bias_ids"][m - 1, 3] = near, -(1 << 31)
        for history in (False, True):
            if history:
                a["history"] = np.resize(np.array(far + [near], kind), (m, 150))
                a["frequency"] = np.full(m, 0.25, np.float32)
            X = logits_of(m, V, "f32", 5)
            rules = sk.LogitRules(m, V, **device(a))
            compare(sk.adjust_logits(X[0], rules), X[1], a, "f32")
            y = X[0].clone()
            compare(sk.adjust_logits(y, rules, out=y), X[1], a, "f32")


def test_adjust_optional_rules():
    """Every rule by itself; none at all gives the logits."""
    m, V = 4, 3001
    full = rules_of(m, V, 9, history=60, biases=5, masks=True)
    X = logits_of(m, V, "bf16", 10)
    for keys in ((), ("history",), ("history", "lengths"), ("history", "prompt_lengths"), ("history", "repetition"),
                 ("history", "lengths", "frequency"), ("history", "presence"), ("bias_ids", "bias_values"), ("mask",),
                 ("mask", "mask_rows"), ("history", "repetition", "mask"), ("bias_ids", "bias_values", "mask")):
        a = {k: full[k] for k in keys}
        rules = sk.LogitRules(m, V, **device(a))
        for ok in ("bf16", "f32"):
            compare(sk.adjust_logits(X[0], rules, out_dtype=DT[ok]), X[1], a, ok)
        y = X[0].clone()
        compare(sk.adjust_logits(y, rules, out=y), X[1], a, "bf16")


def test_adjust_lengths_out_of_range_and_masks_shared():
    m, V = 6, 700
    a = rules_of(m, V, 11, history=30, masks=True)
    a["lengths"][:] = [-5, 0, 31, 1 << 30, 7, 30]
    a["prompt_lengths"][:] = [3, 9, -1, 1 << 30, 100, 30]
    a["mask"] = a["mask"][:2]
    a["mask_rows"][:] = [0, 1, 1, 2, -7, 0]
    X = logits_of(m, V, "f32", 12)
    compare(sk.adjust_logits(X[0], sk.LogitRules(m, V, **device(a))), X[1], a, "f32")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_adjust_empty_masks_and_non_finite_logits(kind):
    """A row whose mask leaves nothing; NaN, infinities and the lowest value."""
    V = 4100
    x = torch.zeros((4, V), dtype=DT[kind], device="cuda")
    x[:, 10], x[:, 11], x[:, 12], x[:, 13] = float("nan"), float("inf"), -float("inf"), torch.finfo(DT[kind]).min
    allowed = np.ones((4, V), bool)
    allowed[0] = False
    allowed[1, 10:14] = False
    mask = torch.from_numpy(pack(allowed)).cuda()
    hist = torch.tensor([[10, 11, 12, 13, 20]] * 4, dtype=torch.int32, device="cuda")
    rules = sk.LogitRules(4, V, history=hist, repetition=torch.full((4,), 2.0, device="cuda"),
                          presence=torch.ones(4, device="cuda"), mask=mask)
    for out in (sk.adjust_logits(x, rules), sk.adjust_logits(x.clone(), rules, out_dtype=torch.float32)):
        o = out.float().cpu()
        assert bool(torch.isneginf(o[0]).all()) and bool(torch.isneginf(o[1, 10:14]).all())
        for r in (2, 3):
            assert o[r, 10].isnan() and o[r, 11] == float("inf") and torch.isneginf(o[r, 12]) and o[r, 20] == -1.0
            # the lowest value times two and less one: past every type but f16 in fp32
            assert o[r, 13] == (-131009.0 if kind == "f16" and out.dtype == torch.float32 else -float("inf"))


@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("kind,ok", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
def test_adjust_alignment_and_strides(offset, kind, ok):
    """Rows that start anywhere, padded histories and masks; what lies beside the
    rows stays."""
    m, V = 4, 4133
    a = rules_of(m, V, 20, history=50, biases=3, masks=True)
    X = logits_of(m, V, kind, 21)

    def strided(shape, pad, dtype, fill):
        big = torch.full((shape[0] * (shape[1] + pad) + 64,), fill, device="cuda").to(dtype)
        return big, big[offset:offset + shape[0] * (shape[1] + pad)].view(shape[0], -1)[:, :shape[1]]

    x = strided((m, V), 7, DT[kind], 77.0)[1].copy_(X[0])
    d = device(a)
    for key, pad in (("history", 3), ("mask", 2)):
        d[key] = strided(tuple(d[key].shape), pad, torch.int32, 0)[1].copy_(d[key])
    big, out = strided((m, V), 9, DT[ok], 77.0)
    rules = sk.LogitRules(m, V, **d)
    sk.adjust_logits(x, rules, out=out)
    torch.cuda.synchronize()
    compare(out, X[1], a, ok)
    rest = torch.ones_like(big, dtype=torch.bool)
    rest[offset:offset + m * (V + 9)].view(m, -1)[:, :V] = False
    assert bool((big[rest] == 77.0).all())
    sk.adjust_logits(x, rules, out=x) if kind == ok else None
    assert kind != ok or torch.equal(x, out)


def test_adjust_expanded_rows_are_copied():
    V = 900
    a = rules_of(5, V, 30, history=20)
    X = logits_of(1, V, "f32", 31)
    out = sk.adjust_logits(X[0].expand(5, V), sk.LogitRules(5, V, **device(a)))
    compare(out, np.repeat(X[1], 5, axis=0), a, "f32")


def test_adjust_reads_the_rules_at_every_call():
    """Streams and graphs: the rules' tensors are filled in place from step to step,
    and every replay equals the eager call."""
    m, V = 7, 20011
    a = rules_of(m, V, 40, history=64, biases=6, masks=True)
    X = logits_of(m, V, "bf16", 41)
    d = device(a)
    rules = sk.LogitRules(m, V, **d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = sk.adjust_logits(X[0], rules, out_dtype=torch.float32, stream=s)
    s.synchronize()
    compare(out, X[1], a, "f32")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = sk.adjust_logits(X[0], rules, out_dtype=torch.float32)
    for k in range(3):
        for key in ARRAYS:
            b = rules_of(m, V, 50 + k, history=64, biases=6, masks=True)
            d[key].copy_(torch.from_numpy(b[key]))
        g.replay()
        eager = sk.adjust_logits(X[0], rules, out_dtype=torch.float32)
        torch.cuda.synchronize()
        compare(cap, X[1], b, "f32")
        assert torch.equal(cap, eager)


def test_adjust_results_are_the_same_every_time():
    """Counts by atomics, in whatever order: the same bits."""
    m, V = 40, 30011
    rules = sk.LogitRules(m, V, **device(rules_of(m, V, 60, history=3001, biases=200, masks=True)))
    x = logits_of(m, V, "f32", 61)[0]
    want = sk.adjust_logits(x, rules)
    assert all(torch.equal(sk.adjust_logits(x, rules), want) for _ in range(5))


def test_adjust_large_offsets():
    """Rows whose places pass 2^31 elements."""
    V, ld = 3001, 1 << 28
    big = torch.empty(9 * ld + V, dtype=torch.float16, device="cuda")
    x = big[:9 * ld].view(9, ld)[:, :V]
    a = rules_of(9, V, 70, history=30, masks=True)
    X = logits_of(9, V, "f16", 71)
    x.copy_(X[0])
    compare(sk.adjust_logits(x, sk.LogitRules(9, V, **device(a)), out=x), X[1], a, "f16")
    del big, x
    torch.cuda.empty_cache()


def test_adjust_refusals():
    V = 100
    i32 = dict(dtype=torch.int32, device="cuda")
    h, f = torch.zeros((2, 5), **i32), torch.ones(2, device="cuda")
    for kw in (dict(lengths=torch.zeros(2, **i32)), dict(presence=f), dict(bias_ids=h), dict(mask_rows=torch.zeros(2, **i32)),
               dict(history=h.float()), dict(history=h[:1]), dict(history=h, repetition=f[:1]), dict(history=h, lengths=f),
               dict(history=h, bias_ids=h.long(), bias_values=h.float()), dict(bias_ids=h, bias_values=h.double()),
               dict(mask=torch.zeros((2, 3), **i32)), dict(mask=torch.zeros((1, 4), **i32)), dict(history=h, frequency=f.cpu()),
               dict(history=torch.zeros((2, 1), **i32).expand(2, 5)), dict(bias_ids=h.t(), bias_values=h.float().t())):
        with pytest.raises(ValueError):
            sk.LogitRules(2, V, **kw)
    rules = sk.LogitRules(2, V, history=h)
    x = torch.zeros((2, V), device="cuda")
    for bad in (x[:1], x[:, :50]):
        with pytest.raises(ValueError):
            sk.adjust_logits(bad, rules)
    with pytest.raises(ValueError):
        sk.adjust_logits(x, rules, out=x[:, :50])
    with pytest.raises(ValueError):
        sk.adjust_logits(x.cpu(), rules)
    with pytest.raises(TypeError):
        sk.adjust_logits(x.double(), rules)
    for kw in (dict(out_dtype=torch.float16), dict(out=x.half())):
        with pytest.raises(sk.SkinnyError):
            sk.adjust_logits(x, rules, **kw)
    big = torch.zeros((3, V), device="cuda")
    with pytest.raises(sk.SkinnyError):  # half over the logits
        sk.adjust_logits(big[:2], rules, out=big[1:])
