"""Argument checks of the C entry points of the operators of a batch of requests
(residual and norm, adapters, logit adjustments): every refusal comes from the
host before any HIP call, so these run without a GPU."""
import ctypes
import os
import re

import pytest

from conftest import ROOT

sk = pytest.importorskip("row_gemv_decode_amd")

lib = sk.lib()


def at(i):  # made-up device addresses, far enough apart not to overlap
    return i << 34


def test_exports_every_declared_symbol():
    with open(os.path.join(ROOT, "include", "skinny_requests.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"SKINNY_API\s+[\w ]+?\**\s*(\w+)\s*\(", text)
    assert len(names) == 4 and set(names) == set(sk.REQUEST_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def norm_run(m=4, d=64, x=at(1), ldx=0, xt=sk.BF16, r=at(2), ldr=0, rt=sk.F32, w=at(3), wt=sk.BF16, eps=1e-6, ro=at(4), ldro=0,
             out=at(5), ldo=0, ot=sk.BF16, q=at(6), ldq=0, s=at(7), group=32):
    return lib.skinny_rms_norm_run(m, d, x, ldx, xt, r, ldr, rt, w, wt, eps, ro, ldro, out, ldo, ot, q, ldq, s, group, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), sk.ERR_INVALID_ARG), (dict(r=None), sk.ERR_INVALID_ARG), (dict(q=None), sk.ERR_INVALID_ARG),
    (dict(s=None), sk.ERR_INVALID_ARG), (dict(ro=None, out=None, q=None, s=None), sk.ERR_INVALID_ARG),
    (dict(m=0), sk.ERR_INVALID_ARG), (dict(m=(1 << 31) + 1), sk.ERR_INVALID_ARG), (dict(d=0), sk.ERR_INVALID_ARG),
    (dict(d=(1 << 24) + 1), sk.ERR_INVALID_ARG), (dict(eps=-1e-6), sk.ERR_INVALID_ARG), (dict(eps=float("nan")), sk.ERR_INVALID_ARG),
    (dict(eps=float("inf")), sk.ERR_INVALID_ARG), (dict(xt=sk.Q8_0), sk.ERR_UNSUPPORTED), (dict(rt=0), sk.ERR_UNSUPPORTED),
    (dict(wt=9), sk.ERR_UNSUPPORTED), (dict(ot=sk.Q4_0), sk.ERR_UNSUPPORTED), (dict(group=16), sk.ERR_UNSUPPORTED),
    (dict(group=-32), sk.ERR_UNSUPPORTED), (dict(ldx=63), sk.ERR_SHAPE), (dict(ldr=-64), sk.ERR_SHAPE), (dict(ldro=1), sk.ERR_SHAPE),
    (dict(ldo=63), sk.ERR_SHAPE), (dict(ldq=63), sk.ERR_SHAPE), (dict(ldo=1 << 41), sk.ERR_INVALID_ARG),
    (dict(x=at(1) + 1), sk.ERR_ALIGNMENT), (dict(r=at(2) + 2), sk.ERR_ALIGNMENT), (dict(w=at(3) + 1), sk.ERR_ALIGNMENT),
    (dict(ro=at(4) + 2), sk.ERR_ALIGNMENT), (dict(out=at(5) + 1), sk.ERR_ALIGNMENT), (dict(s=at(7) + 2), sk.ERR_ALIGNMENT),
    # outputs over inputs (but for the allowed ones), and over one another
    (dict(ro=at(1)), sk.ERR_INVALID_ARG), (dict(ro=at(2) + 4), sk.ERR_INVALID_ARG), (dict(ro=at(2), ldro=68), sk.ERR_INVALID_ARG),
    (dict(out=at(1) + 2), sk.ERR_INVALID_ARG), (dict(out=at(1), ot=sk.F16), sk.ERR_INVALID_ARG), (dict(out=at(2)), sk.ERR_INVALID_ARG),
    (dict(out=at(3)), sk.ERR_INVALID_ARG), (dict(q=at(1) + 8), sk.ERR_INVALID_ARG), (dict(s=at(3) + 4), sk.ERR_INVALID_ARG),
    (dict(out=at(4)), sk.ERR_INVALID_ARG), (dict(q=at(5)), sk.ERR_INVALID_ARG), (dict(s=at(6)), sk.ERR_INVALID_ARG),
])
def test_norm_refusals(kw, status):
    assert norm_run(**kw) == status


def pool(**kw):
    d = dict(struct_size=ctypes.sizeof(sk.AdaptersDesc), dtype=sk.BF16, count=4, rank=16, k=64, n=50, A=at(1), B=at(2), ranks=at(3),
             scaling=at(4))
    d.update(kw)
    return sk.AdaptersDesc(**d)


def adapt_run(m=5, x=at(5), ldx=0, ids=at(6), ids64=0, base=at(7), ldb=0, bt=sk.F32, out=at(8), ldo=0, ot=sk.F32, ws=at(9),
              nbytes=1 << 30, desc=True, **kw):
    p = pool(**kw)
    return lib.skinny_adapters_run(ctypes.addressof(p) if desc else None, m, x, ldx, ids, ids64, base, ldb, bt, out, ldo, ot, ws,
                                   nbytes, None)


POOL_REFUSALS = [
    (dict(struct_size=8), sk.ERR_INVALID_ARG), (dict(dtype=sk.F32), sk.ERR_UNSUPPORTED), (dict(dtype=sk.Q8_0), sk.ERR_UNSUPPORTED),
    (dict(count=0), sk.ERR_INVALID_ARG), (dict(count=8193), sk.ERR_INVALID_ARG), (dict(rank=0), sk.ERR_INVALID_ARG),
    (dict(rank=264), sk.ERR_INVALID_ARG), (dict(k=0), sk.ERR_INVALID_ARG), (dict(k=(1 << 24) + 8), sk.ERR_INVALID_ARG),
    (dict(n=0), sk.ERR_INVALID_ARG), (dict(n=(1 << 24) + 1), sk.ERR_INVALID_ARG), (dict(rank=12), sk.ERR_SHAPE),
    (dict(k=60), sk.ERR_SHAPE), (dict(m=0), sk.ERR_INVALID_ARG), (dict(m=(1 << 20) + 1), sk.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", POOL_REFUSALS + [
    (dict(desc=False), sk.ERR_INVALID_ARG), (dict(A=None), sk.ERR_INVALID_ARG), (dict(B=None), sk.ERR_INVALID_ARG),
    (dict(x=None), sk.ERR_INVALID_ARG), (dict(ids=None), sk.ERR_INVALID_ARG), (dict(out=None), sk.ERR_INVALID_ARG),
    (dict(bt=sk.F16), sk.ERR_UNSUPPORTED), (dict(ot=sk.F16), sk.ERR_UNSUPPORTED), (dict(ot=sk.Q8_0), sk.ERR_UNSUPPORTED),
    (dict(ldx=56), sk.ERR_SHAPE), (dict(ldb=49), sk.ERR_SHAPE), (dict(ldo=-50), sk.ERR_SHAPE), (dict(ldx=1 << 41), sk.ERR_INVALID_ARG),
    (dict(ldx=68), sk.ERR_ALIGNMENT), (dict(x=at(5) + 8), sk.ERR_ALIGNMENT), (dict(A=at(1) + 8), sk.ERR_ALIGNMENT),
    (dict(B=at(2) + 2), sk.ERR_ALIGNMENT), (dict(ranks=at(3) + 2), sk.ERR_ALIGNMENT), (dict(scaling=at(4) + 1), sk.ERR_ALIGNMENT),
    (dict(ids=at(6) + 4, ids64=1), sk.ERR_ALIGNMENT), (dict(base=at(7) + 2), sk.ERR_ALIGNMENT), (dict(out=at(8) + 2), sk.ERR_ALIGNMENT),
    (dict(ws=at(9) + 8), sk.ERR_ALIGNMENT), (dict(ws=None), sk.ERR_WORKSPACE), (dict(nbytes=64), sk.ERR_WORKSPACE),
    (dict(out=at(5)), sk.ERR_INVALID_ARG), (dict(out=at(1)), sk.ERR_INVALID_ARG), (dict(out=at(2)), sk.ERR_INVALID_ARG),
    (dict(out=at(3)), sk.ERR_INVALID_ARG), (dict(out=at(4)), sk.ERR_INVALID_ARG), (dict(out=at(6)), sk.ERR_INVALID_ARG),
    (dict(out=at(7) + 4), sk.ERR_INVALID_ARG), (dict(out=at(7), ldo=60), sk.ERR_INVALID_ARG),
    (dict(out=at(7), ot=sk.BF16), sk.ERR_INVALID_ARG),
])
def test_adapters_refusals(kw, status):
    assert adapt_run(**kw) == status


@pytest.mark.parametrize("kw,status", POOL_REFUSALS)
def test_adapters_workspace_refusals(kw, status):
    kw = dict(kw)
    m, n = kw.pop("m", 5), ctypes.c_size_t()
    p = pool(**kw)
    assert lib.skinny_adapters_workspace_size(ctypes.addressof(p), m, ctypes.byref(n)) == status


def test_adapters_workspace_size():
    n = ctypes.c_size_t()

    def size(m, **kw):
        p = pool(**kw)
        assert lib.skinny_adapters_workspace_size(ctypes.addressof(p), m, ctypes.byref(n)) == sk.OK
        return n.value

    p = pool()
    assert lib.skinny_adapters_workspace_size(ctypes.addressof(p), 1, None) == sk.ERR_INVALID_ARG
    assert lib.skinny_adapters_workspace_size(None, 1, ctypes.byref(n)) == sk.ERR_INVALID_ARG
    assert size(1) >= 16 * 4
    for k in (64, 5120, 1 << 24):  # a part of the inner values for each of at most 32 splits of k
        assert 16 * 16 * 4 <= size(16, k=k) <= 32 * 16 * 16 * 4 + 2048  # (the tiles and their rows)
    # and the lists of sorted rows
    assert size(4096, rank=32, k=5120) >= 4096 * (32 * 4 + 4)
    assert size(1 << 20, count=8192) < 1 << 31


def rules(**kw):
    d = dict(struct_size=ctypes.sizeof(sk.LogitRulesDesc), tokens64=0, history=at(2), ldh=0, history_len=20, lengths=at(3),
             prompt_lengths=at(4), repetition=at(5), frequency=at(6), presence=at(7), bias_ids=at(8), bias_values=at(9), biases=3,
             mask=at(10), ldm=0, masks=4, mask_rows=at(11))
    d.update(kw)
    return sk.LogitRulesDesc(**d)


NO_HISTORY = dict(history=None, history_len=0, lengths=None, prompt_lengths=None, repetition=None, frequency=None, presence=None)
NO_BIAS = dict(bias_ids=None, bias_values=None, biases=0)
NO_MASK = dict(mask=None, masks=0, mask_rows=None)


def adjust_run(m=4, vocab=1000, x=at(1), ld=0, dtype=sk.BF16, out=at(12), ldo=0, ot=sk.F32, desc=True, **kw):
    r = rules(**kw)
    return lib.skinny_adjust_logits_run(m, vocab, x, ld, dtype, ctypes.addressof(r) if desc else None, out, ldo, ot, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), sk.ERR_INVALID_ARG), (dict(out=None), sk.ERR_INVALID_ARG), (dict(desc=False), sk.ERR_INVALID_ARG),
    (dict(struct_size=16), sk.ERR_INVALID_ARG), (dict(m=0), sk.ERR_INVALID_ARG), (dict(vocab=0), sk.ERR_INVALID_ARG),
    (dict(vocab=(1 << 30) + 1), sk.ERR_INVALID_ARG), (dict(m=1 << 30, vocab=1 << 21), sk.ERR_INVALID_ARG),
    (dict(dtype=sk.Q8_0), sk.ERR_UNSUPPORTED), (dict(ot=sk.F16), sk.ERR_UNSUPPORTED), (dict(ot=0), sk.ERR_UNSUPPORTED),
    (dict(history_len=0), sk.ERR_INVALID_ARG), (dict(history_len=-1), sk.ERR_INVALID_ARG), (dict(history_len=(1 << 24) + 1), sk.ERR_INVALID_ARG),
    (dict(history=None), sk.ERR_INVALID_ARG), (dict(NO_HISTORY, lengths=at(3)), sk.ERR_INVALID_ARG),
    (dict(NO_HISTORY, presence=at(3)), sk.ERR_INVALID_ARG), (dict(NO_HISTORY, history_len=5), sk.ERR_INVALID_ARG),
    (dict(biases=-1), sk.ERR_INVALID_ARG), (dict(biases=(1 << 16) + 1), sk.ERR_INVALID_ARG), (dict(biases=0), sk.ERR_INVALID_ARG),
    (dict(bias_ids=None), sk.ERR_INVALID_ARG), (dict(bias_values=None), sk.ERR_INVALID_ARG), (dict(masks=0), sk.ERR_INVALID_ARG),
    (dict(mask=None), sk.ERR_INVALID_ARG), (dict(NO_MASK, mask_rows=at(11)), sk.ERR_INVALID_ARG),
    (dict(ld=999), sk.ERR_SHAPE), (dict(ldo=999), sk.ERR_SHAPE), (dict(ldh=19), sk.ERR_SHAPE), (dict(ldm=31), sk.ERR_SHAPE),
    (dict(ld=-1), sk.ERR_SHAPE), (dict(masks=3, mask_rows=None), sk.ERR_SHAPE), (dict(ld=1 << 41), sk.ERR_INVALID_ARG),
    (dict(x=at(1) + 1), sk.ERR_ALIGNMENT), (dict(out=at(12) + 2), sk.ERR_ALIGNMENT), (dict(history=at(2) + 2), sk.ERR_ALIGNMENT),
    (dict(history=at(2) + 4, tokens64=1), sk.ERR_ALIGNMENT), (dict(bias_ids=at(8) + 4, tokens64=1), sk.ERR_ALIGNMENT),
    (dict(lengths=at(3) + 1), sk.ERR_ALIGNMENT), (dict(mask=at(10) + 2), sk.ERR_ALIGNMENT), (dict(mask_rows=at(11) + 1), sk.ERR_ALIGNMENT),
    (dict(repetition=at(5) + 2), sk.ERR_ALIGNMENT), (dict(bias_values=at(9) + 1), sk.ERR_ALIGNMENT),
    (dict(out=at(1)), sk.ERR_INVALID_ARG), (dict(out=at(1), ot=sk.BF16, ldo=1008), sk.ERR_INVALID_ARG),
    (dict(out=at(1) + 2, ot=sk.BF16), sk.ERR_INVALID_ARG), (dict(out=at(2)), sk.ERR_INVALID_ARG), (dict(out=at(3)), sk.ERR_INVALID_ARG),
    (dict(out=at(8) - 4), sk.ERR_INVALID_ARG), (dict(out=at(9)), sk.ERR_INVALID_ARG), (dict(out=at(10)), sk.ERR_INVALID_ARG),
    (dict(out=at(11)), sk.ERR_INVALID_ARG),
])
def test_adjust_refusals(kw, status):
    assert adjust_run(**kw) == status


def test_adjust_nothing_in_place_is_no_launch():
    """No rule, in place: done before any HIP call."""
    assert adjust_run(out=at(1), ot=sk.BF16, **NO_HISTORY, **NO_BIAS, **NO_MASK) == sk.OK


FAR = [(1 << 23, 1 << 40), ((1 << 23) + 1, 1 << 40), (1 << 30, (1 << 30) + 1), ((1 << 29) + 1, 1 << 35), (1 << 30, 1 << 40)]


@pytest.mark.parametrize("m,ld", FAR)
@pytest.mark.parametrize("name", ["ldx", "ldr", "ldro", "ldo", "ldq"])
def test_norm_rows_further_apart_than_memory_are_refused(name, m, ld):
    """Their bytes pass 63 bits, where the spans that must not overlap came out as any."""
    assert norm_run(m=m, x=at(1), r=at(2), ro=at(3), out=at(4), q=at(5), **{name: ld}) == sk.ERR_INVALID_ARG
    assert norm_run(m=m, r=None, ro=None, q=None, s=None, ldx=ld, out=at(1) + 128, ldo=64) == sk.ERR_INVALID_ARG


@pytest.mark.parametrize("m,ld", FAR)
def test_adjust_rows_further_apart_than_memory_are_refused(m, ld):
    for kw in (dict(ld=ld), dict(ldo=ld), dict(ldh=ld), dict(ldm=ld, masks=m), dict(ld=ld, out=at(1) + 4096)):
        assert adjust_run(**{"m": m, "vocab": 1000, **NO_BIAS, **kw}) == sk.ERR_INVALID_ARG


@pytest.mark.parametrize("i", [1, 2, 3, 4, 5, 6, 7, 8])
def test_adapters_workspace_apart_from_every_operand(i):
    """A, B, ranks, scaling, x, ids, base, out: the workspace is written before they are read."""
    assert adapt_run(ws=at(i)) == sk.ERR_INVALID_ARG
    assert adapt_run(ws=at(i) - 64) == sk.ERR_INVALID_ARG
