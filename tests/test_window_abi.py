"""Argument checks of the decode-window operators' C entry points (4-bit
grouped GEMV, MoE layer, token log probabilities): every refusal comes from
the host before any HIP call, so these run without a GPU."""
import ctypes
import os
import re

import pytest

from conftest import ROOT

sk = pytest.importorskip("row_gemv_decode_amd")

lib = sk.lib()
P = 1 << 20  # made-up device addresses, far enough apart not to overlap
A, CODES, SCALES, ZEROS, C = (i * (1 << 30) + P for i in range(1, 6))


def test_exports_every_declared_symbol():
    with open(os.path.join(ROOT, "include", "skinny_window.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"SKINNY_API\s+[\w ]+?\**\s*(\w+)\s*\(", text)
    assert len(names) == 7 and set(names) == set(sk.WINDOW_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def w4_run(m=2, n=64, k=256, group=64, a=A, lda=0, a_dtype=sk.BF16, codes=CODES, scales=SCALES, zeros=ZEROS, c=C, ldc=0,
           c_dtype=sk.F32, desc=True):
    d = sk.W4Desc(codes, scales, zeros)
    return lib.skinny_w4_mm_run(m, n, k, group, a, lda, a_dtype, ctypes.addressof(d) if desc else None, c, ldc, c_dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(a=0), sk.ERR_INVALID_ARG), (dict(codes=0), sk.ERR_INVALID_ARG), (dict(scales=0), sk.ERR_INVALID_ARG),
    (dict(c=0), sk.ERR_INVALID_ARG), (dict(desc=False), sk.ERR_INVALID_ARG),
    (dict(a_dtype=sk.F32), sk.ERR_UNSUPPORTED), (dict(c_dtype=sk.Q8_0), sk.ERR_UNSUPPORTED),
    (dict(group=16), sk.ERR_UNSUPPORTED), (dict(group=0), sk.ERR_UNSUPPORTED), (dict(group=256), sk.ERR_UNSUPPORTED),
    (dict(m=0), sk.ERR_INVALID_ARG), (dict(m=17), sk.ERR_INVALID_ARG), (dict(n=0), sk.ERR_INVALID_ARG),
    (dict(k=0), sk.ERR_INVALID_ARG), (dict(n=1 << 31), sk.ERR_INVALID_ARG), (dict(k=1 << 31), sk.ERR_INVALID_ARG),
    (dict(k=96), sk.ERR_SHAPE), (dict(lda=248), sk.ERR_SHAPE), (dict(ldc=63), sk.ERR_SHAPE), (dict(lda=-8), sk.ERR_SHAPE),
    (dict(lda=260), sk.ERR_ALIGNMENT), (dict(a=A + 8), sk.ERR_ALIGNMENT), (dict(codes=CODES + 4), sk.ERR_ALIGNMENT),
    (dict(scales=SCALES + 1), sk.ERR_ALIGNMENT), (dict(c=C + 2), sk.ERR_ALIGNMENT),
    (dict(c=A), sk.ERR_INVALID_ARG), (dict(c=CODES + 64), sk.ERR_INVALID_ARG), (dict(c=SCALES - 16), sk.ERR_INVALID_ARG),
    (dict(c=ZEROS), sk.ERR_INVALID_ARG), (dict(lda=1 << 41), sk.ERR_INVALID_ARG),
])
def test_w4_refusals(kw, status):
    assert w4_run(**kw) == status


def moe_desc(**kw):
    d = dict(struct_size=ctypes.sizeof(sk.MoEDesc), dtype=sk.BF16, w_dtype=sk.BF16, out_dtype=sk.F32, group=0, topk=4, max_m=16,
             d=256, inter=128, shared_inter=64, experts=32, ldx=0, ldo=0, flags=0, num_cus=256)
    d.update(kw)
    return sk.MoEDesc(**d)


def moe_create(**kw):
    h = ctypes.c_void_p()
    st = lib.skinny_moe_plan_create(ctypes.byref(moe_desc(**kw)), ctypes.byref(h))
    assert (st == sk.OK) == (h.value is not None)
    return st, h


@pytest.mark.parametrize("kw,status", [
    (dict(struct_size=8), sk.ERR_INVALID_ARG), (dict(dtype=sk.F32), sk.ERR_UNSUPPORTED),
    (dict(w_dtype=sk.F16), sk.ERR_UNSUPPORTED), (dict(w_dtype=sk.Q4_0), sk.ERR_UNSUPPORTED),
    (dict(out_dtype=sk.Q8_0), sk.ERR_UNSUPPORTED), (dict(flags=2), sk.ERR_UNSUPPORTED),
    (dict(group=32), sk.ERR_UNSUPPORTED), (dict(w_dtype=sk.DTYPE_W4), sk.ERR_UNSUPPORTED),
    (dict(w_dtype=sk.DTYPE_W4, group=48), sk.ERR_UNSUPPORTED),
    (dict(max_m=0), sk.ERR_INVALID_ARG), (dict(max_m=17), sk.ERR_INVALID_ARG), (dict(topk=0), sk.ERR_INVALID_ARG),
    (dict(topk=33, experts=64), sk.ERR_INVALID_ARG), (dict(topk=8, experts=7), sk.ERR_INVALID_ARG),
    (dict(experts=1025), sk.ERR_INVALID_ARG), (dict(d=0), sk.ERR_INVALID_ARG), (dict(inter=0), sk.ERR_INVALID_ARG),
    (dict(shared_inter=-32), sk.ERR_INVALID_ARG), (dict(d=(1 << 20) + 32), sk.ERR_INVALID_ARG),
    (dict(d=250), sk.ERR_SHAPE), (dict(inter=100), sk.ERR_SHAPE), (dict(shared_inter=16), sk.ERR_SHAPE),
    (dict(w_dtype=sk.DTYPE_W4, group=128, d=192), sk.ERR_SHAPE), (dict(ldx=248), sk.ERR_SHAPE), (dict(ldo=255), sk.ERR_SHAPE),
    (dict(ldx=260), sk.ERR_ALIGNMENT), (dict(num_cus=-1), sk.ERR_INVALID_ARG),
])
def test_moe_plan_refusals(kw, status):
    assert moe_create(**kw)[0] == status


def test_moe_plan_null_arguments():
    h = ctypes.c_void_p()
    assert lib.skinny_moe_plan_create(None, ctypes.byref(h)) == sk.ERR_INVALID_ARG
    assert lib.skinny_moe_plan_create(ctypes.byref(moe_desc()), None) == sk.ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert lib.skinny_moe_workspace_size(None, ctypes.byref(n)) == sk.ERR_INVALID_ARG
    lib.skinny_moe_plan_destroy(None)


def moe_weights(w4=False, shared=True, **kw):
    w = iter(range(10, 40))

    def one(used=True):
        if not used:
            return sk.W4Desc()
        return sk.W4Desc(next(w) << 32, next(w) << 32, None) if w4 else sk.W4Desc(next(w) << 32)

    d = dict(router=9 << 32, w13=one(), w2=one(), shared13=one(shared), shared2=one(shared),
             shared_gate=8 << 32 if shared else None)
    d.update(kw)
    return sk.MoEWeightsDesc(**d)


def moe_run(plan, w, m=3, x=1 << 32, out=2 << 32, idx=3 << 32, wt=4 << 32, ws=5 << 32, nbytes=1 << 40):
    return lib.skinny_moe_run(plan, m, x, ctypes.addressof(w) if w is not None else None, out, idx, wt, ws, nbytes, None)


def test_moe_run_refusals():
    _, h = moe_create()
    _, h4 = moe_create(w_dtype=sk.DTYPE_W4, group=64, shared_inter=0)
    n = ctypes.c_size_t()
    assert lib.skinny_moe_workspace_size(h, ctypes.byref(n)) == sk.OK and n.value > 0
    good = moe_weights()
    assert moe_run(None, good) == sk.ERR_INVALID_ARG
    assert moe_run(h, None) == sk.ERR_INVALID_ARG
    for kw, st in ((dict(m=0), sk.ERR_INVALID_ARG), (dict(m=17), sk.ERR_INVALID_ARG), (dict(x=None), sk.ERR_INVALID_ARG),
                   (dict(out=None), sk.ERR_INVALID_ARG), (dict(x=(1 << 32) + 2), sk.ERR_ALIGNMENT),
                   (dict(out=(2 << 32) + 2), sk.ERR_ALIGNMENT), (dict(idx=(3 << 32) + 1), sk.ERR_ALIGNMENT),
                   (dict(wt=(4 << 32) + 2), sk.ERR_ALIGNMENT), (dict(ws=None), sk.ERR_WORKSPACE),
                   (dict(nbytes=n.value - 1), sk.ERR_WORKSPACE), (dict(ws=(5 << 32) + 8), sk.ERR_ALIGNMENT),
                   (dict(out=(1 << 32) + 512), sk.ERR_INVALID_ARG)):
        assert moe_run(h, good, **kw) == st, kw
    for kw, st in ((dict(router=None), sk.ERR_INVALID_ARG), (dict(w13=sk.W4Desc()), sk.ERR_INVALID_ARG),
                   (dict(shared2=sk.W4Desc()), sk.ERR_INVALID_ARG), (dict(shared_gate=None), sk.ERR_INVALID_ARG),
                   (dict(w2=sk.W4Desc(7 << 32, 6 << 32)), sk.ERR_INVALID_ARG),
                   (dict(w2=sk.W4Desc(7 << 32, None, 6 << 32)), sk.ERR_INVALID_ARG),
                   (dict(w2=sk.W4Desc((7 << 32) + 8)), sk.ERR_ALIGNMENT), (dict(router=(9 << 32) + 2), sk.ERR_ALIGNMENT)):
        assert moe_run(h, moe_weights(**kw)) == st, kw
    assert moe_run(h4, moe_weights(shared=False)) == sk.ERR_INVALID_ARG           # 4-bit weights need scales
    assert moe_run(h4, moe_weights(w4=True)) == sk.ERR_INVALID_ARG                # a shared expert the plan has not
    assert moe_run(h4, moe_weights(w4=True, shared=False, w13=sk.W4Desc(7 << 32, (6 << 32) + 1))) == sk.ERR_ALIGNMENT
    lib.skinny_moe_plan_destroy(h)
    lib.skinny_moe_plan_destroy(h4)


def lp_run(m=4, vocab=5000, logits=1 << 32, ld=0, dtype=sk.F32, tokens=2 << 32, t64=1, topk=5, lp=3 << 32, ent=4 << 32,
           rank=5 << 32, ids=6 << 32, top=7 << 32, ws=8 << 32, nbytes=1 << 30):
    return lib.skinny_token_logprobs_run(m, vocab, logits, ld, dtype, tokens, t64, topk, lp, ent, rank, ids, top, ws, nbytes,
                                         None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), sk.ERR_INVALID_ARG), (dict(tokens=None), sk.ERR_INVALID_ARG), (dict(lp=None), sk.ERR_INVALID_ARG),
    (dict(ent=None), sk.ERR_INVALID_ARG), (dict(rank=None), sk.ERR_INVALID_ARG), (dict(ids=None), sk.ERR_INVALID_ARG),
    (dict(top=None), sk.ERR_INVALID_ARG), (dict(m=0), sk.ERR_INVALID_ARG), (dict(vocab=0), sk.ERR_INVALID_ARG),
    (dict(vocab=(1 << 30) + 1), sk.ERR_INVALID_ARG), (dict(m=1 << 30, vocab=1 << 21), sk.ERR_INVALID_ARG),
    (dict(topk=33), sk.ERR_INVALID_ARG), (dict(topk=-1), sk.ERR_INVALID_ARG), (dict(vocab=4), sk.ERR_INVALID_ARG),
    (dict(dtype=sk.Q8_0), sk.ERR_UNSUPPORTED), (dict(ld=4999), sk.ERR_SHAPE), (dict(ld=-1), sk.ERR_SHAPE),
    (dict(logits=(1 << 32) + 2), sk.ERR_ALIGNMENT), (dict(tokens=(2 << 32) + 4), sk.ERR_ALIGNMENT),
    (dict(ids=(6 << 32) + 2), sk.ERR_ALIGNMENT), (dict(lp=1 << 32), sk.ERR_INVALID_ARG), (dict(ent=2 << 32), sk.ERR_INVALID_ARG),
    (dict(top=6 << 32), sk.ERR_INVALID_ARG), (dict(ws=None), sk.ERR_WORKSPACE), (dict(nbytes=64), sk.ERR_WORKSPACE),
    (dict(ws=(8 << 32) + 4), sk.ERR_ALIGNMENT),
])
def test_logprobs_refusals(kw, status):
    assert lp_run(**kw) == status


def test_logprobs_workspace_size():
    n = ctypes.c_size_t()

    def size(m, vocab, topk):
        assert lib.skinny_token_logprobs_workspace_size(m, vocab, topk, ctypes.byref(n)) == sk.OK
        return n.value

    assert size(1, 1000, 5) == 0          # one workgroup per row
    assert size(1, 100000, 5) > 0
    assert size(5000, 100000, 5) == 0     # enough rows
    assert size(16, 100000, 32) >= size(1, 100000, 32)
    for bad in ((0, 10, 0), (1, 0, 0), (1, 10, 11), (1, 10, -1)):
        assert lib.skinny_token_logprobs_workspace_size(*bad, ctypes.byref(n)) == sk.ERR_INVALID_ARG
    assert lib.skinny_token_logprobs_workspace_size(1, 10, 0, None) == sk.ERR_INVALID_ARG


@pytest.mark.parametrize("topk,experts,shared_inter", [(10, 256, 1792), (4, 64, 0), (32, 512, 1024)])
def test_moe_workspace_holds_a_row_per_tokens_expert(topk, experts, shared_inter):
    """The inner values and outputs of the m * topk rows that a window has (three
    16-bit planes, and fp32), not of 16 rows for each expert that it may reach."""
    d, inter, m = 5120, 896, 16
    st, h = moe_create(d=d, inter=inter, topk=topk, experts=experts, shared_inter=shared_inter, w_dtype=sk.DTYPE_W4, group=128)
    assert st == sk.OK
    n = ctypes.c_size_t()
    assert lib.skinny_moe_workspace_size(h, ctypes.byref(n)) == sk.OK
    lib.skinny_moe_plan_destroy(h)
    rows = m * (topk * (inter * 6 + d * 4) + (shared_inter * 6 + d * 4 if shared_inter else 0))
    lists = m * experts * 4 + m * topk * 128  # logits, routing
    assert rows <= n.value <= rows + lists + (1 << 14)


@pytest.mark.parametrize("kw,status", [
    # 512 slots of 2^20 inner values: 2^29 / 32 workgroups of 256 threads
    (dict(topk=32, experts=1024, d=32, inter=1 << 20, shared_inter=0), sk.ERR_UNSUPPORTED),
    # 512 parts of 2^20 / 16 sets of columns, two sets per workgroup
    (dict(topk=32, experts=1024, d=1 << 20, inter=576, shared_inter=0), sk.ERR_UNSUPPORTED),
    (dict(topk=32, experts=256, d=32, inter=1 << 20, shared_inter=0), sk.OK),
    (dict(topk=32, experts=1024, d=32, inter=1 << 20, shared_inter=0, max_m=8), sk.OK),
])
def test_moe_plan_refuses_launches_past_a_grid(kw, status):
    """A grid counts threads in 32 bits; a larger launch would be cut off silently."""
    st, h = moe_create(**kw)
    assert st == status
    lib.skinny_moe_plan_destroy(h)
