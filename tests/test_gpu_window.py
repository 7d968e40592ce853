"""The three window operators one after another, as the example runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sk = pytest.importorskip("row_gemv_decode_amd")

PATH = os.path.join(os.path.dirname(__file__), "..", "examples", "decode_window.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_window", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_window_rows_do_not_depend_on_the_window(example):
    """Row i of a window of m rows is the one-row call's, bit for bit, through
    all three operators."""
    w = example.Window(experts=24, topk=4, d=256, inter=192, shared=128, vocab=5003, group=64, seed=5)
    x = torch.randn((16, 256), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    tok = torch.randint(0, 5003, (16,), generator=torch.Generator().manual_seed(7)).cuda()
    one = [w.score(x[i:i + 1], tok[i:i + 1]) for i in range(16)]
    for m in (1, 2, 3, 8, 9, 16):
        logits, s = w.score(x[:m].contiguous(), tok[:m])
        torch.cuda.synchronize()
        for i in range(m):
            assert torch.equal(logits[i], one[i][0][0])
            assert all(torch.equal(a[i], b[0]) for a, b in zip(s, one[i][1]))


def test_window_accepts_the_best_tokens(example):
    w = example.Window(experts=16, topk=2, d=128, inter=128, shared=64, vocab=1000, group=32, seed=8)
    x = torch.randn((7, 128), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    logits, _ = w.score(x, torch.zeros(7, dtype=torch.int64, device="cuda"))
    best = logits.argmax(1)
    for wrong in (0, 3, 6):
        tok = best.clone()
        tok[wrong] = (tok[wrong] + 1) % 1000
        _, s = w.score(x, tok)
        assert example.accepted(s) == wrong
        assert torch.equal(s.top_ids[:, 0].long(), best)
    assert example.accepted(w.score(x, best)[1]) == 7
