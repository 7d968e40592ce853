"""The operators of a batch of requests one after another, around the shared
projections, as the example runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sk = pytest.importorskip("row_gemv_decode_amd")

PATH = os.path.join(os.path.dirname(__file__), "..", "examples", "decode_requests.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_requests", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def batch(example, n, **kw):
    s = example.Step(n, d=512, vocab=5003, room=40, **kw)
    s.start([[3 * i + 1, 7, 7, i % 2, 11 * i + 2] for i in range(n)])
    s.adapters.copy_(torch.arange(n, device="cuda") % 5 - 1)
    s.repetition.copy_(torch.linspace(1.0, 1.6, n))
    s.presence.fill_(0.5)
    s.frequency.fill_(0.25)
    s.allow(1, [5, 9, 4000, 5002])
    return s


def plain(s, raw):
    """The rules in 64 bits, from their definition."""
    x = raw.double().cpu()
    for i in range(x.shape[0]):
        held = s.history[i, :int(s.lengths[i])].tolist()
        made = held[int(s.prompts[i]):]
        for t in set(held):
            v = float(x[i, t])
            v = v / float(s.repetition[i]) if v > 0 else v * float(s.repetition[i])
            x[i, t] = v - (float(s.frequency[i]) * made.count(t) + float(s.presence[i]) * (t in made))
        if int(s.mask_rows[i]) >= 0:
            word = s.mask[int(s.mask_rows[i])].cpu().long()
            for t in range(x.shape[1]):
                if not int(word[t // 32]) >> (t % 32) & 1:
                    x[i, t] = -float("inf")
    return x


def test_steps_follow_the_rules(example):
    s = batch(example, 7)
    for _ in range(4):
        raw, logits = s.logits()
        want = plain(s, raw)
        got = logits.double().cpu()
        assert torch.equal(got.isneginf(), want.isneginf())
        fin = want.isfinite()
        # quotient, product, two sums: each rounds by half a step of numbers below 32
        assert bool(((got - want)[fin].abs() <= 4 * 32 * 2.0 ** -24).all())
        tokens, lp = s.step()
        assert torch.equal(tokens, logits.argmax(1)) and bool((lp <= 0).all())
    assert set(s.history[1, 5:9].tolist()) <= {5, 9, 4000, 5002}


def test_adapters_change_their_requests_only(example):
    s = batch(example, 6)
    raw, _ = s.logits()
    s.adapters.fill_(-1)
    bare, _ = s.logits()
    for i in range(6):
        assert torch.equal(raw[i], bare[i]) == (i % 5 == 0)


def test_a_captured_step_replays_the_eager_one(example):
    """The whole step in one graph: the histories grow from replay to replay."""
    s, e = batch(example, 5), batch(example, 5)
    for x in (s, e):
        x.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.logits()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tokens, lp = s.step()
    for _ in range(5):
        g.replay()
        want_tokens, want_lp = e.step()
        torch.cuda.synchronize()
        assert torch.equal(tokens, want_tokens) and torch.equal(lp, want_lp)
        assert torch.equal(s.history, e.history) and torch.equal(s.lengths, e.lengths)


def test_full_histories_stay_as_they_are(example):
    """Steps past the histories' room, eager and replayed: what is held stays."""
    s = example.Step(3, d=512, vocab=5003, room=6)
    s.start([[5, 9, 2], [7], [1, 2, 3, 4, 5, 6]])
    s.step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    assert s.lengths.tolist() == [4, 2, 6]
    held = s.history.clone()
    for n in ([5, 3, 6], [6, 4, 6], [6, 5, 6], [6, 6, 6], [6, 6, 6]):
        g.replay()
        assert s.lengths.tolist() == n and s.history[2].tolist() == [1, 2, 3, 4, 5, 6]
    assert torch.equal(s.history[0, :4], held[0, :4]) and torch.equal(s.history[1, :2], held[1, :2])
    full = s.history.clone()
    s.step()
    assert torch.equal(s.history, full) and s.lengths.tolist() == [6, 6, 6]


def test_prompts_that_do_not_fit_are_refused(example):
    s = example.Step(2, d=512, vocab=5003, room=4)
    for bad in ([[1, 2]], [[1], []], [[1], [1, 2, 3, 4, 5]], [[1], [2], [3]], [[1], [5003]], [[-1], [1]]):
        with pytest.raises(ValueError):
            s.start(bad)


def test_example_runs_more_steps_than_its_usual_room(example, monkeypatch, capsys):
    monkeypatch.setattr(example.sys, "argv", ["decode_requests.py", "--requests", "2", "--steps", "70"])
    example.main()
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 2 and all(len(line.split("[")[1].split(",")) == 73 for line in lines)
