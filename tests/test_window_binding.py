"""The Python side of the decode-window operators, on the host: what the
binding hands to the library, recorded by a stand-in for it.  Tensors lie in
host memory and no kernel runs."""
import contextlib
import ctypes
import threading
import time

import pytest

torch = pytest.importorskip("torch")
sk = pytest.importorskip("row_gemv_decode_amd")


class Recorder:
    """Stands in for the library: keeps the arguments of every call."""

    def __init__(self):
        self.calls = []
        self.need = 0  # workspace bytes
        self.during = None  # called within each run

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_size"):
                args[-1]._obj.value = self.need
            else:
                self.calls.append((name, args))
            if self.during is not None:
                self.during(name, args)
            return sk.OK

        return call


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(sk, "_lib", rec)
    monkeypatch.setattr(sk, "_gpu", lambda where, t: -1)
    monkeypatch.setattr(sk, "_handle", lambda index, stream: 0)
    monkeypatch.setattr(sk, "_current_device", lambda: -1, raising=False)
    monkeypatch.setattr(sk, "_logprob_need", {})
    return rec


def head(n=8, k=64):
    return sk.W4(torch.zeros((n, k // 2), dtype=torch.uint8), torch.ones((n, k // 32), dtype=torch.bfloat16))


def shared_rows(m, length, dtype):
    """Matrices of m rows whose memory holds fewer: one row for all, and rows
    that begin half a row apart."""
    one = torch.arange(length, dtype=torch.float32).to(dtype)
    half = torch.arange((m + 1) * length // 2, dtype=torch.float32).to(dtype)
    return one.expand(m, -1), half.as_strided((m, length), (length // 2, 1))


def test_w4_rows_that_share_memory_are_copied(lib):
    for a in shared_rows(4, 64, torch.bfloat16):
        seen = []

        def during(name, args, a=a, seen=seen):
            m, _, k, _, ptr, lda = args[:6]
            assert ptr != a.data_ptr(), "read as rows that lie apart"
            lda = lda or k
            raw = ctypes.string_at(ptr, 2 * ((m - 1) * lda + k))
            got = torch.frombuffer(bytearray(raw), dtype=torch.bfloat16).as_strided((m, k), (lda, 1))
            seen.append(torch.equal(got, a))

        lib.during = during
        sk.mm_w4(a, head())
        assert seen == [True]


def test_logprobs_rows_that_share_memory_are_copied(lib):
    for x in shared_rows(3, 50, torch.float32):
        seen = []

        def during(name, args, x=x, seen=seen):
            if name != "skinny_token_logprobs_run":
                return
            m, vocab, ptr, ld = args[:4]
            assert ptr != x.data_ptr(), "read as rows that lie apart"
            ld = ld or vocab
            raw = ctypes.string_at(ptr, 4 * ((m - 1) * ld + vocab))
            got = torch.frombuffer(bytearray(raw), dtype=torch.float32).as_strided((m, vocab), (ld, 1))
            seen.append(torch.equal(got, x))

        lib.during = during
        sk.token_logprobs(x, torch.zeros(3, dtype=torch.int64), topk=2)
        assert seen == [True]


def test_w4_output_rows_that_share_memory_are_refused(lib):
    a = torch.zeros((4, 64), dtype=torch.bfloat16)
    for n, out in ((8, torch.zeros(8).expand(4, -1)), (8, torch.zeros(40).as_strided((4, 8), (4, 1))),
                   (1, torch.zeros((1, 1)).expand(4, 1))):
        with pytest.raises(ValueError, match="share memory"):
            sk.mm_w4(a, head(n), out=out)
    assert lib.calls == []


def test_columns_that_lie_apart_are_refused(lib):
    for a in (torch.zeros((64, 4), dtype=torch.bfloat16).t(), torch.zeros((4, 1), dtype=torch.bfloat16).expand(4, 64)):
        with pytest.raises(ValueError, match="contiguous rows"):
            sk.mm_w4(a, head())
    assert lib.calls == []


def test_rows_that_lie_apart_are_read_where_they_are(lib):
    a = torch.zeros((4, 80), dtype=torch.bfloat16)[:, :64]
    x = torch.zeros((3, 60))[:, :50]
    sk.mm_w4(a, head())
    sk.mm_w4(a[:1], head())
    sk.token_logprobs(x, torch.zeros(3, dtype=torch.int64))
    got = [args for name, args in lib.calls]
    assert (got[0][4], got[0][5]) == (a.data_ptr(), 80)
    assert (got[1][4], got[1][5]) == (a.data_ptr(), 0)
    assert (got[2][2], got[2][3]) == (x.data_ptr(), 60)


@pytest.mark.parametrize("stream", [None, object()])
def test_a_capture_never_takes_the_streams_workspace(lib, monkeypatch, stream):
    """A graph outlives the stream's workspace, which a larger call replaces:
    it gets one of its own, with zeroed counters, and leaves the stream's."""
    lib.need = 3 * sk.WINDOW_COUNTER_BYTES
    cached = torch.zeros(lib.need, dtype=torch.uint8)
    cache = {(-1, 5): cached}
    capturing = [True]
    monkeypatch.setattr(sk, "_logprob_ws", cache)
    monkeypatch.setattr(sk, "_handle", lambda index, stream: 5)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: None)
    monkeypatch.setattr(sk, "_capturing", lambda handle, *stream: handle == 5 and capturing[0])
    used = []

    def during(name, args):
        if name == "skinny_token_logprobs_run":
            used.append(args[13])
            if capturing[0]:
                assert args[14] == lib.need
                assert ctypes.string_at(args[13], sk.WINDOW_COUNTER_BYTES) == bytes(sk.WINDOW_COUNTER_BYTES)

    lib.during = during
    x, t = torch.zeros((2, 50)), torch.zeros(2, dtype=torch.int64)
    sk.token_logprobs(x, t, stream=stream)
    assert used[0] != cached.data_ptr() and cache == {(-1, 5): cached}
    capturing[0] = False
    sk.token_logprobs(x, t, stream=stream)
    assert used[1] == cached.data_ptr()
    monkeypatch.setattr(sk, "_logprob_need", {})
    lib.need *= 2
    sk.token_logprobs(x, t, stream=stream)  # a larger call replaces the stream's
    assert used[2] != cached.data_ptr() and cache[-1, 5].numel() == lib.need


def moe_layer(d=64, inter=32, experts=4):
    half = torch.bfloat16
    return sk.MoELayer(torch.zeros((experts, d), dtype=half), torch.zeros((experts, 2 * inter, d), dtype=half),
                       torch.zeros((experts, d, inter), dtype=half), topk=2)


def test_threads_do_not_enqueue_a_layers_runs_at_once(lib, monkeypatch):
    """A run is several launches over one workspace: another thread's must not
    come between them."""
    monkeypatch.setattr(sk, "_stream_workspace", lambda *a: torch.zeros(16, dtype=torch.uint8))
    layer = moe_layer()
    inside, most = [0], [0]

    def during(name, args):
        if name == "skinny_moe_run":
            inside[0] += 1
            most[0] = max(most[0], inside[0])
            time.sleep(0.05)  # (as the library's call does, without the interpreter's lock)
            inside[0] -= 1

    lib.during = during
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    threads = [threading.Thread(target=layer, args=(x,)) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sum(name == "skinny_moe_run" for name, _ in lib.calls) == 4 and most[0] == 1


def test_the_tensors_gpu_is_current_during_a_call(lib, monkeypatch):
    """The library launches on the current device, whatever the stream's."""
    monkeypatch.setattr(sk, "_stream_workspace", lambda *a: torch.zeros(16, dtype=torch.uint8))
    layer = moe_layer()
    current, seen = [3], []

    @contextlib.contextmanager
    def device(index):
        was, current[0] = current[0], index
        yield
        current[0] = was

    monkeypatch.setattr(sk, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    lib.during = lambda name, args: seen.append((name, current[0])) if name.endswith("_run") else None
    sk.mm_w4(torch.zeros((2, 64), dtype=torch.bfloat16), head())
    layer(torch.zeros((2, 64), dtype=torch.bfloat16))
    sk.token_logprobs(torch.zeros((2, 50)), torch.zeros(2, dtype=torch.int64), topk=1)
    assert seen == [("skinny_w4_mm_run", -1), ("skinny_moe_run", -1), ("skinny_token_logprobs_run", -1)]
    assert current == [3]
