"""The Python side of the operators of a batch of requests, on the host: what the
binding hands to the library, recorded by a stand-in for it.  Tensors lie in host
memory and no kernel runs."""
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
        self.need = 64  # workspace bytes
        self.during = None

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
    monkeypatch.setattr(sk, "_current_device", lambda: -1)
    monkeypatch.setattr(sk, "_adapter_ws", {})
    monkeypatch.setattr(sk, "_stream_workspace", lambda *a: torch.zeros(64, dtype=torch.uint8))
    return rec


half = torch.bfloat16


def adapters(count=2, rank=8, k=16, n=12):
    return sk.Adapters(torch.zeros((count, rank, k), dtype=half), torch.zeros((count, n, rank), dtype=half))


def shared_rows(m, length, dtype):
    one = torch.arange(length, dtype=torch.float32).to(dtype)
    return one.expand(m, -1), torch.arange((m + 1) * length // 2).to(dtype).as_strided((m, length), (length // 2, 1))


def read(ptr, ld, like):
    m, n = like.shape
    raw = bytearray(ctypes.string_at(ptr, like.element_size() * ((m - 1) * (ld or n) + n)))
    return torch.frombuffer(raw, dtype=like.dtype).as_strided((m, n), (ld or n, 1))


def test_rows_that_share_memory_are_copied(lib):
    for x in shared_rows(4, 16, half):
        seen = []
        lib.during = lambda name, a, x=x: seen.append(
            [torch.equal(read(p, ld, x), x) and p != x.data_ptr() for p, ld in
             (((a[2], a[3]), (a[5], a[6])) if "norm" in name else ((a[2], a[3]), (a[6], a[7])) if "adapters_run" in name else
              ((a[2], a[3]),))] if name.endswith("_run") else None)
        sk.rms_norm(x, residual=x)
        pool = adapters(n=16)
        sk.add_adapters(x, pool, torch.zeros(4, dtype=torch.int32), x)
        sk.adjust_logits(x, sk.LogitRules(4, 16, history=torch.zeros((4, 3), dtype=torch.int64)))
        assert [s for s in seen if s is not None] == [[True, True], [True, True], [True]]


def test_outputs_that_share_memory_are_refused(lib):
    x = torch.zeros((4, 16), dtype=half)
    for out in shared_rows(4, 16, half):
        for call in (lambda: sk.rms_norm(x, out=out), lambda: sk.rms_norm(x, residual=x, residual_out=out),
                     lambda: sk.add_adapters(x, adapters(n=16), torch.zeros(4, dtype=torch.int32), out=out),
                     lambda: sk.adjust_logits(x, sk.LogitRules(4, 16), out=out)):
            with pytest.raises(ValueError, match="share memory"):
                call()
    assert lib.calls == []


@pytest.mark.parametrize("shape", [(16,), (2, 3, 16), ()])
def test_inputs_that_are_no_matrices_are_refused(lib, shape):
    x, ids = torch.zeros(shape, dtype=half), torch.zeros(3, dtype=torch.int32)
    for name, call in (("x", lambda: sk.rms_norm(x)), ("residual", lambda: sk.rms_norm(torch.zeros((3, 16)), residual=x)),
                       ("x", lambda: sk.add_adapters(x, adapters(), ids)),
                       ("base", lambda: sk.add_adapters(torch.zeros((3, 16), dtype=half), adapters(), ids, x)),
                       ("logits", lambda: sk.adjust_logits(x, sk.LogitRules(3, 16)))):
        with pytest.raises(ValueError, match=f"{name} must be a matrix"):
            call()
    assert lib.calls == []


def test_norm_arguments(lib):
    x, r = torch.zeros((3, 40), dtype=half)[:, :32], torch.zeros((3, 32))
    got = sk.rms_norm(x, torch.ones(32), 1e-5, residual=r, residual_out=r, quant=0)
    (_, a), = lib.calls
    assert a[:5] == (3, 32, x.data_ptr(), 40, sk.BF16) and a[5:8] == (r.data_ptr(), 0, sk.F32) and a[9:13] == (
        sk.F32, 1e-5, r.data_ptr(), 0)
    assert a[13] is None and got.out is None and got.residual is r          # 8 bits only
    assert got.q.dtype is torch.float8_e4m3fn and tuple(got.scales.shape) == (3, 1) and a[19] == 0
    got = sk.rms_norm(x, out_dtype=torch.float16, quant=32)
    assert got.out.dtype is torch.float16 and tuple(got.scales.shape) == (3, 1) and got.residual is None
    got = sk.rms_norm(torch.zeros((2, 130)), quant=64, out_dtype=half)
    assert tuple(got.scales.shape) == (2, 3) and lib.calls[-1][1][19] == 64
    assert sk.rms_norm(x).out.dtype is half


def test_adapter_arguments(lib):
    pool = adapters()
    x, ids = torch.zeros((3, 24), dtype=half)[:, :16], torch.zeros(3, dtype=torch.int64)
    base = torch.zeros((3, 20))[:, 4:16]
    assert sk.add_adapters(x, pool, ids, base, out=base) is base
    _, a = lib.calls[-1]
    assert a[1:4] == (3, x.data_ptr(), 24) and a[4:6] == (ids.data_ptr(), True) and a[6:9] == (base.data_ptr(), 20, sk.F32)
    assert a[9:12] == (base.data_ptr(), 20, sk.F32) and a[13] == 64
    assert sk.add_adapters(x, pool, ids.int(), base).dtype is torch.float32
    assert sk.add_adapters(x, pool, ids.int()).dtype is half and lib.calls[-1][1][6] is None
    assert sk.add_adapters(x, pool, ids.int(), base, out_dtype=half).dtype is half


def test_logit_rule_arguments(lib):
    h, n = torch.zeros((2, 9), dtype=torch.int64)[:, :7], torch.zeros(2, dtype=torch.int32)
    mask = torch.zeros((5, 6), dtype=torch.int32)[:, :4]
    r = sk.LogitRules(2, 100, history=h, lengths=n, presence=n.float(), mask=mask, mask_rows=n)
    d = r._desc
    assert (d.tokens64, d.history, d.ldh, d.history_len, d.lengths, d.prompt_lengths) == (1, h.data_ptr(), 9, 7, n.data_ptr(), None)
    assert (d.mask, d.ldm, d.masks, d.mask_rows, d.biases, d.bias_ids) == (mask.data_ptr(), 6, 5, n.data_ptr(), 0, None)
    x = torch.zeros((2, 100), dtype=half)
    assert sk.adjust_logits(x, r, out=x) is x
    assert sk.adjust_logits(x, r, out_dtype=torch.float32).dtype is torch.float32
    # lists without room are none
    e = sk.LogitRules(2, 100, history=h[:, :0], lengths=n, bias_ids=h[:, :0].int().long().contiguous(),
                      bias_values=torch.zeros((2, 0)))._desc
    assert (e.history, e.history_len, e.lengths, e.biases, e.bias_ids, e.bias_values) == (None, 0, None, 0, None, None)


def test_threads_do_not_enqueue_adapter_runs_at_once(lib):
    """A run is several launches over one workspace: another thread's must not come
    between them."""
    pool, x, ids = adapters(), torch.zeros((3, 16), dtype=half), torch.zeros(3, dtype=torch.int32)
    inside, most = [0], [0]

    def during(name, args):
        if name == "skinny_adapters_run":
            inside[0] += 1
            most[0] = max(most[0], inside[0])
            time.sleep(0.05)  # (as the library's call does, without the interpreter's lock)
            inside[0] -= 1

    lib.during = during
    threads = [threading.Thread(target=sk.add_adapters, args=(x, pool, ids)) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sum(name == "skinny_adapters_run" for name, _ in lib.calls) == 4 and most[0] == 1


def test_the_tensors_gpu_is_current_during_a_call(lib, monkeypatch):
    """The library launches on the current device, whatever the stream's."""
    current, seen = [3], []

    @contextlib.contextmanager
    def device(index):
        was, current[0] = current[0], index
        yield
        current[0] = was

    monkeypatch.setattr(sk, "_current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    lib.during = lambda name, args: seen.append((name, current[0])) if name.endswith("_run") else None
    x = torch.zeros((2, 16), dtype=half)
    sk.rms_norm(x)
    sk.add_adapters(x, adapters(), torch.zeros(2, dtype=torch.int32))
    sk.adjust_logits(x, sk.LogitRules(2, 16, history=torch.zeros((2, 1), dtype=torch.int32)))
    assert seen == [("skinny_rms_norm_run", -1), ("skinny_adapters_run", -1), ("skinny_adjust_logits_run", -1)]
    assert current == [3]
