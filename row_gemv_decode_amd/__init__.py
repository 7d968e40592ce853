"""Thin Python binding of libskinny.so, the MI355X weight-streaming skinny matmul.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI (include/skinny.h).  PyTorch supplies device memory
and the current stream; nothing here computes a result, and there is no CPU
fallback -- importing this package fails loudly when the library is missing.

    C = mm(A, W)                       # f16/bf16 rows x [n][k] weight
    C = mm(A, (qs, d))                 # Q8_0-style weight: int8 codes, f16 scales
                                       # (Q4_0 / Q2_0: packed uint8 codes)
    logits, idx, val = gemv_topk(A, W, topk=10)
    w16 = dequant_q8_0(qs, d)

W is stored [n][k] (k-contiguous): stored row j is column j of the logical
W[k, n] in C[m, n] = A[m, k] . W[k, n].
"""
import ctypes
import os
import threading
from typing import NamedTuple

# torch first: it brings its own HIP runtime (soname libamdhip64.so.7); loaded
# afterwards, libskinny.so binds to that same runtime, so torch's streams and
# device memory are the library's.  Loaded the other way round the process
# would hold two HIP runtimes that do not share devices or streams.
import torch  # noqa: F401

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libskinny.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m row_gemv_decode_amd.build` "
        "(or __graft_entry__.build()); there is no fallback implementation")

_lib = ctypes.CDLL(LIB_PATH)

# --- C ABI mirror -----------------------------------------------------------
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_SHAPE, ERR_HIP, ERR_WORKSPACE, ERR_SCRATCH = range(8)
F16, BF16, F32, Q8_0, Q4_0, Q2_0 = 1, 2, 3, 4, 5, 6
DTYPE_W4 = 7
# stored codes per byte of the block-quantised weight kinds
CODES_PER_BYTE = {Q8_0: 1, Q4_0: 2, Q2_0: 4}
FORCE_GEMV, FORCE_GEMM, GEMM_SPLIT_LAUNCH, GEMM_ONE_LAUNCH = 0x1, 0x2, 0x4, 0x8
EPILOGUE_SIGMOID = 0x10
GEMM_FOLD_LAUNCH = 0x20
GEMV_MAX_M = 16
TOPK_MAX = 32
MOE_RENORM = 0x1
MOE_MAX_EXPERTS = 1024
WINDOW_COUNTER_BYTES = 4096

EXPORTS = (
    "skinny_mm_plan", "skinny_mm_plan_destroy", "skinny_mm_workspace_size", "skinny_mm_run",
    "gemv_topk_run", "skinny_dequant_q8_0_run", "skinny_dequant_q4_0_run", "skinny_dequant_q2_0_run",
    "skinny_mm_plan_info",
    "skinny_gemm_tile_count",
    "skinny_gemm_tile_name", "skinny_status_string", "skinny_abi_version", "skinny_cast_f32_bf16_run",
    "skinny_moe_combine_run", "skinny_mm_run_static",
)
# the entry points of include/skinny_window.h
WINDOW_EXPORTS = (
    "skinny_w4_mm_run",
    "skinny_moe_plan_create", "skinny_moe_plan_destroy", "skinny_moe_workspace_size", "skinny_moe_run",
    "skinny_token_logprobs_workspace_size", "skinny_token_logprobs_run",
)
STATIC_SCRATCH_BYTES = 32 << 20
STATIC_COUNTER_BYTES = 1 << 20


class MMDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("a_dtype", ctypes.c_int32),
        ("w_dtype", ctypes.c_int32),
        ("c_dtype", ctypes.c_int32),
        ("max_m", ctypes.c_int64),
        ("n", ctypes.c_int64),
        ("k", ctypes.c_int64),
        ("lda", ctypes.c_int64),
        ("ldc", ctypes.c_int64),
        ("flags", ctypes.c_uint32),
        ("tile_id", ctypes.c_int32),
        ("num_cus", ctypes.c_int32),
    ]


class W4Desc(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p)]


class MoEDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("w_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("max_m", ctypes.c_int64),
        ("d", ctypes.c_int64),
        ("inter", ctypes.c_int64),
        ("shared_inter", ctypes.c_int64),
        ("experts", ctypes.c_int64),
        ("ldx", ctypes.c_int64),
        ("ldo", ctypes.c_int64),
        ("flags", ctypes.c_uint32),
        ("num_cus", ctypes.c_int32),
    ]


class MoEWeightsDesc(ctypes.Structure):
    _fields_ = [("router", ctypes.c_void_p), ("w13", W4Desc), ("w2", W4Desc), ("shared13", W4Desc),
                ("shared2", W4Desc), ("shared_gate", ctypes.c_void_p)]


_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_lib.skinny_mm_plan.argtypes = [ctypes.POINTER(MMDesc), ctypes.POINTER(_vp)]
_lib.skinny_mm_plan.restype = ctypes.c_int
_lib.skinny_mm_plan_destroy.argtypes = [_vp]
_lib.skinny_mm_plan_destroy.restype = None
_lib.skinny_mm_workspace_size.argtypes = [_vp, ctypes.POINTER(_sz)]
_lib.skinny_mm_workspace_size.restype = ctypes.c_int
_lib.skinny_mm_run.argtypes = [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.skinny_mm_run.restype = ctypes.c_int
_lib.skinny_mm_run_static.argtypes = [_vp, _i64, _vp, _vp, _vp, _vp, _vp]
_lib.skinny_mm_run_static.restype = ctypes.c_int
_lib.gemv_topk_run.argtypes = [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _sz, _vp]
_lib.gemv_topk_run.restype = ctypes.c_int
_lib.skinny_dequant_q8_0_run.argtypes = [_i64, _i64, _vp, _vp, _vp, _vp]
_lib.skinny_dequant_q8_0_run.restype = ctypes.c_int
_lib.skinny_dequant_q4_0_run.argtypes = [_i64, _i64, _vp, _vp, _vp, _vp]
_lib.skinny_dequant_q4_0_run.restype = ctypes.c_int
_lib.skinny_dequant_q2_0_run.argtypes = [_i64, _i64, _vp, _vp, _vp, _vp]
_lib.skinny_dequant_q2_0_run.restype = ctypes.c_int
_lib.skinny_cast_f32_bf16_run.argtypes = [_i64, _vp, _vp, _vp]
_lib.skinny_cast_f32_bf16_run.restype = ctypes.c_int
_lib.skinny_moe_combine_run.argtypes = [_i64, _i64, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _vp]
_lib.skinny_moe_combine_run.restype = ctypes.c_int
_lib.skinny_w4_mm_run.argtypes = [_i64, _i64, _i64, _i32, _vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp]
_lib.skinny_w4_mm_run.restype = ctypes.c_int
_lib.skinny_moe_plan_create.argtypes = [ctypes.POINTER(MoEDesc), ctypes.POINTER(_vp)]
_lib.skinny_moe_plan_create.restype = ctypes.c_int
_lib.skinny_moe_plan_destroy.argtypes = [_vp]
_lib.skinny_moe_plan_destroy.restype = None
_lib.skinny_moe_workspace_size.argtypes = [_vp, ctypes.POINTER(_sz)]
_lib.skinny_moe_workspace_size.restype = ctypes.c_int
_lib.skinny_moe_run.argtypes = [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.skinny_moe_run.restype = ctypes.c_int
_lib.skinny_token_logprobs_workspace_size.argtypes = [_i64, _i64, _i32, ctypes.POINTER(_sz)]
_lib.skinny_token_logprobs_workspace_size.restype = ctypes.c_int
_lib.skinny_token_logprobs_run.argtypes = [_i64, _i64, _vp, _i64, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                           _vp]
_lib.skinny_token_logprobs_run.restype = ctypes.c_int
_lib.skinny_mm_plan_info.argtypes = [_vp, _i64, ctypes.c_char_p, _sz]
_lib.skinny_mm_plan_info.restype = ctypes.c_int
_lib.skinny_gemm_tile_count.argtypes = []
_lib.skinny_gemm_tile_count.restype = _i32
_lib.skinny_gemm_tile_name.argtypes = [_i32]
_lib.skinny_gemm_tile_name.restype = ctypes.c_char_p
_lib.skinny_status_string.argtypes = [ctypes.c_int]
_lib.skinny_status_string.restype = ctypes.c_char_p
_lib.skinny_abi_version.argtypes = []
_lib.skinny_abi_version.restype = _i32


class SkinnyError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = int(status)
        msg = _lib.skinny_status_string(self.status).decode()
        super().__init__(f"{where}: {msg} (status {self.status})" if where else msg)


def _check(status: int, where: str):
    if status != OK:
        raise SkinnyError(status, where)


def lib() -> ctypes.CDLL:
    return _lib


def abi_version() -> int:
    return int(_lib.skinny_abi_version())


def gemm_tiles():
    return [_lib.skinny_gemm_tile_name(i).decode() for i in range(_lib.skinny_gemm_tile_count())]


# --- torch plumbing ---------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t, what):
    torch = _torch()
    if t == torch.float16:
        return F16
    if t == torch.bfloat16:
        return BF16
    if t == torch.float32:
        return F32
    raise TypeError(f"{what}: unsupported dtype {t}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


class Plan:
    """A skinny_mm_plan: host-only, immutable, reusable across streams (the
    workspaces it hands out are kept per device and stream)."""

    def __init__(self, n, k, max_m, a_dtype=F16, w_dtype=F16, c_dtype=F32, lda=0, ldc=0,
                 flags=0, tile_id=-1, num_cus=0):
        d = MMDesc(ctypes.sizeof(MMDesc), a_dtype, w_dtype, c_dtype, max_m, n, k, lda, ldc,
                   flags, tile_id, num_cus)
        h = ctypes.c_void_p()
        _check(_lib.skinny_mm_plan(ctypes.byref(d), ctypes.byref(h)), "skinny_mm_plan")
        self._h = h
        self.n, self.k, self.max_m = n, k, max_m
        self.a_dtype, self.w_dtype, self.c_dtype = a_dtype, w_dtype, c_dtype
        self.lda, self.ldc = lda or k, ldc or n
        sz = ctypes.c_size_t()
        _check(_lib.skinny_mm_workspace_size(self._h, ctypes.byref(sz)), "skinny_mm_workspace_size")
        self.workspace_bytes = int(sz.value)
        self._ws = {}

    @property
    def handle(self):
        return self._h

    def info(self, m: int) -> str:
        buf = ctypes.create_string_buffer(256)
        _check(_lib.skinny_mm_plan_info(self._h, m, buf, 256), "skinny_mm_plan_info")
        return buf.value.decode()

    def workspace(self, device, stream=None):
        """A zero-initialised device workspace of this plan for one (device,
        stream) pair (None when none is needed).  Runs on one stream are
        ordered, so they may share it; runs on different streams may be in
        flight at once and must not (the workspace holds arrival counters and
        partial sums), so every stream gets its own.  It is allocated and
        zero-filled on that stream, so the fill precedes the stream's first
        run.  Each plan keeps its own: one plan's counters must not be
        overwritten by another plan's partial sums."""
        if self.workspace_bytes == 0:
            return None
        torch = _torch()
        dev = torch.device(device)
        if stream is None:
            stream = torch.cuda.current_stream(dev)
        key = (str(dev), int(stream.cuda_stream))
        ws = self._ws.get(key)
        if ws is None:
            with torch.cuda.stream(stream):
                ws = torch.zeros(self.workspace_bytes, dtype=torch.uint8, device=dev)
            self._ws[key] = ws
        return ws

    def _resolve(self, A, workspace, stream):
        torch = _torch()
        if stream is None:
            stream = torch.cuda.current_stream(A.device)
        ws = workspace if workspace is not None else self.workspace(A.device, stream)
        nbytes = 0 if ws is None else ws.numel() * ws.element_size()
        return ws, nbytes, ctypes.c_void_p(stream.cuda_stream)

    def run(self, m, A, W, C, scales=None, workspace=None, stream=None):
        ws, nbytes, st = self._resolve(A, workspace, stream)
        _check(_lib.skinny_mm_run(self._h, m, _ptr(A), _ptr(W), _ptr(scales), _ptr(C), _ptr(ws),
                                  nbytes, st), "skinny_mm_run")

    def run_topk(self, m, A, W, logits, idx, val, topk, scales=None, workspace=None, stream=None):
        ws, nbytes, st = self._resolve(A, workspace, stream)
        _check(_lib.gemv_topk_run(self._h, m, _ptr(A), _ptr(W), _ptr(scales), _ptr(logits),
                                  _ptr(idx), _ptr(val), topk, _ptr(ws), nbytes, st),
               "gemv_topk_run")

    def run_static(self, m, A, W, C, scales=None, stream=None):
        """skinny_mm_run_static: the run without a workspace argument (the
        library's own static scratch; calls in flight at once on one GPU race)."""
        torch = _torch()
        if stream is None:
            stream = torch.cuda.current_stream(A.device)
        _check(_lib.skinny_mm_run_static(self._h, m, _ptr(A), _ptr(W), _ptr(scales), _ptr(C),
                                         ctypes.c_void_p(stream.cuda_stream)), "skinny_mm_run_static")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            try:
                _lib.skinny_mm_plan_destroy(h)
            except Exception:  # interpreter shutdown
                pass
            self._h = None


def new_workspace(plan, device):
    """A fresh zero-filled workspace for `plan` (None when it needs none)."""
    torch = _torch()
    if plan.workspace_bytes == 0:
        return None
    return torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=device)


_plan_cache = {}


def _dense(where, **tensors):
    """The library reads every tensor as a dense row-major block: reject views
    with other strides instead of reading them wrongly."""
    for name, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous (pass a Plan with lda/ldc for strided rows)")


def _weight_kind(W, k):
    """(dtype code, weight or codes, scales or None) of a weight for reduction
    length k.  Packed uint8 codes are Q4_0 when a row holds k/2 bytes and
    Q2_0 when it holds k/4."""
    torch = _torch()
    if isinstance(W, tuple):
        qs, d = W
        if qs.dtype not in (torch.int8, torch.uint8) or d.dtype != torch.float16 or qs.dim() != 2:
            raise TypeError("a block-quantised weight is (int8 codes [n][k] (Q8_0), or uint8 packed "
                            "4-bit codes [n][k/2] (Q4_0) or 2-bit codes [n][k/4] (Q2_0), float16 "
                            "scales [n][k/32])")
        if qs.dtype == torch.int8:
            kind = Q8_0
        else:
            kind = Q4_0 if 2 * qs.shape[1] == k else Q2_0
        if qs.shape[1] * CODES_PER_BYTE[kind] != k or tuple(d.shape) != (qs.shape[0], k // 32):
            raise ValueError(f"block-quantised weight: codes {tuple(qs.shape)} and scales {tuple(d.shape)} "
                             f"do not fit k = {k}")
        _dense("block-quantised weight", codes=qs, scales=d)
        return kind, qs, d
    _dense("weight", W=W)
    return _dtype_code(W.dtype, "W"), W, None


def get_plan(n, k, max_m, a_dtype, w_dtype, c_dtype, flags=0, tile_id=-1) -> Plan:
    key = (n, k, max_m, a_dtype, w_dtype, c_dtype, flags, tile_id)
    p = _plan_cache.get(key)
    if p is None:
        p = Plan(n, k, max_m, a_dtype, w_dtype, c_dtype, flags=flags, tile_id=tile_id)
        _plan_cache[key] = p
    return p


def mm(A, W, out=None, out_dtype=None, flags=0, tile_id=-1, max_m=None, stream=None):
    """C = A . W^T_storage for A [m][k] (f16/bf16, contiguous rows) and W [n][k]
    (same dtype), or W = (qs int8 [n][k], d f16 [n][k/32]) for Q8_0, or
    W = (qs uint8 [n][k/2] packed 4-bit codes, d f16 [n][k/32]) for Q4_0, or
    W = (qs uint8 [n][k/4] packed 2-bit codes, d f16 [n][k/32]) for Q2_0."""
    torch = _torch()
    m, k = A.shape
    wk, Wt, scales = _weight_kind(W, k)
    n = Wt.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or torch.float32, device=A.device)
    _dense("mm", A=A, out=out)
    plan = get_plan(n, k, max_m or m, _dtype_code(A.dtype, "A"), wk, _dtype_code(out.dtype, "C"),
                    flags, tile_id)
    plan.run(m, A, Wt, out, scales=scales, stream=stream)
    return out


def gemv_topk(A, W, topk=10, flags=0, max_m=None, stream=None):
    """(logits f32 [m][n], idx int32 [m][topk], val f32 [m][topk]) of the router step."""
    torch = _torch()
    m, k = A.shape
    wk, Wt, scales = _weight_kind(W, k)
    n = Wt.shape[0]
    logits = torch.empty((m, n), dtype=torch.float32, device=A.device)
    idx = torch.empty((m, topk), dtype=torch.int32, device=A.device)
    val = torch.empty((m, topk), dtype=torch.float32, device=A.device)
    _dense("gemv_topk", A=A)
    plan = get_plan(n, k, max_m or m, _dtype_code(A.dtype, "A"), wk, F32, flags)
    plan.run_topk(m, A, Wt, logits, idx, val, topk, scales=scales, stream=stream)
    return logits, idx, val


def dequant_q2_0(qs, d, out=None, stream=None):
    """f16 [n][k] weight of a Q2_0-style (packed codes uint8 [n][k/4], scales) pair."""
    torch = _torch()
    n, kq = qs.shape
    if out is None:
        out = torch.empty((n, 4 * kq), dtype=torch.float16, device=qs.device)
    _dense("dequant_q2_0", qs=qs, d=d, out=out)
    _check(_lib.skinny_dequant_q2_0_run(n, 4 * kq, _ptr(qs), _ptr(d), _ptr(out), _stream(stream)),
           "skinny_dequant_q2_0_run")
    return out


def dequant_q4_0(qs, d, out=None, stream=None):
    """f16 [n][k] weight of a Q4_0-style (packed codes uint8 [n][k/2], scales) pair."""
    torch = _torch()
    n, kh = qs.shape
    if out is None:
        out = torch.empty((n, 2 * kh), dtype=torch.float16, device=qs.device)
    _dense("dequant_q4_0", qs=qs, d=d, out=out)
    _check(_lib.skinny_dequant_q4_0_run(n, 2 * kh, _ptr(qs), _ptr(d), _ptr(out), _stream(stream)),
           "skinny_dequant_q4_0_run")
    return out


def dequant_q8_0(qs, d, out=None, stream=None):
    """f16 [n][k] weight of a Q8_0-style (codes, scales) pair."""
    torch = _torch()
    n, k = qs.shape
    if out is None:
        out = torch.empty((n, k), dtype=torch.float16, device=qs.device)
    _dense("dequant_q8_0", qs=qs, d=d, out=out)
    _check(_lib.skinny_dequant_q8_0_run(n, k, _ptr(qs), _ptr(d), _ptr(out), _stream(stream)),
           "skinny_dequant_q8_0_run")
    return out


def cast_f32_bf16(x, out=None, stream=None):
    """bf16 copy of a contiguous fp32 tensor (round to nearest even), one launch."""
    torch = _torch()
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise TypeError("cast_f32_bf16 takes a contiguous float32 tensor")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _check(_lib.skinny_cast_f32_bf16_run(x.numel(), _ptr(x), _ptr(out), _stream(stream)),
           "skinny_cast_f32_bf16_run")
    return out


def moe_combine(rows, weights, shared=None, gate=None, out=None, out_dtype=None, stream=None):
    """MoE combine: out[t] = sum_i weights[t][i] * rows[t][i] (+ gate[t] * shared[t]),
    rows [m][topk][d] float32 or bfloat16 (contiguous), weights float32 [m][topk],
    shared [m][d] like rows and gate float32 [m] (both or neither); one launch."""
    torch = _torch()
    m, topk, d = rows.shape
    if out is None:
        out = torch.empty((m, d), dtype=out_dtype or torch.float32, device=rows.device)
    _dense("moe_combine", rows=rows, weights=weights, shared=shared, gate=gate, out=out)
    if weights.dtype != torch.float32 or tuple(weights.shape) != (m, topk):
        raise ValueError("moe_combine: weights must be float32 [m][topk]")
    if shared is not None and (tuple(shared.shape) != (m, d) or shared.dtype != rows.dtype):
        raise ValueError("moe_combine: shared must be [m][d] with the rows' dtype")
    if gate is not None and (gate.dtype != torch.float32 or tuple(gate.shape) != (m,)):
        raise ValueError("moe_combine: gate must be float32 [m]")
    if tuple(out.shape) != (m, d):
        raise ValueError("moe_combine: out must be [m][d]")
    _check(_lib.skinny_moe_combine_run(m, d, topk, _ptr(rows), _ptr(weights), _ptr(shared), _ptr(gate),
                                       _dtype_code(rows.dtype, "rows"), _ptr(out),
                                       _dtype_code(out.dtype, "out"), _stream(stream)),
           "skinny_moe_combine_run")
    return out


def gate(A, W, max_m=None, out=None, stream=None):
    """Scalar gate of fp32 window rows: sigmoid(bf16(A) . W) for A [m][k] fp32
    (contiguous rows) and W bf16 [n][k] (n = 1 for one gate per row), in one
    GEMV launch that rounds A to bf16 as it loads it and applies the sigmoid
    as it stores."""
    torch = _torch()
    m, k = A.shape
    n = W.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=A.device)
    _dense("gate", A=A, out=out)
    plan = get_plan(n, k, max_m or m, _dtype_code(A.dtype, "A"), _dtype_code(W.dtype, "W"),
                    _dtype_code(out.dtype, "C"), EPILOGUE_SIGMOID)
    plan.run(m, A, W, out, stream=stream)
    return out


class W4:
    """A 4-bit grouped weight [n][k] (or a stack [e][n][k]): packed codes uint8
    [n][k/2] (element kk in byte kk/2, the low nibble for even kk), scales
    [n][k/g] in the rows' 16-bit type for groups of g = 32, 64 or 128 along k,
    and zero points uint8 [n][k/g] (None: 8 everywhere);
    weight = scale * (code - zero).  Checked once, here; the tensors are kept
    alive and read at every call."""

    __slots__ = ("codes", "scales", "zeros", "shape", "group", "dtype", "device", "_desc", "_addr", "_index")

    def __init__(self, codes, scales, zeros=None):
        if codes.dtype != torch.uint8 or scales.dtype not in (torch.float16, torch.bfloat16) or \
                (zeros is not None and zeros.dtype != torch.uint8):
            raise TypeError("W4: uint8 codes, float16 or bfloat16 scales, uint8 zero points (or None)")
        if codes.dim() < 2 or scales.dim() != codes.dim() or codes.shape[:-1] != scales.shape[:-1]:
            raise ValueError(f"W4: scales {tuple(scales.shape)} do not fit codes {tuple(codes.shape)}")
        k, groups = 2 * codes.shape[-1], scales.shape[-1]
        if groups < 1 or k % groups or k // groups not in (32, 64, 128):
            raise ValueError(f"W4: {groups} scales for {k} elements: groups of 32, 64 or 128 are taken")
        if zeros is not None and zeros.shape != scales.shape:
            raise ValueError(f"W4: zero points {tuple(zeros.shape)} do not fit scales {tuple(scales.shape)}")
        _dense("W4", codes=codes, scales=scales, zeros=zeros)
        _on("W4", codes.device, scales, zeros)
        self.codes, self.scales, self.zeros = codes, scales, zeros
        self.shape, self.group = (*codes.shape[:-1], k), k // groups
        self.dtype, self.device = scales.dtype, codes.device
        self._desc = W4Desc(codes.data_ptr(), scales.data_ptr(), 0 if zeros is None else zeros.data_ptr())
        self._addr = ctypes.addressof(self._desc)
        self._index = codes.get_device()


def _on(where, device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"{where}: every tensor must be on {device}, got one on {t.device}")


def _rows(where, name, t):
    """Row stride of a matrix whose rows are dense and lie apart (0: a single
    row, which the library takes as a dense one)."""
    shape = t.shape
    if len(shape) != 2 or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{where}: {name} must be a matrix with contiguous rows")
    if shape[0] < 2:
        return 0
    ld = t.stride(0)
    if ld < shape[1]:
        raise ValueError(f"{where}: {name}'s rows of {shape[1]} elements share memory (row stride {ld})")
    return ld


def _input_rows(where, name, t, stream):
    """(t, its row stride) of an input.  Rows that share memory (a row expanded
    to several, windows that overlap) are copied apart on the stream that reads
    them: the library takes no row stride below the rows' length."""
    shape = t.shape
    if len(shape) == 2:
        ld, step = t.stride()
        if step == 1:
            if shape[0] < 2:
                return t, 0
            if ld >= shape[1]:
                return t, ld
            if stream is None:
                t = t.contiguous()
            else:
                with torch.cuda.stream(stream):
                    t = t.contiguous()
    return t, _rows(where, name, t)


# A window's calls take a few microseconds on the GPU, so what the host does
# for each of them counts: types are looked up, streams come as raw handles.
_CODES = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
_raw_stream = torch._C._cuda_getCurrentRawStream
# (the library launches on the current device: a call whose tensors lie on
# another GPU makes that one current first)
_current_device = torch._C._cuda_getDevice


def _handle(index, stream):
    """Raw handle of `stream`, or of the current stream of GPU `index`."""
    return _raw_stream(index) if stream is None else stream.cuda_stream


def _gpu(where, t):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{where}: tensors must be on a GPU")
    return index


def _empty(shape, dtype, device, stream):
    """An output, allocated on the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


# (from the HIP runtime that the library is linked with)
_is_capturing = _lib.hipStreamIsCapturing
_is_capturing.argtypes = [_vp, ctypes.POINTER(ctypes.c_int)]
_is_capturing.restype = ctypes.c_int


def _capturing(handle):
    """Whether a stream is being captured (the default stream, handle 0, cannot be)."""
    if handle == 0:
        return False
    status = ctypes.c_int()
    if _is_capturing(handle, ctypes.byref(status)) != 0:
        raise SkinnyError(ERR_HIP, "hipStreamIsCapturing")
    return status.value != 0


def _stream_workspace(cache, key, nbytes, counters, device, handle, stream):
    """The workspace of at least nbytes that `cache` holds for a stream, made
    and zeroed on that stream (a run leaves its counters at zero).  A capture
    always gets one of its own, from the graph's memory, whose first `counters`
    bytes the graph zeroes at every replay: the stream's may be replaced by a
    larger one, and eager runs may use it, while the graph lives."""
    capturing = _capturing(handle)
    ws = None if capturing else cache.get(key)
    if ws is None or ws.numel() < nbytes:
        with torch.cuda.stream(torch.cuda.current_stream(device) if stream is None else stream):
            if capturing:
                ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
                if counters:
                    ws[:counters].zero_()
            else:
                ws = cache[key] = torch.zeros(nbytes, dtype=torch.uint8, device=device)
    return ws


def mm_w4(A, W, out=None, out_dtype=None, stream=None):
    """C = A . W for A [m][k] (m <= 16, float16 or bfloat16, dense rows of any
    stride that is a multiple of 8) and a 4-bit grouped weight W (a W4 whose
    scales have A's type), in one launch; C is float32 unless `out` or
    `out_dtype` says otherwise.  Rows of A that share memory (A.expand(m, k) of
    one row) are copied apart first; those of `out` must not."""
    A, lda = _input_rows("mm_w4", "A", A, stream)
    m, k = A.shape
    dtype = A.dtype
    if not isinstance(W, W4) or W.dtype is not dtype:
        raise TypeError(f"mm_w4: the weight must be a W4 with scales of A's type ({dtype})")
    if len(W.shape) != 2 or W.shape[1] != k:
        raise ValueError(f"mm_w4: a weight {W.shape} does not fit k = {k}")
    n = W.shape[0]
    index = _gpu("mm_w4", A)
    if W._index != index:
        raise ValueError(f"mm_w4: A is on {A.device}, the weight on {W.device}")
    if _current_device() != index:
        with torch.cuda.device(index):
            return mm_w4(A, W, out, out_dtype, stream)
    if out is None:
        out_dtype = out_dtype or torch.float32
        out = _empty((m, n), out_dtype, W.device, stream)
        ldc = n
    else:
        ldc = _rows("mm_w4", "out", out)
        out_dtype = out.dtype
        if tuple(out.shape) != (m, n):
            raise ValueError("mm_w4: out must be [m][n]")
        _on("mm_w4", W.device, out)
    _check(_lib.skinny_w4_mm_run(m, n, k, W.group, A.data_ptr(), lda, _CODES[dtype], W._addr, out.data_ptr(), ldc,
                                 _CODES.get(out_dtype, 0), _handle(index, stream)), "skinny_w4_mm_run")
    return out


class MoELayer:
    """A whole mixture-of-experts layer for decode windows of up to max_m <= 16
    tokens: router, top-k and softmax (renormalised over the top-k when
    `renorm`), the routed experts' gated products silu(gate) * up, the optional
    shared expert behind sigmoid(x . shared_gate), and the weighted sum.

        layer = MoELayer(router, w13, w2, topk=10)
        out = layer(x)                               # x [m][d] -> out [m][d]

    router [experts][d] float16 or bfloat16; w13 [experts][2 inter][d] (each
    expert's gate rows, then its up rows) and w2 [experts][d][inter], tensors
    of the router's type or both W4 of one group length; shared13
    [2 shared_inter][d] and shared2 [d][shared_inter] likewise, with
    shared_gate [d].  x is contiguous and has the router's type; out has
    out_dtype (x's type by default).  Several threads may call a layer at once."""

    def __init__(self, router, w13, w2, topk, renorm=True, out_dtype=None, max_m=16, shared13=None, shared2=None,
                 shared_gate=None, num_cus=0):
        if router.dim() != 2 or router.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("MoELayer: router must be a float16 or bfloat16 matrix [experts][d]")
        experts, d = router.shape
        dtype, device = router.dtype, router.device
        w4 = isinstance(w13, W4)
        if len(w13.shape) != 3 or w13.shape[1] % 2:
            raise ValueError("MoELayer: w13 must be [experts][2 inter][d]")
        inter = w13.shape[1] // 2
        shared = [t is not None for t in (shared13, shared2, shared_gate)]
        if any(shared) != all(shared):
            raise ValueError("MoELayer: shared13, shared2 and shared_gate go together")
        shared_inter = 0
        if all(shared):
            if len(shared13.shape) != 2 or shared13.shape[0] % 2 or shared13.shape[0] < 2:
                raise ValueError("MoELayer: shared13 must be [2 shared_inter][d]")
            shared_inter = shared13.shape[0] // 2
            if tuple(shared_gate.shape) != (d,) or shared_gate.dtype != dtype:
                raise ValueError("MoELayer: shared_gate must be [d] of the router's type")
        group = w13.group if w4 else 0
        descs = []
        for name, w, shape in (("w13", w13, (experts, 2 * inter, d)), ("w2", w2, (experts, d, inter)),
                               ("shared13", shared13, (2 * shared_inter, d)), ("shared2", shared2, (d, shared_inter))):
            if w is None:
                descs.append(W4Desc())
                continue
            if isinstance(w, W4) != w4 or w.dtype != dtype or (w4 and w.group != group):
                raise TypeError(f"MoELayer: {name} must be a weight of the router's type, like the others")
            if tuple(w.shape) != shape:
                raise ValueError(f"MoELayer: {name} is {tuple(w.shape)}, not {shape}")
            if not w4:
                _dense("MoELayer", **{name: w})
            _on("MoELayer", device, w)
            descs.append(W4Desc(w._desc.codes, w._desc.scales, w._desc.zeros) if w4 else W4Desc(w.data_ptr()))
        _dense("MoELayer", router=router, shared_gate=shared_gate)
        _on("MoELayer", device, shared_gate)
        self._keep = (router, w13, w2, shared13, shared2, shared_gate)
        self.experts, self.d, self.inter, self.shared_inter, self.topk = experts, d, inter, shared_inter, topk
        self.dtype, self.device, self.max_m = dtype, device, max_m
        self.out_dtype = out_dtype or dtype
        self._index = _gpu("MoELayer", router)
        self._weights = MoEWeightsDesc(router.data_ptr(), *descs, shared_gate.data_ptr() if shared_inter else None)
        self._weights_addr = ctypes.addressof(self._weights)
        code = _dtype_code(dtype, "router")
        desc = MoEDesc(ctypes.sizeof(MoEDesc), code, DTYPE_W4 if w4 else code, _dtype_code(self.out_dtype, "out"), group,
                       topk, max_m, d, inter, shared_inter, experts, 0, 0, MOE_RENORM if renorm else 0, num_cus)
        self._h = None
        h = ctypes.c_void_p()
        _check(_lib.skinny_moe_plan_create(ctypes.byref(desc), ctypes.byref(h)), "skinny_moe_plan_create")
        self._h = h
        sz = ctypes.c_size_t()
        _check(_lib.skinny_moe_workspace_size(h, ctypes.byref(sz)), "skinny_moe_workspace_size")
        self.workspace_bytes = int(sz.value)
        # (the layer's only counters are its router GEMV's, where that splits k over workgroups)
        self._counters = WINDOW_COUNTER_BYTES if Plan(experts, d, max_m, code, code, F32).workspace_bytes else 0
        self._ws = {}
        self._lock = threading.Lock()

    def __call__(self, x, out=None, topk_idx=None, topk_weight=None, stream=None):
        """out [m][d]; topk_idx (int32 [m][topk]) and topk_weight (float32
        [m][topk]) receive the routing when given."""
        shape = x.shape
        if len(shape) != 2 or shape[1] != self.d or x.dtype is not self.dtype or not x.is_contiguous():
            raise ValueError(f"MoELayer: x must be contiguous [m][{self.d}] of type {self.dtype}")
        if x.get_device() != self._index:
            raise ValueError(f"MoELayer: x must be on {self.device}")
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self(x, out, topk_idx, topk_weight, stream)
        m = shape[0]
        if out is None:
            out = _empty((m, self.d), self.out_dtype, self.device, stream)
        else:
            if tuple(out.shape) != (m, self.d) or out.dtype != self.out_dtype:
                raise ValueError(f"MoELayer: out must be [{m}][{self.d}] of type {self.out_dtype}")
            _dense("MoELayer", out=out)
            _on("MoELayer", self.device, out)
        if topk_idx is not None or topk_weight is not None:
            for name, t, dt in (("topk_idx", topk_idx, torch.int32), ("topk_weight", topk_weight, torch.float32)):
                if t is not None:
                    if tuple(t.shape) != (m, self.topk) or t.dtype != dt:
                        raise ValueError(f"MoELayer: {name} must be {dt} [{m}][{self.topk}]")
                    _dense("MoELayer", **{name: t})
                    _on("MoELayer", self.device, t)
        handle = _handle(self._index, stream)
        # Runs on different streams may be in flight at once: each stream has its
        # own workspace.  A run is several launches over it, so two threads on one
        # stream must not interleave theirs.
        with self._lock:
            ws = _stream_workspace(self._ws, handle, self.workspace_bytes, self._counters, self.device, handle, stream)
            _check(_lib.skinny_moe_run(self._h, m, x.data_ptr(), self._weights_addr, out.data_ptr(), _ptr(topk_idx),
                                       _ptr(topk_weight), ws.data_ptr(), self.workspace_bytes, handle), "skinny_moe_run")
        return out

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            try:
                _lib.skinny_moe_plan_destroy(h)
            except Exception:  # interpreter shutdown
                pass
            self._h = None


class TokenLogprobs(NamedTuple):
    """What token_logprobs gives: per row the token's log probability, the
    distribution's entropy in nats, the token's rank (1: the largest logit),
    and the top alternatives' ids and log probabilities.  The five share one
    allocation."""
    logprob: "torch.Tensor"       # float32 [m]
    entropy: "torch.Tensor"       # float32 [m]
    rank: "torch.Tensor"          # int32 [m]
    top_ids: "torch.Tensor"       # int32 [m][topk]
    top_logprobs: "torch.Tensor"  # float32 [m][topk]


_logprob_need = {}  # (m, vocab, topk) -> workspace bytes
_logprob_ws = {}


def token_logprobs(logits, tokens, topk=0, stream=None):
    """Log probabilities of tokens[i] under softmax(logits[i]), with entropy,
    rank and the topk <= 32 top alternatives (see TokenLogprobs), in one launch
    that reads the logits once.  logits [m][vocab] float32, float16 or bfloat16
    with dense rows of any stride (rows that share memory, as in scoring several
    tokens of one row by row.expand(m, vocab), are copied apart first); tokens
    [m] int64 or int32.  A logit of -inf is masked out; a token outside the row
    gives NaN and rank 0."""
    logits, ld = _input_rows("token_logprobs", "logits", logits, stream)
    m, vocab = logits.shape
    t64 = tokens.dtype is torch.int64
    if tuple(tokens.shape) != (m,) or not (t64 or tokens.dtype is torch.int32) or not tokens.is_contiguous():
        raise ValueError(f"token_logprobs: tokens must be contiguous int64 or int32 [{m}]")
    dtype = _CODES.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"token_logprobs: unsupported dtype {logits.dtype}")
    index = _gpu("token_logprobs", logits)
    if tokens.get_device() != index:
        raise ValueError("token_logprobs: logits and tokens must be on one GPU")
    if _current_device() != index:
        with torch.cuda.device(index):
            return token_logprobs(logits, tokens, topk, stream)
    need = _logprob_need.get((m, vocab, topk))
    if need is None:
        sz = ctypes.c_size_t()
        _check(_lib.skinny_token_logprobs_workspace_size(m, vocab, topk, ctypes.byref(sz)), "token_logprobs")
        if len(_logprob_need) > 4096:
            _logprob_need.clear()
        need = _logprob_need[m, vocab, topk] = int(sz.value)
    handle = _handle(index, stream)
    ws = None
    if need:
        ws = _stream_workspace(_logprob_ws, (index, handle), need, WINDOW_COUNTER_BYTES, logits.device, handle, stream)
    # one allocation for the five results, each at a multiple of 4 bytes
    flat = _empty(m * (3 + 2 * topk), torch.float32, logits.device, stream)
    lp, ent, top, rank, ids = flat.split_with_sizes((m, m, m * topk, m, m * topk))
    p = flat.data_ptr()
    p_rank = p + 4 * m * (2 + topk)
    _check(_lib.skinny_token_logprobs_run(m, vocab, logits.data_ptr(), ld, dtype, tokens.data_ptr(), t64, topk, p, p + 4 * m,
                                          p_rank, p_rank + 4 * m, p + 8 * m, None if ws is None else ws.data_ptr(), need, handle),
           "skinny_token_logprobs_run")
    return TokenLogprobs(lp, ent, rank.view(torch.int32), ids.view(torch.int32).view(m, topk), top.view(m, topk))
