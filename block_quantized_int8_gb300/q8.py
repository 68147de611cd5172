"""Thin ctypes binding of libq8 (include/q8.h): argument marshalling only.

Every entry point takes torch CUDA tensors, passes their device pointers and
the current (or given) CUDA stream to the C ABI, and raises ``Q8Error`` on a
non-OK status.  There is no fallback: if ``libq8.so`` is missing or a call
fails, the call raises.  Outputs may be pre-allocated by the caller or are
allocated here with torch (device memory is the only thing torch is used for).

Tensor conventions (raw bits are accepted in any 16-bit dtype):
  q  int8 [N, K]           codes
  s  16-bit [N, K/32]      binary16 scale bits (torch.float16 or int16/uint16)
  x  16-bit [M, K]         bf16 activation bits (torch.bfloat16 or int16/uint16)
  y  float32 [M, N]        (bf16 [M, N] for q8_gemm)
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libq8.so")

Q8_OK = 0
Q8_ERR_ARG, Q8_ERR_ALIGN, Q8_ERR_SHAPE, Q8_ERR_WORKSPACE, Q8_ERR_ARCH, Q8_ERR_CUDA, Q8_ERR_UNSUPPORTED = range(1, 8)
Q8_DEV_NONFINITE = 0x1
Q8_DEV_SCALE_OVF = 0x2
Q8_DEV_TIMEOUT = 0x4
Q8_DEV_BAD_INDEX = 0x8
Q8_DEV_NO_PAGE = 0x10
Q8_DTYPE_F32, Q8_DTYPE_BF16 = 0, 1
Q8_SKINNY_MAX_M = 32
Q8_MAX_BATCH = 64
Q8_VARIANT_AUTO, Q8_VARIANT_SIMT, Q8_VARIANT_MMA, Q8_VARIANT_BATCH_INVARIANT, Q8_VARIANT_W8A8 = 0, 1, 2, 3, 4
Q8_GEMM_TILE_AUTO, Q8_GEMM_TILE_256x128, Q8_GEMM_TILE_128x128, Q8_GEMM_TILE_64x128 = 0, 1, 2, 3
Q8_GEMM_MAX_SPLITS = 8
Q8_ATTN_ZEROED_BYTES, Q8_MOE_ZEROED_BYTES, Q8_CHUNK_ZEROED_BYTES = 16384, 256, 4096
Q8_QUANT_EXACT, Q8_QUANT_FL32 = 0, 1
Q8_NORM_MAX_WIDTH = 32768
Q8_ROPE_HALF, Q8_ROPE_INTERLEAVED = 0, 1
Q8_ROPE_MAX_FREQ = 65536.0
Q8_PLAN_MAX_BATCH = 1 << 20

EXPORTS = ("q8_quantize_rows", "q8_gemv", "q8_gemm_skinny", "q8_linear_batch", "q8_linear_batch_ex",
           "q8_linear_batch_chained", "q8_workspace_size", "q8_linear_batch_workspace_size", "q8_linear_batch_workspace_size_ex", "q8_gemm", "q8_status_str",
           "q8_abi_version", "q8_gemm_skinny_noalloc", "q8_gemm_ex", "q8_gguf_to_planar",
           "q8_planar_to_gguf", "q8_quantize_rows_ex", "q8_selftest_wait_timeout",
           "q8_stream_read", "q8_stream_read_out_words", "q8_linear_chain", "q8_linear_chain_workspace_size",
           "q8_gemm_w8a8", "q8_gemm_w8a8_workspace_size", "q8_kv_append", "q8_kv_read", "q8_attn_decode",
           "q8_attn_decode_workspace_size", "q8_moe", "q8_moe_workspace_size",
           "q8_sample", "q8_workspace_zero", "q8_rms_norm", "q8_rope_turns", "q8_rope", "q8_rope_append", "q8_kv_plan",
           "q8_attn_chunk", "q8_attn_chunk_workspace_size")
Q8_NOALLOC_SCRATCH_BYTES = 4 << 20


class Q8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} (status {status})")


class LinearDesc(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class ChainStep(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64), ("next", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _CKvCache(ctypes.Structure):
    _fields_ = [("kq", ctypes.c_void_p), ("ks", ctypes.c_void_p), ("vq", ctypes.c_void_p), ("vs", ctypes.c_void_p),
                ("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


# how the next step of a chain takes its x from this step's y
Q8_CHAIN_END = 0
Q8_CHAIN_RMSNORM = 1
Q8_CHAIN_SWIGLU_RMSNORM = 2
Q8_MAX_CHAIN = 4096

_lib = None


def lib():
    """Load libq8.so from the package directory (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m block_quantized_int8_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, SZ, U32P = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
        L.q8_quantize_rows.argtypes = [P, I64, I64, P, P, U32P, P]
        L.q8_quantize_rows_ex.argtypes = [P, I64, I64, P, P, I32, U32P, P]
        L.q8_gemv.argtypes = [P, P, I64, I64, P, P, P, SZ, U32P, P]
        L.q8_gemm_skinny.argtypes = [P, P, I64, I64, P, I64, I32, P, I64, P, SZ, U32P, P]
        L.q8_linear_batch.argtypes = [ctypes.POINTER(LinearDesc), I32, I32, P, SZ, U32P, P]
        L.q8_linear_batch_ex.argtypes = [ctypes.POINTER(LinearDesc), I32, I32, I32, P, SZ, U32P, P]
        L.q8_linear_batch_chained.argtypes = [ctypes.POINTER(LinearDesc), I32, I32, P, SZ, U32P, P]
        L.q8_workspace_size.argtypes = [I64, I64, I32]
        L.q8_workspace_size.restype = SZ
        L.q8_linear_batch_workspace_size.argtypes = [ctypes.POINTER(LinearDesc), I32, I32]
        L.q8_linear_batch_workspace_size.restype = SZ
        L.q8_linear_batch_workspace_size_ex.argtypes = [ctypes.POINTER(LinearDesc), I32, I32, I32]
        L.q8_linear_batch_workspace_size_ex.restype = SZ
        L.q8_linear_chain.argtypes = [ctypes.POINTER(ChainStep), I32, I32, P, SZ, U32P, P]
        L.q8_linear_chain_workspace_size.argtypes = [ctypes.POINTER(ChainStep), I32, I32]
        L.q8_linear_chain_workspace_size.restype = SZ
        L.q8_gemm_w8a8.argtypes = [P, P, I64, I64, P, I64, I32, P, I64, P, SZ, U32P, P]
        L.q8_gemm_w8a8_workspace_size.argtypes = [I64, I64, I32]
        L.q8_gemm_w8a8_workspace_size.restype = SZ
        L.q8_gemm.argtypes = [P, P, I64, I64, P, I64, I32, P, I64, U32P, P]
        L.q8_gemm_ex.argtypes = [P, P, I64, I64, P, I64, I32, P, I64, I32, I32, U32P, P]
        L.q8_gemm_skinny_noalloc.argtypes = [P, P, I64, I64, P, I64, I32, P, I64, U32P, P]
        L.q8_gguf_to_planar.argtypes = [P, I64, I64, P, P, P]
        L.q8_planar_to_gguf.argtypes = [P, P, I64, I64, P, P]
        L.q8_selftest_wait_timeout.argtypes = [ctypes.c_uint64, U32P, P, P]
        L.q8_selftest_wait_timeout.restype = ctypes.c_int
        L.q8_stream_read.argtypes = [P, SZ, P, P]
        L.q8_stream_read.restype = ctypes.c_int
        L.q8_stream_read_out_words.restype = SZ
        L.q8_kv_append.argtypes = [P, P, P, I64, I64, I32, P, I64, P, P]
        L.q8_kv_read.argtypes = [P, P, I64, P, P, I64, I64, I32, P, P]
        L.q8_attn_decode.argtypes = [P, P, I64, I32, P, I32, P, I32, ctypes.c_float, ctypes.c_float, I32, P, P, P, SZ, P, P]
        L.q8_attn_decode_workspace_size.argtypes = [I32, I32, I32, I32]
        L.q8_attn_decode_workspace_size.restype = SZ
        L.q8_moe.argtypes = [P, I64, P, I64, I32, I32, I32, I32, P, P, P, P, I64, I64, P, I64, P, P, P, SZ, P, P]
        L.q8_moe_workspace_size.argtypes = [I32, I32, I64, I64, I32]
        L.q8_moe_workspace_size.restype = SZ
        L.q8_sample.argtypes = [P, I32, I64, I32, I64, P, P, P, P, P, P, P, P, P, P]
        L.q8_workspace_zero.argtypes = [P, SZ, P]
        F32 = ctypes.c_float
        L.q8_rms_norm.argtypes = [P, I64, I32, P, I64, I32, P, I64, P, F32, F32, I64, I64, P, I64, P, P, P, P]
        L.q8_rope_turns.argtypes = [P, I32, P]
        L.q8_rope.argtypes = [P, I64, I32, P, I64, I32, I32, I32, I32, F32, P, P, I64, P]
        L.q8_rope_append.argtypes = [P, P, I64, I32, P, P, I64, I64, I32, I32, I32, F32, P, P, P, I64, P, I64, P, P]
        L.q8_kv_plan.argtypes = [P, I32, I32, I32, P, P, I32, P, I32, P, P, I64, P, P, P, P, P, P]
        L.q8_attn_chunk.argtypes = [P, P, I64, I32, I64, P, I32, P, P, I32, F32, F32, I32, P, P, P, SZ, P, P]
        L.q8_attn_chunk_workspace_size.argtypes = [I32, I32, I32]
        L.q8_attn_chunk_workspace_size.restype = SZ
        L.q8_status_str.argtypes = [ctypes.c_int]
        L.q8_status_str.restype = ctypes.c_char_p
        L.q8_abi_version.restype = I32
        for name in ("q8_quantize_rows", "q8_quantize_rows_ex", "q8_gemv", "q8_gemm_skinny", "q8_linear_batch",
                     "q8_linear_batch_ex", "q8_linear_batch_chained", "q8_gguf_to_planar",
                     "q8_planar_to_gguf", "q8_gemm", "q8_gemm_ex", "q8_gemm_skinny_noalloc", "q8_linear_chain", "q8_gemm_w8a8",
                     "q8_kv_append", "q8_kv_read", "q8_attn_decode", "q8_moe",
                     "q8_sample", "q8_workspace_zero", "q8_rms_norm", "q8_rope_turns", "q8_rope", "q8_rope_append", "q8_kv_plan",
                     "q8_attn_chunk"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_str(st: int) -> str:
    return lib().q8_status_str(int(st)).decode()


def _check(st: int, what: str):
    if st != Q8_OK:
        raise Q8Error(st, what)


# The current stream's handle, without making a Stream object (3 us of a call's 15 on the
# host); through that object where the build lacks the short way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _get_device is not None:
            return _raw_stream(_get_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(t, name, dtypes, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    return t


def _status(t):
    """The address of a status word, which kernels write to."""
    if t is None:
        return None
    if not (t.is_cuda and t.element_size() == 4 and t.numel() > 0):
        _cuda(t, "dev_status", (t.dtype,))
        raise TypeError("dev_status must hold a 32-bit word")
    return t.data_ptr()


def _work(ws):
    """(address, bytes) of a workspace."""
    if ws is None:
        return None, 0
    if not (ws.is_cuda and ws.is_contiguous()):
        _cuda(ws, "ws", (ws.dtype,))
        if not ws.is_contiguous():
            raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


_B16 = (torch.bfloat16, torch.float16, torch.int16, torch.uint16)


def workspace(nbytes: int, device=None) -> torch.Tensor | None:
    """A zeroed workspace of ``nbytes`` (None if 0).  Zero once, reuse freely."""
    if nbytes == 0:
        return None
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")


def _new(stream, make):
    """make() with its allocations (and zeroing) ordered on the call's stream."""
    if not isinstance(stream, torch.cuda.Stream):
        # handle 0 is the default stream (an ExternalStream of 0 is some other, new one)
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return make()


def _alloc(stream, make):
    """As _new, or on the current stream where none is given."""
    return make() if stream is None else _new(stream, make)


# ---------------------------------------------------------------------------
def q8_quantize_rows(w, q=None, s=None, dev_status=None, stream=None, mode=Q8_QUANT_EXACT):
    """Q8_0-quantize float32 w[rows, K] -> (q int8 [rows, K], s float16 [rows, K/32]);
    ``mode`` picks the code rule (Q8_QUANT_EXACT or Q8_QUANT_FL32)."""
    _cuda(w, "w", (torch.float32,), 2)
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    rows, K = w.shape
    if q is None:
        q = _alloc(stream, lambda: torch.empty((rows, K), dtype=torch.int8, device=w.device))
    if s is None:
        s = _alloc(stream, lambda: torch.empty((rows, max(K // 32, 0)), dtype=torch.float16, device=w.device))
    st = lib().q8_quantize_rows_ex(_p(w), rows, K, _p(q), _p(s), int(mode), _status(dev_status), _stream(stream))
    _check(st, "q8_quantize_rows")
    return q, s


def q8_gguf_to_planar(blocks, rows: int, K: int, q=None, s=None, stream=None):
    """GGUF Q8_0 bytes (uint8, rows * K/32 blocks of 34 bytes) -> (q int8 [rows, K],
    s float16 [rows, K/32])."""
    _cuda(blocks, "blocks", (torch.uint8,))
    if not blocks.is_contiguous() or blocks.numel() != rows * (K // 32) * 34:
        raise ValueError("blocks must be contiguous and hold rows * K/32 blocks of 34 bytes")
    if q is None:
        q = _alloc(stream, lambda: torch.empty((rows, K), dtype=torch.int8, device=blocks.device))
    if s is None:
        s = _alloc(stream, lambda: torch.empty((rows, K // 32), dtype=torch.float16, device=blocks.device))
    st = lib().q8_gguf_to_planar(_p(blocks), rows, K, _p(q), _p(s), _stream(stream))
    _check(st, "q8_gguf_to_planar")
    return q, s


def q8_planar_to_gguf(q, s, blocks=None, stream=None):
    """(q int8 [rows, K], s binary16 [rows, K/32]) -> GGUF Q8_0 bytes (uint8)."""
    _cuda(q, "q", (torch.int8,), 2)
    _cuda(s, "s", _B16, 2)
    rows, K = q.shape
    if blocks is None:
        blocks = _alloc(stream, lambda: torch.empty(rows * (K // 32) * 34, dtype=torch.uint8, device=q.device))
    st = lib().q8_planar_to_gguf(_p(q), _p(s), rows, K, _p(blocks), _stream(stream))
    _check(st, "q8_planar_to_gguf")
    return blocks


def q8_workspace_size(N: int, K: int, M: int) -> int:
    return int(lib().q8_workspace_size(N, K, M))


def _desc(q, s, x, y):
    _cuda(q, "q", (torch.int8,), 2)
    _cuda(s, "s", _B16, 2)
    _cuda(x, "x", _B16)
    _cuda(y, "y", (torch.float32,))
    N, K = q.shape
    x2 = x if x.dim() == 2 else x.view(1, -1)
    y2 = y if y.dim() == 2 else y.view(1, -1)
    if x2.stride(1) != 1 or y2.stride(1) != 1 or not q.is_contiguous() or not s.is_contiguous():
        raise ValueError("q, s must be contiguous; x, y must have unit inner stride")
    return LinearDesc(q.data_ptr(), s.data_ptr(), x2.data_ptr(), y2.data_ptr(), N, K,
                      x2.stride(0) if x2.shape[0] > 1 else K, y2.stride(0) if y2.shape[0] > 1 else max(N, 1)), x2.shape[0]


def q8_gemv(q, s, x, y=None, ws=None, dev_status=None, stream=None):
    """y[N] = dequant(q, s) @ x[K] (fp32)."""
    _cuda(q, "q", (torch.int8,), 2)
    _cuda(s, "s", _B16)
    _cuda(x, "x", _B16)
    N, K = q.shape
    if y is None:
        y = _alloc(stream, lambda: torch.empty(N, dtype=torch.float32, device=q.device))
    else:
        _cuda(y, "y", (torch.float32,))
    need = q8_workspace_size(N, K, 1)
    if ws is None and need:
        ws = _alloc(stream, lambda: workspace(need, q.device))
    st = lib().q8_gemv(_p(q), _p(s), N, K, _p(x), _p(y), *_work(ws), _status(dev_status), _stream(stream))
    _check(st, "q8_gemv")
    return y


def q8_gemm_skinny(q, s, x, y=None, ws=None, dev_status=None, stream=None):
    """y[M, N] = x[M, K] @ dequant(q, s)^T (fp32), 1 <= M <= 32."""
    N, K = q.shape
    M = x.shape[0]
    if y is None:
        y = _alloc(stream, lambda: torch.empty((M, N), dtype=torch.float32, device=q.device))
    d, _ = _desc(q, s, x, y)
    need = q8_workspace_size(N, K, M)
    if ws is None and need:
        ws = _alloc(stream, lambda: workspace(need, q.device))
    st = lib().q8_gemm_skinny(_p(q), _p(s), N, K, _p(x), d.ldx, M, _p(y), d.ldy, *_work(ws), _status(dev_status), _stream(stream))
    _check(st, "q8_gemm_skinny")
    return y


def q8_gemm_skinny_noalloc(q, s, x, y=None, dev_status=None, stream=None):
    """As q8_gemm_skinny, for callers that cannot allocate device memory: the
    split-K scratch is the library's built-in device array (shapes needing more
    than Q8_NOALLOC_SCRATCH_BYTES are rejected).  Calls that may overlap on the
    GPU must not use it concurrently."""
    N, K = q.shape
    M = x.shape[0]
    if y is None:
        y = _alloc(stream, lambda: torch.empty((M, N), dtype=torch.float32, device=q.device))
    d, _ = _desc(q, s, x, y)
    st = lib().q8_gemm_skinny_noalloc(_p(q), _p(s), N, K, _p(x), d.ldx, M, _p(y), d.ldy,
                                      _status(dev_status), _stream(stream))
    _check(st, "q8_gemm_skinny_noalloc")
    return y


def make_descs(mats):
    """[(q, s, x, y), ...] -> (ctypes array of LinearDesc, M)."""
    arr = (LinearDesc * len(mats))()
    M = None
    for i, (q, s, x, y) in enumerate(mats):
        arr[i], m = _desc(q, s, x, y)
        if M is not None and m != M:
            raise ValueError("all matrices of a batch share M")
        M = m
    return arr, (M or 0)


def q8_linear_batch_workspace_size(descs, M: int) -> int:
    return int(lib().q8_linear_batch_workspace_size(descs, len(descs), M))


def q8_linear_batch(mats=None, ws=None, variant=Q8_VARIANT_AUTO, dev_status=None, stream=None,
                    descs=None, M=None, chained=False):
    """Run several skinny matmuls in one launch.  ``mats`` = [(q, s, x, y), ...],
    or pass prepared ``descs`` (from make_descs) and ``M``.  ``chained=True``
    calls q8_linear_batch_chained (no earlier work in the stream may write
    the weights; the variant is then automatic)."""
    if descs is None:
        descs, M = make_descs(mats)
    need = int(lib().q8_linear_batch_workspace_size_ex(descs, len(descs), M, variant))
    if ws is None and need:
        ws = _alloc(stream, lambda: workspace(need))
    if chained:
        if variant != Q8_VARIANT_AUTO:
            raise ValueError("a chained call uses the automatic variant")
        st = lib().q8_linear_batch_chained(descs, len(descs), M, *_work(ws), _status(dev_status), _stream(stream))
    else:
        st = lib().q8_linear_batch_ex(descs, len(descs), M, variant, *_work(ws), _status(dev_status),
                                      _stream(stream))
    _check(st, "q8_linear_batch")


def make_chain(steps):
    """[(q, s, x, y, next), ...] -> (ctypes array of ChainStep, M).  Step 0's
    x is the input; every later x is a buffer the chain writes (bf16 [M][K]);
    y is fp32 [M][N]; `next` is a Q8_CHAIN_* code (Q8_CHAIN_END last)."""
    arr = (ChainStep * len(steps))()
    M = None
    for i, (q, s, x, y, nxt) in enumerate(steps):
        d, m = _desc(q, s, x, y)
        if M is not None and m != M:
            raise ValueError("all steps of a chain share M")
        M = m
        arr[i] = ChainStep(d.q, d.s, d.x, d.y, d.N, d.K, d.ldx, d.ldy, int(nxt), 0)
    return arr, (M or 0)


def q8_linear_chain_workspace_size(steps, M: int) -> int:
    return int(lib().q8_linear_chain_workspace_size(steps, len(steps), M))


def q8_linear_chain(steps, M, ws=None, dev_status=None, stream=None):
    """Run a chain from make_chain(): each step's matmul, then the next
    step's x made from its y on the device (q8_linear_chain)."""
    need = q8_linear_chain_workspace_size(steps, M)
    if ws is None and need:
        ws = _alloc(stream, lambda: workspace(need))
    st = lib().q8_linear_chain(steps, len(steps), M, *_work(ws), _status(dev_status), _stream(stream))
    _check(st, "q8_linear_chain")


def q8_gemm_w8a8(q, s, x, y=None, ws=None, dev_status=None, stream=None):
    """y[M, N] (fp32) = the W8A8 product of x[M, K] (bf16, rows quantized to
    Q8_0) and dequant(q, s)^T, any M (q8_gemm_w8a8)."""
    _cuda(q, "q", (torch.int8,), 2)
    _cuda(s, "s", _B16)
    _cuda(x, "x", _B16, 2)
    N, K = q.shape
    M = x.shape[0]
    if y is None:
        y = _alloc(stream, lambda: torch.empty((M, N), dtype=torch.float32, device=q.device))
    else:
        _cuda(y, "y", (torch.float32,), 2)
    need = int(lib().q8_gemm_w8a8_workspace_size(N, K, M))
    if ws is None and need:
        ws = _alloc(stream, lambda: workspace(need, q.device))
    st = lib().q8_gemm_w8a8(_p(q), _p(s), N, K, _p(x), x.stride(0), M, _p(y), y.stride(0), *_work(ws),
                            _status(dev_status), _stream(stream))
    _check(st, "q8_gemm_w8a8")
    return y


def q8_gemm(q, s, x, y=None, dev_status=None, stream=None, tile=0, splits=0):
    """y[M, N] (bf16) = x[M, K] @ dequant(q, s)^T for M > 32 (tcgen05 path);
    `tile` is one of the Q8_GEMM_TILE_* shapes and `splits` the number of
    CTAs sharing a tile's K range (0: automatic for either)."""
    _cuda(q, "q", (torch.int8,), 2)
    _cuda(s, "s", _B16)
    _cuda(x, "x", _B16, 2)
    N, K = q.shape
    M = x.shape[0]
    if y is None:
        y = _alloc(stream, lambda: torch.empty((M, N), dtype=torch.bfloat16, device=q.device))
    else:
        _cuda(y, "y", _B16, 2)
    st = lib().q8_gemm_ex(_p(q), _p(s), N, K, _p(x), x.stride(0), M, _p(y), y.stride(0), int(tile), int(splits),
                          _status(dev_status), _stream(stream))
    _check(st, "q8_gemm")
    return y


# ---------------------------------------------------------------------------
# the rest of a decode step
#
# These calls take 10 to 20 us of kernel at their smallest, so what the host spends on them
# counts: arguments are looked at in one expression, and one by one (for the message) only
# where that fails.
# ---------------------------------------------------------------------------
_I8, _I32, _I64, _F32, _BF16 = torch.int8, torch.int32, torch.int64, torch.float32, torch.bfloat16


def _counting_workspace(nbytes, zeroed, device):
    """A workspace of which only the words that the kernels count with are zeroed."""
    if nbytes == 0:
        return None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _check(lib().q8_workspace_zero(ws.data_ptr(), zeroed, _stream(None)), "q8_workspace_zero")
    return ws


class KvCache:
    """A paged key-value cache in Q8_0 blocks (q8_kv_cache): codes int8
    [pages, kv_heads, page_size, head_dim], scales 16-bit [..., head_dim / 32].
    Holds the tensors; make it once per cache."""

    def __init__(self, kq, ks, vq, vs):
        for n, t in (("kq", kq), ("vq", vq)):
            _cuda(t, n, (torch.int8,), 4)
        for n, t in (("ks", ks), ("vs", vs)):
            _cuda(t, n, _B16, 4)
        shape = tuple(kq.shape)
        scales = shape[:3] + (shape[3] // 32,)
        if tuple(vq.shape) != shape or tuple(ks.shape) != scales or tuple(vs.shape) != scales:
            raise ValueError("keys and values share the shape [pages, kv_heads, page_size, head_dim], scales [..., head_dim / 32]")
        if not all(t.is_contiguous() for t in (kq, ks, vq, vs)):
            raise ValueError("the cache's tensors must be contiguous")
        if len({t.device for t in (kq, ks, vq, vs)}) != 1:
            raise ValueError("the cache's tensors must be on one device")
        self.kq, self.ks, self.vq, self.vs = kq, ks, vq, vs
        self.pages, self.kv_heads, self.page_size, self.head_dim = shape
        self.device = kq.device
        self.get_device = kq.get_device
        self._c = _CKvCache(kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(), shape[0], shape[2], shape[1], shape[3])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
        """An uninitialised cache of that shape."""
        a = (pages, kv_heads, page_size, head_dim)
        b = (pages, kv_heads, page_size, head_dim // 32)
        return cls(torch.empty(a, dtype=torch.int8, device=device), torch.empty(b, dtype=torch.float16, device=device),
                   torch.empty(a, dtype=torch.int8, device=device), torch.empty(b, dtype=torch.float16, device=device))


_ROW_DTYPES = {torch.float32: Q8_DTYPE_F32, torch.bfloat16: Q8_DTYPE_BF16}


def _kv_rows(cache, t, name, n, dtype):
    """The row stride of [n, kv_heads * head_dim] or [n, kv_heads, head_dim] rows (heads contiguous)."""
    if not t.is_cuda or t.dtype not in _ROW_DTYPES or t.dtype is not dtype:
        raise TypeError(f"{name} must be a float32 or bfloat16 CUDA tensor, keys and values alike")
    sh, sd, h, d = t.shape, t.stride(), cache.kv_heads, cache.head_dim
    if sh == (n, h, d):
        ok = sd[2] == 1 and (sd[1] == d or h == 1)
    else:
        ok = sh == (n, h * d) and sd[1] == 1
    if not ok and n > 0:
        raise ValueError(f"{name} must hold {n} rows of {h} x {d} values, each row contiguous")
    return sd[0] if n > 1 else h * d


def _slots(slots):
    if not (slots.is_cuda and slots.dtype is _I64 and slots.dim() == 1):
        _cuda(slots, "slots", (_I64,), 1)
    n = slots.shape[0]
    if n > 1 and slots.stride(0) != 1:
        raise ValueError("slots must be contiguous")
    return n


def q8_kv_append(cache, k, v, slots, dev_status=None, stream=None):
    """Quantize the rows k, v ([T, kv_heads, head_dim] or [T, kv_heads * head_dim], fp32 or
    bf16) into the cache's slots (int64 [T], each at most once; negative: skipped)."""
    n, t = _slots(slots), k.dtype
    ldk, ldv = _kv_rows(cache, k, "k", n, t), _kv_rows(cache, v, "v", n, t)
    st = lib().q8_kv_append(cache._ref, k.data_ptr(), v.data_ptr(), ldk, ldv, _ROW_DTYPES[t], slots.data_ptr(), n,
                            _status(dev_status), _stream(stream))
    if st:
        _check(st, "q8_kv_append")


def q8_kv_read(cache, slots, k=None, v=None, dtype=torch.float32, dev_status=None, stream=None):
    """The values of the cache's slots: (k, v), each [T, kv_heads, head_dim] in `dtype`
    (or in the given rows' own type); a negative slot gives zeros."""
    n, h, d = _slots(slots), cache.kv_heads, cache.head_dim
    if k is not None or v is not None:
        dtype = (v if k is None else k).dtype
    if dtype not in _ROW_DTYPES:
        raise TypeError("the values are given as float32 or bfloat16")
    row = h * d
    if k is not None:
        ldk = _kv_rows(cache, k, "k", n, dtype)
    else:
        k, ldk = torch.empty((n, h, d), dtype=dtype, device=cache.device) if stream is None else _new(
            stream, lambda: torch.empty((n, h, d), dtype=dtype, device=cache.device)), row
    if v is not None:
        ldv = _kv_rows(cache, v, "v", n, dtype)
    else:
        v, ldv = torch.empty((n, h, d), dtype=dtype, device=cache.device) if stream is None else _new(
            stream, lambda: torch.empty((n, h, d), dtype=dtype, device=cache.device)), row
    st = lib().q8_kv_read(cache._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), ldk, ldv, _ROW_DTYPES[dtype],
                          _status(dev_status), _stream(stream))
    if st:
        _check(st, "q8_kv_read")
    return k, v


def q8_attn_decode_workspace_size(batch: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().q8_attn_decode_workspace_size(batch, q_heads, kv_heads, head_dim))


def q8_attn_decode(q, cache, table, lens, scale=None, softcap=0.0, window=0, out=None, lse=None, ws=None, dev_status=None,
                   stream=None):
    """Attention of one new token per sequence over the cache: q bf16 [B, q_heads, head_dim],
    table int32 [B, pages of a sequence], lens int32 [B] (the new token included).
    Returns (out bf16 [B, q_heads, head_dim], lse fp32 [B, q_heads]).  scale defaults to
    1 / sqrt(head_dim); softcap 0: none; window 0: all tokens."""
    sq = q.stride()
    if not (q.is_cuda and table.is_cuda and lens.is_cuda and q.dtype is _BF16 and table.dtype is _I32 and lens.dtype is _I32
            and len(sq) == 3 and table.dim() == 2 and lens.dim() == 1):
        _cuda(q, "q", (_BF16,), 3)
        _cuda(table, "table", (_I32,), 2)
        _cuda(lens, "lens", (_I32,), 1)
    B, H, D = q.shape
    n, width = table.shape
    if D != cache.head_dim or n != B or lens.shape[0] != B:
        raise ValueError("q is [B, q_heads, head_dim] with the cache's head_dim, table [B, pages], lens [B]")
    if (sq[2] != 1 or (H > 1 and sq[1] != D)) and B > 0:
        raise ValueError("each row of q must be contiguous")
    if not (table.is_contiguous() and lens.is_contiguous()):
        raise ValueError("table and lens must be contiguous")
    if out is None:
        out = torch.empty((B, H, D), dtype=_BF16, device=cache.device) if stream is None else _new(
            stream, lambda: torch.empty((B, H, D), dtype=_BF16, device=cache.device))
    elif _cuda(out, "out", (_BF16,), 3).shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape")
    if lse is None:
        lse = torch.empty((B, H), dtype=_F32, device=cache.device) if stream is None else _new(
            stream, lambda: torch.empty((B, H), dtype=_F32, device=cache.device))
    elif _cuda(lse, "lse", (_F32,), 2).shape != (B, H) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous, [B, q_heads]")
    if ws is None:
        nbytes = q8_attn_decode_workspace_size(B, H, cache.kv_heads, D)
        ws = _alloc(stream, lambda: _counting_workspace(nbytes, Q8_ATTN_ZEROED_BYTES, cache.device))
    st = lib().q8_attn_decode(cache._ref, q.data_ptr(), sq[0] if B > 1 else H * D, H, table.data_ptr(), width, lens.data_ptr(), B,
                              D ** -0.5 if scale is None else scale, softcap, window if window < 2 ** 31 else 2 ** 31 - 1,
                              out.data_ptr(), lse.data_ptr(),
                              *_work(ws), _status(dev_status), _stream(stream))
    if st:
        _check(st, "q8_attn_decode")
    return out, lse


def q8_moe_workspace_size(T: int, E: int, H: int, F: int, top_k: int) -> int:
    return int(lib().q8_moe_workspace_size(T, E, H, F, top_k))


def q8_moe(x, logits, q13, s13, q2, s2, top_k, renorm=True, y=None, ids=None, weights=None, ws=None, dev_status=None,
           stream=None):
    """A mixture-of-experts layer for T <= 32 tokens: x bf16 [T, H], router logits fp32 [T, E],
    experts' gate and up rows (q13 int8 [E, 2 F, H], s13) and down rows (q2 int8 [E, H, F], s2).
    Returns (y fp32 [T, H], ids int32 [T, top_k], weights fp32 [T, top_k])."""
    sx, sl = x.stride(), logits.stride()
    if not (x.is_cuda and logits.is_cuda and q13.is_cuda and s13.is_cuda and q2.is_cuda and s2.is_cuda and x.dtype is _BF16
            and logits.dtype is _F32 and q13.dtype is _I8 and q2.dtype is _I8 and s13.dtype in _B16 and s2.dtype in _B16
            and len(sx) == 2 and len(sl) == 2):
        _cuda(x, "x", (_BF16,), 2)
        _cuda(logits, "logits", (_F32,), 2)
        for name, t, types in (("q13", q13, (_I8,)), ("q2", q2, (_I8,)), ("s13", s13, _B16), ("s2", s2, _B16)):
            _cuda(t, name, types, 3)
    T, H = x.shape
    n, E = logits.shape
    F = q2.shape[-1]
    if n != T or q13.shape != (E, 2 * F, H) or q2.shape != (E, H, F):
        raise ValueError("x is [T, H], logits [T, E], q13 [E, 2 F, H] and q2 [E, H, F]")
    if s13.shape != (E, 2 * F, H // 32) or s2.shape != (E, H, F // 32):
        raise ValueError("s13 and s2 hold a scale per 32 codes")
    if not (q13.is_contiguous() and s13.is_contiguous() and q2.is_contiguous() and s2.is_contiguous()):
        raise ValueError("the experts' tensors must be contiguous")
    if T > 0 and (sx[1] != 1 or sl[1] != 1):
        raise ValueError("x and logits must have unit inner stride")
    dev = x.device
    if y is None:
        y, ldy = torch.empty((T, H), dtype=_F32, device=dev) if stream is None else _new(
            stream, lambda: torch.empty((T, H), dtype=_F32, device=dev)), H
    else:
        if _cuda(y, "y", (_F32,), 2).shape != (T, H) or y.stride(1) != 1:
            raise ValueError("y must be [T, H] with unit inner stride")
        ldy = H if T <= 1 else y.stride(0)
    if ids is None:
        ids = torch.empty((T, top_k), dtype=_I32, device=dev) if stream is None else _new(
            stream, lambda: torch.empty((T, top_k), dtype=_I32, device=dev))
    elif _cuda(ids, "ids", (_I32,), 2).shape != (T, top_k) or not ids.is_contiguous():
        raise ValueError("ids must be contiguous, [T, top_k]")
    if weights is None:
        weights = torch.empty((T, top_k), dtype=_F32, device=dev) if stream is None else _new(
            stream, lambda: torch.empty((T, top_k), dtype=_F32, device=dev))
    elif _cuda(weights, "weights", (_F32,), 2).shape != (T, top_k) or not weights.is_contiguous():
        raise ValueError("weights must be contiguous, [T, top_k]")
    if ws is None:
        nbytes = q8_moe_workspace_size(T, E, H, F, top_k)
        ws = _alloc(stream, lambda: _counting_workspace(nbytes, Q8_MOE_ZEROED_BYTES, dev))
    one = T <= 1
    st = lib().q8_moe(x.data_ptr(), H if one else sx[0], logits.data_ptr(), E if one else sl[0], T, E, top_k, 1 if renorm else 0,
                      q13.data_ptr(), s13.data_ptr(), q2.data_ptr(), s2.data_ptr(), H, F, y.data_ptr(), ldy, ids.data_ptr(),
                      weights.data_ptr(), *_work(ws), _status(dev_status), _stream(stream))
    if st:
        _check(st, "q8_moe")
    return y, ids, weights


def _per_row(t, name, n, dtype):
    if t is None:
        return None
    if not (t.is_cuda and t.dtype is dtype):
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must hold one value per row, contiguous")
    return t.data_ptr()


def q8_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, token=None, logprob=None, kept=None,
              dev_status=None, stream=None):
    """Draw one word per row of logits [rows, V] (fp32 or bf16) from uniform numbers u fp32
    [rows] in [0, 1).  temperature, top_p, min_p fp32 [rows] and top_k int32 [rows] may be
    None.  Returns (token int32, logprob fp32, kept int32), each [rows]."""
    if not logits.is_cuda or logits.dtype not in _ROW_DTYPES:
        raise TypeError("logits must be a float32 or bfloat16 CUDA tensor")
    sl = logits.stride()
    if len(sl) != 2 or (logits.shape[1] > 1 and sl[1] != 1):
        raise ValueError("logits must be [rows, V] with unit inner stride")
    n, V = logits.shape
    dev = logits.device
    if token is None:
        token = torch.empty(n, dtype=_I32, device=dev) if stream is None else _new(
            stream, lambda: torch.empty(n, dtype=_I32, device=dev))
    if logprob is None:
        logprob = torch.empty(n, dtype=_F32, device=dev) if stream is None else _new(
            stream, lambda: torch.empty(n, dtype=_F32, device=dev))
    if kept is None:
        kept = torch.empty(n, dtype=_I32, device=dev) if stream is None else _new(
            stream, lambda: torch.empty(n, dtype=_I32, device=dev))
    st = lib().q8_sample(logits.data_ptr(), _ROW_DTYPES[logits.dtype], sl[0] if n > 1 else V, n, V,
                         _per_row(temperature, "temperature", n, _F32), _per_row(top_k, "top_k", n, _I32),
                         _per_row(top_p, "top_p", n, _F32), _per_row(min_p, "min_p", n, _F32), _per_row(u, "u", n, _F32),
                         _per_row(token, "token", n, _I32), _per_row(logprob, "logprob", n, _F32), _per_row(kept, "kept", n, _I32),
                         _status(dev_status), _stream(stream))
    if st:
        _check(st, "q8_sample")
    return token, logprob, kept


# ---------------------------------------------------------------------------
# a prompt step
# ---------------------------------------------------------------------------
def _here(first, *others):
    """All of a call's tensors (the status word among them) are on one device, the current one."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("the tensors of a call must be on one device")
    if dev >= 0 and _get_device is not None and dev != _get_device():
        raise ValueError("the tensors of a call must be on the current device")


def _rows(t, name, n, width):
    """The stride of n rows of `width` values (one or more inner dimensions, contiguous)."""
    sh = t.shape
    if t.is_contiguous() and len(sh) >= 2 and sh[0] == n and t.numel() == n * width and n > 0:
        return width
    sd = t.stride()
    want = 1
    ok = len(sh) >= 2 and sh[0] == n
    for i in range(len(sh) - 1, 0, -1):
        ok = ok and (sd[i] == want or sh[i] == 1)
        want *= sh[i]
    if not ok or want != width:
        raise ValueError(f"{name} must hold {n} rows of {width} values, each row contiguous")
    return sd[0] if n > 1 else width


def _out(stream, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device) if stream is None else _new(
        stream, lambda: torch.empty(shape, dtype=dtype, device=device))


def q8_rms_norm(x, weight=None, offset=0.0, eps=1e-6, residual=None, residual_out=None, y=None, q=None, s=None, bf16=True,
                quantized=False, dev_status=None, stream=None):
    """h = x + residual and its root-mean-square norm times (weight + offset): x [T, W] fp32 or
    bf16, residual [T, W] fp32 or bf16 (updated in place, or to `residual_out`), weight fp32 [W].
    Returns (y bf16 [T, W], q int8 [T, W], s float16 [T, W / 32]): y unless bf16=False, the
    Q8_0 rows if `quantized` (or q and s are given), None in the place of what is not asked for."""
    xt, xd = x.dtype, x.shape
    if not (x.is_cuda and xt in _ROW_DTYPES and len(xd) == 2):
        _cuda(x, "x", tuple(_ROW_DTYPES), 2)
    T, W = xd
    ldx = _rows(x, "x", T, W)
    kind, ldr, ldo, ldy = xt, W, W, W
    if residual is not None:
        kind = residual.dtype
        if residual_out is None:
            residual_out = residual
        if not (residual.is_cuda and residual_out.is_cuda and kind in _ROW_DTYPES and residual_out.dtype is kind):
            _cuda(residual, "residual", tuple(_ROW_DTYPES), 2)
            _cuda(residual_out, "residual_out", (kind,), 2)
        ldr, ldo = _rows(residual, "residual", T, W), _rows(residual_out, "residual_out", T, W)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if weight is not None and not (weight.is_cuda and weight.dtype is _F32 and weight.shape == (W,) and weight.is_contiguous()):
        _cuda(weight, "weight", (_F32,), 1)
        raise ValueError("weight must hold W values, contiguous")
    if y is not None:
        ldy = _rows(_cuda(y, "y", (_BF16,), 2), "y", T, W)
    elif bf16:
        y = _out(stream, xd, _BF16, x.device)
    if quantized or q is not None or s is not None:
        if q is None:
            q = _out(stream, xd, _I8, x.device)
        if s is None:
            s = _out(stream, (T, W // 32), torch.float16, x.device)
        if _cuda(q, "q", (_I8,), 2).shape != xd or not q.is_contiguous():
            raise ValueError("q must be contiguous, [T, W]")
        if _cuda(s, "s", _B16, 2).shape != (T, W // 32) or not s.is_contiguous():
            raise ValueError("s must be contiguous, [T, W / 32]")
    status = _status(dev_status)
    _here(x, weight, residual, residual_out, y, q, s, dev_status)
    st = lib().q8_rms_norm(x.data_ptr(), ldx, _ROW_DTYPES[xt], _a(residual), ldr, _ROW_DTYPES[kind], _a(residual_out), ldo,
                           _a(weight), offset, eps, T, W, _a(y), ldy, _a(q), _a(s), status, _stream(stream))
    if st:
        _check(st, "q8_rms_norm")
    return y, q, s


def _a(t):
    return None if t is None else t.data_ptr()


def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, trained=4096, fast=32.0, slow=1.0):
    """(radians a token for each of rot / 2 pairs, the factor on cosines and sines), in 64 bits.
    base ** (-2 i / rot) for pair i, and for contexts `factor` times the `trained` length:
      "linear": all frequencies divided by `factor`;
      "ntk":    the base raised so that the slowest pair is;
      "yarn":   pairs that turn less than `slow` times in `trained` tokens divided, those that turn
                more than `fast` times kept, a ramp between, and 1 + 0.1 log(factor) on the result."""
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError("scaling is None, 'linear', 'ntk' or 'yarn'")
    if rot < 4 or rot % 2 or not factor >= 1.0:
        raise ValueError("rot is even, 4 at least, and factor 1 at least")
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling != "yarn":
        return f, 1.0

    def pair(turns):  # the (fractional) pair that turns so many times in the trained length
        return rot * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
    return [x / factor * r + x * (1.0 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


def rope_turns(inv_freq, device=None):
    """The table of q8_rope from frequencies in radians a token (a list, or a tensor of any
    device): int64 [pairs] on `device` (the tensor's, else the current one).  Made once."""
    if isinstance(inv_freq, torch.Tensor):
        device = device or (inv_freq.device if inv_freq.is_cuda else None)
        inv_freq = inv_freq.detach().to("cpu", torch.float64)
    f = torch.as_tensor(inv_freq, dtype=torch.float64).contiguous()
    if f.dim() != 1:
        raise ValueError("inv_freq has one value per pair")
    turns = torch.empty(f.shape, dtype=_I64)
    _check(lib().q8_rope_turns(f.data_ptr(), f.shape[0], turns.data_ptr()), "q8_rope_turns")
    return turns.to(device or "cuda")


def _rope_args(turns, positions, n, d):
    if not (turns.is_cuda and positions.is_cuda and turns.dtype is _I64 and positions.dtype is _I32):
        _cuda(turns, "turns", (_I64,))
        _cuda(positions, "positions", (_I32,))
    if turns.dim() != 1 or not turns.is_contiguous() or 2 * turns.shape[0] > d:
        raise ValueError("turns holds a contiguous value per pair, of head_dim / 2 pairs at most")
    if positions.shape != (n,) or not positions.is_contiguous():
        raise ValueError("positions must hold one value per token, contiguous")
    return 2 * turns.shape[0]


def q8_rope(x, positions, turns, interleaved=False, factor=1.0, y=None, stream=None):
    """Rotary positions of x [T, heads, head_dim] (fp32 or bf16) at positions int32 [T], with the
    table of rope_turns: the first 2 * len(turns) dimensions of each head turn.  Returns y
    bf16 [T, heads, head_dim] (y may be x itself)."""
    if not (x.is_cuda and x.dtype in _ROW_DTYPES and x.dim() == 3):
        _cuda(x, "x", tuple(_ROW_DTYPES), 3)
    n, h, d = x.shape
    rot = _rope_args(turns, positions, n, d)
    ldx = _rows(x, "x", n, h * d)
    if y is None:
        y = _out(stream, (n, h, d), _BF16, x.device)
    elif _cuda(y, "y", (_BF16,), 3).shape != x.shape:
        raise ValueError("y has x's shape")
    _here(x, positions, turns, y)
    st = lib().q8_rope(x.data_ptr(), ldx, _ROW_DTYPES[x.dtype], y.data_ptr(), _rows(y, "y", n, h * d), h, d, rot,
                       1 if interleaved else 0, factor, turns.data_ptr(), positions.data_ptr(), n, _stream(stream))
    if st:
        _check(st, "q8_rope")
    return y


def q8_rope_append(q, k, v, cache, positions, slots, turns, interleaved=False, factor=1.0, y=None, dev_status=None, stream=None):
    """q8_rope of the query heads q [T, q_heads, head_dim], and of the key heads k on their way
    into the cache's slots with the values v ([T, kv_heads, head_dim] or [T, kv_heads * head_dim]),
    all fp32 or all bf16.  Returns the turned queries, bf16 [T, q_heads, head_dim]."""
    n, t = _slots(slots), k.dtype
    ldk, ldv = _kv_rows(cache, k, "k", n, t), _kv_rows(cache, v, "v", n, t)
    _cuda(q, "q", (t,), 3)
    h, d = q.shape[1], cache.head_dim
    if q.shape[0] != n or q.shape[2] != d:
        raise ValueError("q is [T, q_heads, head_dim] with a slot per token and the cache's head_dim")
    rot = _rope_args(turns, positions, n, d)
    ldq = _rows(q, "q", n, h * d)
    if y is None:
        y = _out(stream, (n, h, d), _BF16, q.device)
    elif _cuda(y, "y", (_BF16,), 3).shape != q.shape:
        raise ValueError("y has q's shape")
    status = _status(dev_status)
    _here(q, k, v, cache, positions, slots, turns, y, dev_status)
    st = lib().q8_rope_append(cache._ref, q.data_ptr(), ldq, h, k.data_ptr(), v.data_ptr(), ldk, ldv, _ROW_DTYPES[t], rot,
                              1 if interleaved else 0, factor, turns.data_ptr(), positions.data_ptr(), slots.data_ptr(), n,
                              y.data_ptr(), _rows(y, "y", n, h * d), status, _stream(stream))
    if st:
        _check(st, "q8_rope_append")
    return y


def _ints(t, name, shape, dtype=_I32):
    if not (t.is_cuda and t.dtype is dtype):
        _cuda(t, name, (dtype,))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {tuple(shape)}")
    return t.data_ptr()


def q8_kv_plan(table, lens, new_tokens, page_size, pages, T, free_pages=None, free_count=None, free_left=None, starts=None,
               slots=None, positions=None, lens_out=None, dev_status=None, stream=None):
    """Where each new token goes: table int32 [B, width] (updated), lens int32 [B] tokens in the
    cache, new_tokens int32 [B], T rows.  Pages are taken from the end of the first free_count
    (int32 [1]) of free_pages (int32); without free_pages the table is complete.  Returns (starts int32
    [B + 1], slots int64 [T], positions int32 [T], lens_out int32 [B], free_left int32 [1] or None)."""
    _cuda(table, "table", (_I32,), 2)
    B, width = table.shape
    if not table.is_contiguous():
        raise ValueError("table must be contiguous")
    dev = table.device
    if free_pages is None and (free_count is not None or free_left is not None):
        raise ValueError("free_count and free_left belong to free_pages")
    if free_pages is not None and free_count is None:
        raise ValueError("free_pages needs free_count")
    starts = _out(stream, (B + 1,), _I32, dev) if starts is None else starts
    slots = _out(stream, (T,), _I64, dev) if slots is None else slots
    positions = _out(stream, (T,), _I32, dev) if positions is None else positions
    lens_out = _out(stream, (B,), _I32, dev) if lens_out is None else lens_out
    if free_pages is not None and free_left is None:
        free_left = _out(stream, (1,), _I32, dev)
    args = [_ints(lens, "lens", (B,)), _ints(new_tokens, "new_tokens", (B,)), B]
    if free_pages is None:
        args += [None, 0, None, None]
    else:
        n = _cuda(free_pages, "free_pages", (_I32,), 1).shape[0]
        # an empty list is a list all the same (its address, and an empty table's, are NULL; nothing is read there)
        at = _ints(free_pages, "free_pages", (n,)) or starts.data_ptr()
        args += [at, n, _ints(free_count, "free_count", (1,)), _ints(free_left, "free_left", (1,))]
    status = _status(dev_status)
    _here(table, lens, new_tokens, free_pages, free_count, free_left, starts, slots, positions, lens_out, dev_status)
    st = lib().q8_kv_plan(table.data_ptr(), width, pages, page_size, *args, T, _ints(starts, "starts", (B + 1,)),
                          _ints(slots, "slots", (T,), _I64), _ints(positions, "positions", (T,)), _ints(lens_out, "lens_out", (B,)),
                          status, _stream(stream))
    if st:
        _check(st, "q8_kv_plan")
    return starts, slots, positions, lens_out, free_left


def q8_attn_chunk_workspace_size(q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().q8_attn_chunk_workspace_size(q_heads, kv_heads, head_dim))


def q8_attn_chunk(q, cache, table, lens, starts, scale=None, softcap=0.0, window=0, out=None, lse=None, return_lse=False, ws=None,
                  dev_status=None, stream=None):
    """Causal attention of each sequence's newest tokens over the cache: q bf16 [T, q_heads,
    head_dim], the rows starts[b] .. starts[b + 1] - 1 (int32 [B + 1]) being the last of the lens[b]
    (int32 [B]) tokens of sequence b, table int32 [B, pages of a sequence].  Returns (out
    bf16 [T, q_heads, head_dim], lse fp32 [T, q_heads] if asked for or given, else None).  Rows of no
    sequence are left as they are.  scale defaults to 1 / sqrt(head_dim); softcap 0: none; window 0: all."""
    if not (q.is_cuda and table.is_cuda and q.dtype is _BF16 and table.dtype is _I32 and q.dim() == 3 and table.dim() == 2):
        _cuda(q, "q", (_BF16,), 3)
        _cuda(table, "table", (_I32,), 2)
    T, H, D = q.shape
    B, width = table.shape
    if D != cache.head_dim:
        raise ValueError("q has the cache's head_dim")
    if not table.is_contiguous():
        raise ValueError("table must be contiguous")
    ldq = _rows(q, "q", T, H * D)
    n_at, s_at = _ints(lens, "lens", (B,)), _ints(starts, "starts", (B + 1,))
    if out is None:
        out = _out(stream, (T, H, D), _BF16, cache.device)
    elif _cuda(out, "out", (_BF16,), 3).shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape")
    if lse is None:
        if return_lse:
            lse = _out(stream, (T, H), _F32, cache.device)
    elif _cuda(lse, "lse", (_F32,), 2).shape != (T, H) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous, [T, q_heads]")
    status = _status(dev_status)
    _here(q, cache, table, lens, starts, out, lse, ws, dev_status)
    if ws is None:
        nbytes = q8_attn_chunk_workspace_size(H, cache.kv_heads, D)
        ws = _alloc(stream, lambda: _counting_workspace(nbytes, Q8_CHUNK_ZEROED_BYTES, cache.device))
    st = lib().q8_attn_chunk(cache._ref, q.data_ptr(), ldq, H, T, table.data_ptr(), width, n_at, s_at, B,
                             D ** -0.5 if scale is None else scale, softcap, window if window < 2 ** 31 else 2 ** 31 - 1,
                             out.data_ptr(), _a(lse), *_work(ws), status, _stream(stream))
    if st:
        _check(st, "q8_attn_chunk")
    return out, lse
