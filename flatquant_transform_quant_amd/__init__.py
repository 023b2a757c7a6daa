"""Python binding of libfq (include/fq.h): argument marshalling only.

Every step of the operator runs in the HIP kernels of ``libfq.so``; this module only
turns torch tensors into ``fq_tensor`` descriptors, calls the two C entry points and
allocates the workspace through torch.  If the shared library has not been built the
import fails loudly -- there is no fallback path.

Output storage in torch:
  * ``int32`` mode: out is ``torch.int32`` [K, M, N/8] (8 int4 codes per word, low nibble
    first), quantScale ``torch.float32`` [K];
  * ``int4``  mode: out is ``torch.uint8`` [K, M, N/2] holding the logical INT4 [K, M, N]
    (2 codes per byte, low nibble first), quantScale ``torch.float32`` [K];
  * ``fp4``   mode: out is ``torch.uint8`` (or ``torch.float4_e2m1fn_x2``) [K, M*N/2]
    holding the logical FLOAT4_E2M1 [K, M*N], quantScale ``torch.uint8`` (or
    ``torch.float8_e8m0fnu``) [K, ceilDiv(M*N, 64), 2];
  * ``int8`` / ``e4m3`` / ``e5m2`` modes (per-token 8-bit codes): out is ``torch.int8`` /
    ``torch.float8_e4m3fn`` / ``torch.float8_e5m2`` (or ``torch.uint8``) [K, M, N],
    quantScale ``torch.float32`` [K].

A paged key-value cache in the same formats is a :class:`KVCache` (``empty_kv_cache`` allocates
one); ``kv_write``, ``kv_read``, ``attn_decode`` (one new token per sequence), ``attn_prefill`` (packed prompts) and
``attn_chunk`` (any number of new tokens per sequence, with a window) are the calls on it.  ``qk_rope`` normalizes and
rotates queries and keys, ``kv_append`` does that and writes keys and values to the cache.  ``int4_gemm``, ``mx_gemm`` and
``int8_gemm`` multiply codes.

Streams: a call runs on the current stream, or on ``stream``.  Results and workspaces that a call allocates
come from that stream's memory; another stream reads a result after waiting for it.  Tensors that the caller
passes in are the caller's to keep in order (and, if freed early, to ``record_stream``).
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfq.so")

FQ_SUCCESS = 0
FQ_ERR_PARAM_NULLPTR = 161001
FQ_ERR_PARAM_INVALID = 161002
FQ_ERR_RUNTIME = 161003

DT_FLOAT16, DT_BFLOAT16, DT_FLOAT32, DT_INT32, DT_INT4, DT_FLOAT4_E2M1, DT_FLOAT8_E8M0 = range(1, 8)
DT_INT8, DT_FLOAT8_E4M3FN, DT_FLOAT8_E5M2 = range(8, 11)
BYTE_MODES = {"int8": DT_INT8, "e4m3": DT_FLOAT8_E4M3FN, "e5m2": DT_FLOAT8_E5M2}
PER_TOKEN_MODES = ("int32", "int4") + tuple(BYTE_MODES)
KERNEL_AUTO, KERNEL_GENERIC, KERNEL_MFMA_SMALL, KERNEL_MFMA_WIDE, KERNEL_MFMA_WIDE_T, KERNEL_MFMA_WIDE_L = 0, 1, 2, 3, 4, 5


class FqTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("strides", ctypes.c_int64 * 4)]


class FqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = lib.fq_last_error().decode() if status == FQ_ERR_RUNTIME else ""
        self.detail = detail
        super().__init__(f"{what}: {status_string(status)} ({status})" + (f": {detail}" if detail else ""))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libfq is not built ({LIB_PATH} missing): run __graft_entry__.build()")
    # torch ships its own HIP runtime under the same soname as the system one.  Loading
    # torch first makes libfq bind to that copy, so the process holds one HIP runtime and
    # the device pointers and streams torch hands over are valid handles in libfq too.
    # (Loaded the other way round, two runtimes coexist, each with its own device state.)
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(FqTensor)
    vp = ctypes.c_void_p
    L.fq_get_workspace_size.argtypes = [P, P, P, ctypes.c_double, ctypes.c_double, P, P,
                                        ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(vp)]
    L.fq_get_workspace_size.restype = ctypes.c_int32
    L.fq_run.argtypes = [vp, ctypes.c_uint64, vp, vp]
    L.fq_run.restype = ctypes.c_int32
    L.fq_run_no_alloc.argtypes = [vp, vp]
    L.fq_run_no_alloc.restype = ctypes.c_int32
    L.fq_executor_destroy.argtypes = [vp]
    L.fq_executor_destroy.restype = None
    L.fq_executor_set_repeatable.argtypes = [vp, ctypes.c_int32]
    L.fq_executor_set_repeatable.restype = ctypes.c_int32
    L.fq_executor_set_kernel.argtypes = [vp, ctypes.c_int32]
    L.fq_executor_set_kernel.restype = ctypes.c_int32
    L.fq_executor_kernel.argtypes = [vp]
    L.fq_executor_kernel.restype = ctypes.c_int32
    L.fq_status_string.argtypes = [ctypes.c_int32]
    L.fq_status_string.restype = ctypes.c_char_p
    L.fq_last_error.argtypes = []
    L.fq_last_error.restype = ctypes.c_char_p
    L.fq_v1_get_workspace_size.argtypes = [P, P, P, ctypes.c_double, P, P,
                                           ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(vp)]
    L.fq_v1_get_workspace_size.restype = ctypes.c_int32
    L.fq_mx_gemm.argtypes = [P, P, P, P, P, vp]
    L.fq_mx_gemm.restype = ctypes.c_int32
    L.fq_int4_gemm.argtypes = [P, P, P, P, P, vp]
    L.fq_int4_gemm.restype = ctypes.c_int32
    L.fq_dequant.argtypes = [P, P, P, vp]
    L.fq_dequant.restype = ctypes.c_int32
    # (descriptors of the calls below are passed by address, see _Desc)
    dbl, u64 = ctypes.c_double, ctypes.c_uint64
    L.fq_kv_write.argtypes = [vp, vp, vp, dbl, dbl, vp, vp, vp, vp, vp]
    L.fq_kv_read.argtypes = [vp] * 9
    L.fq_attn_decode_get_workspace_size.argtypes = [vp, vp, vp, ctypes.POINTER(u64)]
    L.fq_attn_decode.argtypes = [vp] * 7 + [dbl, vp, vp, vp, u64, vp]
    L.fq_attn_prefill_get_workspace_size.argtypes = [vp, vp, vp, ctypes.c_int32, ctypes.POINTER(u64)]
    L.fq_attn_prefill.argtypes = [vp] * 5 + [ctypes.c_int32, dbl, vp, vp, vp, u64, vp]
    L.fq_qk_rope.argtypes = [vp] * 4 + [dbl, vp, vp, vp, ctypes.c_int32, vp, vp, vp]
    L.fq_kv_append.argtypes = [vp] * 6 + [dbl, vp, vp, vp, ctypes.c_int32, dbl, dbl] + [vp] * 6
    L.fq_int8_gemm.argtypes = [vp] * 6
    L.fq_attn_chunk_get_workspace_size.argtypes = [vp] * 4 + [ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(u64)]
    L.fq_attn_chunk.argtypes = [vp] * 8 + [ctypes.c_int32, ctypes.c_int32, dbl, vp, vp, vp, u64, vp]
    for f in (L.fq_int8_gemm, L.fq_attn_chunk_get_workspace_size, L.fq_attn_chunk, L.fq_qk_rope, L.fq_kv_append, L.fq_kv_write, L.fq_kv_read, L.fq_attn_decode_get_workspace_size, L.fq_attn_decode,
              L.fq_attn_prefill_get_workspace_size, L.fq_attn_prefill):
        f.restype = ctypes.c_int32
    return L


lib = _load()
EXPORTS = ("fq_get_workspace_size", "fq_run", "fq_executor_destroy", "fq_executor_set_repeatable",
           "fq_executor_set_kernel", "fq_executor_kernel", "fq_status_string", "fq_last_error", "fq_dequant",
           "fq_v1_get_workspace_size", "fq_mx_gemm", "fq_int4_gemm", "fq_run_no_alloc", "fq_kv_write", "fq_kv_read",
           "fq_attn_decode_get_workspace_size", "fq_attn_decode", "fq_attn_prefill_get_workspace_size",
           "fq_attn_prefill", "fq_qk_rope", "fq_kv_append", "fq_attn_chunk_get_workspace_size", "fq_attn_chunk",
           "fq_int8_gemm")
NO_ALLOC_SCRATCH_BYTES = 64 << 20  # FQ_NO_ALLOC_SCRATCH_BYTES of include/fq.h


def status_string(status: int) -> str:
    return lib.fq_status_string(status).decode()


# ---- raw C entry points, same names as the C ABI ------------------------------------

def make_tensor(data_ptr: int, dtype: int, shape, strides=None) -> FqTensor:
    shape = list(shape)
    if strides is None:
        strides, acc = [], 1
        for d in reversed(shape):
            strides.insert(0, acc)
            acc *= d
    t = FqTensor()
    t.data = data_ptr or None
    t.dtype = dtype
    t.ndim = len(shape)
    for i, (s, st) in enumerate(zip(shape, strides)):
        t.shape[i] = int(s)
        t.strides[i] = int(st)
    return t


def fq_get_workspace_size(x: FqTensor, p1: FqTensor, p2: FqTensor, clip_ratio: float,
                          dst_type_max: float, out: FqTensor, quant_scale: FqTensor):
    """Returns (status, workspace_size, executor_handle)."""
    ws = ctypes.c_uint64(0)
    ex = ctypes.c_void_p(None)
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    st = lib.fq_get_workspace_size(ref(x), ref(p1), ref(p2), float(clip_ratio), float(dst_type_max),
                                   ref(out), ref(quant_scale), ctypes.byref(ws), ctypes.byref(ex))
    return st, ws.value, ex.value


def fq_v1_get_workspace_size(x: FqTensor, p1: FqTensor, p2: FqTensor, clip_ratio: float,
                             out: FqTensor, quant_scale: FqTensor):
    """The V1 form (no dstTypeMax). Returns (status, workspace_size, executor_handle)."""
    ws = ctypes.c_uint64(0)
    ex = ctypes.c_void_p(None)
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    st = lib.fq_v1_get_workspace_size(ref(x), ref(p1), ref(p2), float(clip_ratio), ref(out), ref(quant_scale),
                                      ctypes.byref(ws), ctypes.byref(ex))
    return st, ws.value, ex.value


def fq_run(workspace_ptr: int, workspace_size: int, executor: int, stream_ptr: int) -> int:
    return lib.fq_run(workspace_ptr or None, workspace_size, executor, stream_ptr or None)


def fq_run_no_alloc(executor: int, stream_ptr: int) -> int:
    return lib.fq_run_no_alloc(executor, stream_ptr or None)


def fq_executor_destroy(executor: int) -> None:
    lib.fq_executor_destroy(executor)


def fq_executor_set_repeatable(executor: int, repeat: bool) -> int:
    return lib.fq_executor_set_repeatable(executor, 1 if repeat else 0)


def fq_executor_set_kernel(executor: int, variant: int) -> int:
    return lib.fq_executor_set_kernel(executor, variant)


def fq_executor_kernel(executor: int) -> int:
    return lib.fq_executor_kernel(executor)


def fq_status_string(status: int) -> str:
    return status_string(status)


def fq_last_error() -> str:
    return lib.fq_last_error().decode()


def fq_int4_gemm(a: FqTensor, a_scale: FqTensor, w: FqTensor, w_scale: FqTensor, c: FqTensor, stream_ptr: int) -> int:
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    return lib.fq_int4_gemm(ref(a), ref(a_scale), ref(w), ref(w_scale), ref(c), stream_ptr or None)


def fq_mx_gemm(a: FqTensor, a_scale: FqTensor, w: FqTensor, w_scale: FqTensor, c: FqTensor, stream_ptr: int) -> int:
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    return lib.fq_mx_gemm(ref(a), ref(a_scale), ref(w), ref(w_scale), ref(c), stream_ptr or None)


def fq_dequant(codes: FqTensor, scale: FqTensor, out: FqTensor, stream_ptr: int) -> int:
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    return lib.fq_dequant(ref(codes), ref(scale), ref(out), stream_ptr or None)


# ---- torch marshalling ---------------------------------------------------------------

def _torch():
    import torch
    return torch


def describe_input(t) -> FqTensor:
    torch = _torch()
    dt = {torch.float16: DT_FLOAT16, torch.bfloat16: DT_BFLOAT16}.get(t.dtype)
    if dt is None:
        dt = -1  # rejected by validation
    return make_tensor(t.data_ptr(), dt, t.shape, t.stride())


def describe_out(out, mode: str, K: int, M: int, N: int) -> FqTensor:
    """Logical descriptor of the code tensor stored in `out` (see the module docstring)."""
    if mode == "int32":
        return make_tensor(out.data_ptr(), DT_INT32, out.shape, out.stride())
    st = list(out.stride())
    if mode == "int4":
        # uint8 [K, M, N/2] storage -> INT4 [K, M, N]: strides in nibbles
        return make_tensor(out.data_ptr(), DT_INT4, (K, M, N), (2 * st[0], 2 * st[1], 1 if st[2] == 1 else 2 * st[2]))
    if mode == "fp4":
        return make_tensor(out.data_ptr(), DT_FLOAT4_E2M1, (K, M * N), (2 * st[0], 1 if st[1] == 1 else 2 * st[1]))
    if mode in BYTE_MODES:
        return make_tensor(out.data_ptr(), BYTE_MODES[mode], out.shape, out.stride())
    raise ValueError(f"unknown mode {mode!r}")


def describe_scale(scale, mode: str) -> FqTensor:
    dt = DT_FLOAT32 if mode in PER_TOKEN_MODES else DT_FLOAT8_E8M0
    return make_tensor(scale.data_ptr(), dt, scale.shape, scale.stride())


def empty_outputs(K: int, M: int, N: int, mode: str, device="cuda"):
    """Allocate (out, quant_scale) for a mode, in the storage described above."""
    torch = _torch()
    if mode == "int32":
        return (torch.empty((K, M, N // 8), dtype=torch.int32, device=device),
                torch.empty((K,), dtype=torch.float32, device=device))
    if mode == "int4":
        return (torch.empty((K, M, N // 2), dtype=torch.uint8, device=device),
                torch.empty((K,), dtype=torch.float32, device=device))
    if mode == "fp4":
        return (torch.empty((K, M * N // 2), dtype=torch.uint8, device=device),
                torch.empty((K, -(-(M * N) // 64), 2), dtype=torch.uint8, device=device))
    if mode in BYTE_MODES:
        dt = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[mode]
        return (torch.empty((K, M, N), dtype=dt, device=device),
                torch.empty((K,), dtype=torch.float32, device=device))
    raise ValueError(f"unknown mode {mode!r}")


class Executor:
    """A planned call (first stage).  Repeatable: run() may be called many times.  Its workspace comes from
    the memory of the stream that is current when it is planned: a first run on another stream has to
    come after that stream's work, by the caller's own event or wait (quantize() plans on the stream it runs on)."""

    def __init__(self, x, p1, p2, out, quant_scale, mode: str, clip_ratio: float = 1.0,
                 dst_type_max: float = 0.0, kernel: int = KERNEL_AUTO, repeatable: bool = True):
        torch = _torch()
        K, M, N = x.shape
        if p2 is None:
            p2 = torch.empty((0, 0), dtype=x.dtype, device=x.device)
        self._keep = (x, p1, p2, out, quant_scale)
        st, ws, ex = fq_get_workspace_size(describe_input(x), describe_input(p1), describe_input(p2),
                                           clip_ratio, dst_type_max, describe_out(out, mode, K, M, N),
                                           describe_scale(quant_scale, mode))
        if st != FQ_SUCCESS:
            raise FqError(st, "fq_get_workspace_size")
        self.handle = ex
        self.workspace_size = ws
        self.workspace = torch.empty((max(ws, 1),), dtype=torch.uint8, device=x.device) if ws else None
        # streams (handles) the caching allocator knows the workspace is used on: the
        # allocating one, then every other stream a run was enqueued on
        self._ws_streams = set()
        if self.workspace is not None and x.device.type == "cuda":
            self._ws_streams.add(torch.cuda.current_stream(x.device).cuda_stream)
        if repeatable:
            fq_executor_set_repeatable(ex, True)
        self.repeatable = repeatable
        if kernel != KERNEL_AUTO:
            st = fq_executor_set_kernel(ex, kernel)
            if st != FQ_SUCCESS:
                self.destroy()
                raise FqError(st, f"fq_executor_set_kernel({kernel})")

    @property
    def kernel(self) -> int:
        return fq_executor_kernel(self.handle)

    def run(self, stream=None) -> None:
        torch = _torch()
        if self.handle is None:
            raise RuntimeError("executor already released")
        s = stream if stream is not None else torch.cuda.current_stream(self._keep[0].device)
        wsp = self.workspace.data_ptr() if self.workspace is not None else 0
        if self.workspace is not None and s.cuda_stream not in self._ws_streams:
            # The workspace was allocated on the planning thread's current stream; the
            # kernels may run on another one.  Tell the caching allocator (once per stream:
            # it keeps the set until the block is freed), so that a workspace freed right
            # after this call (quantize() drops its executor) is not handed to work on the
            # allocating stream while these kernels still use it.
            self.workspace.record_stream(s)
            self._ws_streams.add(s.cuda_stream)
        st = fq_run(wsp, self.workspace_size, self.handle, s.cuda_stream)
        if not self.repeatable:
            self.handle = None
        if st != FQ_SUCCESS:
            raise FqError(st, "fq_run")

    def destroy(self) -> None:
        if self.handle is not None:
            fq_executor_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def quantize(x, p1, p2, out, quant_scale, mode: str, clip_ratio: float = 1.0,
             dst_type_max: float = 0.0, stream=None, kernel: int = KERNEL_AUTO) -> None:
    """One fused call: plan (single-use executor) and enqueue on `stream`."""
    _same_gpu(stream, x, p1, None if p2 is None or p2.numel() == 0 else p2, out, quant_scale)
    ex = _new(stream, lambda: Executor(x, p1, p2, out, quant_scale, mode, clip_ratio, dst_type_max, kernel=kernel,
                                       repeatable=False), result=False)  # (its workspace)
    ex.run(stream)


def dequantize(codes, quant_scale, mode: str, M: int, N: int, dtype, out=None, stream=None):
    """Values of quantizer outputs (as stored by ``empty_outputs``) in ``dtype``
    (torch.bfloat16 or torch.float16): a [K, M, N] tensor, ``out`` when given."""
    torch = _torch()
    K = codes.shape[0]
    _same_gpu(stream, codes, quant_scale, out)
    if out is None:
        out = _new(stream, lambda: torch.empty((K, M, N), dtype=dtype, device=codes.device))
    dt = {torch.float16: DT_FLOAT16, torch.bfloat16: DT_BFLOAT16}.get(out.dtype, -1)
    st = fq_dequant(describe_out(codes, mode, K, M, N), describe_scale(quant_scale, mode),
                    make_tensor(out.data_ptr(), dt, out.shape, out.stride()),
                    (stream if stream is not None else torch.cuda.current_stream(codes.device)).cuda_stream)
    if st != FQ_SUCCESS:
        raise FqError(st, "fq_dequant")
    return out


def mx_gemm(a_codes, a_scale, w_codes, w_scale, H: int, out_dtype=None, out=None, stream=None):
    """C [T, O] = A . W^T for operands in the quantizer's per-group storage: codes uint8
    [rows, H/2] (or the fp4 out of ``empty_outputs``), e8m0 uint8 [rows, ceilDiv(H, 64), 2].
    C is torch.bfloat16 (default) or torch.float32."""
    torch = _torch()
    for t in (a_codes, a_scale, w_codes, w_scale):
        if not t.is_contiguous():
            raise ValueError("mx_gemm operands must be contiguous")
    _same_gpu(stream, a_codes, a_scale, w_codes, w_scale, out)
    T, O = a_codes.shape[0], w_codes.shape[0]
    if out is None:
        out = _new(stream, lambda: torch.empty((T, O), dtype=out_dtype or torch.bfloat16, device=a_codes.device))
    cdt = {torch.bfloat16: DT_BFLOAT16, torch.float32: DT_FLOAT32}.get(out.dtype, -1)
    G = -(-H // 64)
    st = fq_mx_gemm(make_tensor(a_codes.data_ptr(), DT_FLOAT4_E2M1, (T, H)),
                    make_tensor(a_scale.data_ptr(), DT_FLOAT8_E8M0, (T, G, 2)),
                    make_tensor(w_codes.data_ptr(), DT_FLOAT4_E2M1, (O, H)),
                    make_tensor(w_scale.data_ptr(), DT_FLOAT8_E8M0, (O, G, 2)),
                    make_tensor(out.data_ptr(), cdt, out.shape, out.stride()),
                    (stream if stream is not None else torch.cuda.current_stream(a_codes.device)).cuda_stream)
    if st != FQ_SUCCESS:
        raise FqError(st, "fq_mx_gemm")
    return out


def int4_gemm(a_codes, a_scale, w_codes, w_scale, H: int, out_dtype=None, out=None, stream=None):
    """C [T, O] = a_scale[t] w_scale[o] (A . W^T) for int4 codes in the quantizer's per-token
    storage: codes uint8 [rows, H/2] (the int4 / int32 out of ``empty_outputs`` viewed as
    bytes), scales float32 [rows].  C is torch.bfloat16 (default) or torch.float32."""
    torch = _torch()
    for t in (a_codes, a_scale, w_codes, w_scale):
        if not t.is_contiguous():
            raise ValueError("int4_gemm operands must be contiguous")
    _same_gpu(stream, a_codes, a_scale, w_codes, w_scale, out)
    T, O = a_codes.shape[0], w_codes.shape[0]
    if out is None:
        out = _new(stream, lambda: torch.empty((T, O), dtype=out_dtype or torch.bfloat16, device=a_codes.device))
    cdt = {torch.bfloat16: DT_BFLOAT16, torch.float32: DT_FLOAT32}.get(out.dtype, -1)
    st = fq_int4_gemm(make_tensor(a_codes.data_ptr(), DT_INT4, (T, H)),
                      make_tensor(a_scale.data_ptr(), DT_FLOAT32, (T,)),
                      make_tensor(w_codes.data_ptr(), DT_INT4, (O, H)),
                      make_tensor(w_scale.data_ptr(), DT_FLOAT32, (O,)),
                      make_tensor(out.data_ptr(), cdt, out.shape, out.stride()),
                      (stream if stream is not None else torch.cuda.current_stream(a_codes.device)).cuda_stream)
    if st != FQ_SUCCESS:
        raise FqError(st, "fq_int4_gemm")
    return out


def int8_gemm(a_codes, a_scale, w_codes, w_scale, out_dtype=None, out=None, stream=None):
    """C [T, O] = a_scale[t] w_scale[o] (A . W^T) for int8 codes: torch.int8 [rows, H] (the int8 out of ``empty_outputs``
    viewed as [K, M*N], say), scales float32 [rows].  C is torch.bfloat16 (default), torch.float16 or torch.float32."""
    torch = _torch()
    _same_gpu(stream, a_codes, a_scale, w_codes, w_scale, out)
    if out is None:
        make = lambda: torch.empty((a_codes.shape[0], w_codes.shape[0]), dtype=out_dtype or torch.bfloat16, device=a_codes.device)  # noqa: E731
        out = make() if stream is None else _new(stream, make)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out is of another type than out_dtype")
    d = _Descs(a_codes, a_scale, w_codes, w_scale, out)
    _call(lib.fq_int8_gemm, "fq_int8_gemm", a_codes.device, *d.ptrs, _stream(stream, a_codes.device))
    return out


# ---- paged key-value cache and attention ---------------------------------------------------

_DESC_BYTES = 80  # sizeof(fq_tensor): data, dtype, ndim, shape[4], strides[4]
# by number of dimensions (the unused sizes and strides are padding, left at 0)
_DESC = tuple(struct.Struct(f"=Qii{n}q{8 * (4 - n)}x{n}q{8 * (4 - n)}x") for n in range(5))
_codes = {}  # torch dtype -> fq_dtype, filled on first use


def _dtype_codes():
    if not _codes:
        torch = _torch()
        _codes.update({torch.float16: DT_FLOAT16, torch.bfloat16: DT_BFLOAT16, torch.float32: DT_FLOAT32,
                       torch.int32: DT_INT32, torch.int8: DT_INT8, torch.float8_e4m3fn: DT_FLOAT8_E4M3FN})
    return _codes


class _Descs:
    """fq_tensor descriptors of a call's tensors side by side in one buffer, passed by address (a
    call builds them anew, so building is kept cheap); None gives a null pointer."""
    __slots__ = ("raw", "ptrs")

    def __init__(self, *tensors):
        n = len(tensors)
        self.raw = raw = ctypes.create_string_buffer(n * _DESC_BYTES)
        at = ctypes.addressof(raw)
        codes = _codes or _dtype_codes()
        self.ptrs = ptrs = []
        for i, t in enumerate(tensors):
            if t is None:
                ptrs.append(None)
                continue
            shape = t.shape
            # (an unknown dtype, or more than four dimensions, is for the library's checks to refuse)
            nd = len(shape)
            if nd <= 4:
                _DESC[nd].pack_into(raw, i * _DESC_BYTES, t.data_ptr(), codes.get(t.dtype, -1), nd, *shape, *t.stride())
            else:
                _DESC[0].pack_into(raw, i * _DESC_BYTES, t.data_ptr(), -1, nd)
            ptrs.append(at + i * _DESC_BYTES)


class _Desc:
    """One descriptor with a given dtype, sizes and strides."""
    __slots__ = ("raw", "ptr")

    def __init__(self, data_ptr, dtype, shape, strides):
        self.raw = ctypes.create_string_buffer(_DESC[len(shape)].pack(data_ptr, dtype, len(shape), *shape, *strides), _DESC_BYTES)
        self.ptr = ctypes.addressof(self.raw)


def _same_device(first, *others):
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError(f"tensors on {first.device} and {t.device} in one call")


def _same_gpu(stream, first, *others):
    """The checks of a launching call: all tensors on one GPU (a host address must not reach a kernel), the
    caller's stream one of that GPU's."""
    d = first.get_device()
    if d < 0:
        raise ValueError(f"tensors on {first.device}: this call runs on a GPU")
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError(f"tensors on {first.device} and {t.device} in one call")
    if stream is not None and stream.device != first.device:
        raise ValueError(f"a stream of {stream.device} for tensors on {first.device}")


def _call(fn, name, device, *args):
    """A launching call, on the tensors' device whichever is current."""
    torch = _torch()
    if device.type == "cuda" and device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            st = fn(*args)
    else:
        st = fn(*args)
    if st != FQ_SUCCESS:
        raise FqError(st, name)


_raw_stream = []  # the function that gives a device's current stream as a handle


def _stream(stream, device):
    """The stream's handle; of the current stream without building a Stream object, where torch can (2 us less a call)."""
    if stream is not None:
        return stream.cuda_stream or None
    if not _raw_stream:
        torch = _torch()
        torch.cuda.current_stream(device)  # (initialises)
        _raw_stream.append(getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream))
    return _raw_stream[0](device.index) or None


def _new(stream, make, result=True):
    """What ``make()`` allocates, for work on the caller's `stream`: out of that stream's own pool, so that
    whatever held the memory before is done when the work begins (a block of the current stream's pool may
    still be in use by kernels that the caller's stream does not wait for).  A result is read on the current
    stream as a rule, so its memory also waits for that one when it is freed."""
    torch = _torch()
    if stream is None:
        return make()
    current = torch.cuda.current_stream(stream.device)
    if stream == current:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    if result:
        t.record_stream(current)
    return t


KV_MODES = ("f16", "bf16", "int8", "e4m3", "int4", "fp4")


class KVCache:
    """The two sides of a paged key-value cache and their descriptors (include/fq.h).

    Storage, P tokens a page: ``f16`` / ``bf16`` codes of that dtype [pages, Hkv, P, D], no
    scales; ``int8`` torch.int8 and ``e4m3`` torch.float8_e4m3fn (or uint8) [pages, Hkv, P, D],
    ``int4`` uint8 [pages, Hkv, P, D/2], each with float32 scales [pages, Hkv, P]; ``fp4`` uint8
    [pages, Hkv, P, D/2] with uint8 e8m0 scales [pages, Hkv, P, 2 * ceilDiv(D, 64)].  The
    first dimension may be strided (both sides in one allocation).

    ``k``, ``v``, ``k_scale`` and ``v_scale`` are the tensors it was made of and cannot be replaced (other
    tensors are another cache); memory that one of them moves to (``resize_``, ``set_``) is followed."""

    def __init__(self, mode: str, k, v, k_scale=None, v_scale=None):
        if mode not in KV_MODES:
            raise ValueError(f"unknown cache mode {mode!r}")
        _same_device(k, v, k_scale, v_scale)
        self.mode, self.device = mode, k.device
        self._tensors = (k, v, k_scale, v_scale)
        self._describe()

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    def _describe(self):
        torch = _torch()
        mode, (k, v, k_scale, v_scale) = self.mode, self._tensors
        codes = {"f16": (torch.float16,), "bf16": (torch.bfloat16,), "int8": (torch.int8, torch.uint8),
                 "e4m3": (torch.float8_e4m3fn, torch.uint8)}.get(mode, (torch.uint8,))
        scales = None if mode in ("f16", "bf16") else torch.uint8 if mode == "fp4" else torch.float32
        dt = {"f16": DT_FLOAT16, "bf16": DT_BFLOAT16, "int8": DT_INT8, "e4m3": DT_FLOAT8_E4M3FN, "int4": DT_INT4,
              "fp4": DT_FLOAT4_E2M1}[mode]
        sdt = DT_FLOAT8_E8M0 if mode == "fp4" else DT_FLOAT32

        def side(c, s):
            if c.dim() != 4 or c.dtype not in codes or (s is None) != (scales is None) or (s is not None and s.dtype != scales):
                raise ValueError(f"storage of a {mode} cache: see KVCache")
            shape, st = list(c.shape), list(c.stride())
            if mode in ("int4", "fp4"):  # two codes a byte: sizes and strides in codes
                shape[3] *= 2
                st = [2 * n for n in st[:3]] + [1 if st[3] == 1 else 2 * st[3]]
            return _Desc(c.data_ptr(), dt, shape, st), None if s is None else _Desc(s.data_ptr(), sdt, s.shape, s.stride())

        at = tuple((t.data_ptr, t.data_ptr()) for t in self._tensors if t is not None)
        (self._kc, self._ks), (self._vc, self._vs) = side(k, k_scale), side(v, v_scale)
        self.pages, self.heads, self.page_size = k.shape[:3]
        self.head_dim = k.shape[3] * (2 if mode in ("int4", "fp4") else 1)
        self._ptrs = (self._kc.ptr, self._ks.ptr if self._ks else None, self._vc.ptr, self._vs.ptr if self._vs else None)
        self._at = at

    def _args(self):
        """Addresses of the four descriptors of a call (built anew where a tensor's memory has moved)."""
        for address, was in self._at:
            if address() != was:
                self._describe()
                break
        return self._ptrs


def empty_kv_cache(pages: int, heads: int, page_size: int, head_dim: int, mode: str, device="cuda") -> KVCache:
    """A cache with uninitialised contents."""
    torch = _torch()
    if mode not in KV_MODES:
        raise ValueError(f"unknown cache mode {mode!r}")
    shape = (pages, heads, page_size)
    dt = {"f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}.get(mode, torch.uint8)
    codes = lambda: torch.empty(shape + (head_dim // 2 if mode in ("int4", "fp4") else head_dim,), dtype=dt, device=device)  # noqa: E731

    def scales():
        if mode in ("f16", "bf16"):
            return None
        if mode == "fp4":
            return torch.empty(shape + (2 * (-(-head_dim // 64)),), dtype=torch.uint8, device=device)
        return torch.empty(shape, dtype=torch.float32, device=device)

    return KVCache(mode, codes(), codes(), scales(), scales())


def kv_write(cache: KVCache, k, v, slots, clip_ratio: float = 1.0, dst_type_max: float = 0.0, stream=None) -> None:
    """Quantize rows k, v [T, Hkv, D] (bfloat16 or float16) into the cache at slots [T] (int32:
    page * page_size + offset; negative: not written)."""
    _same_gpu(stream, cache.k, k, v, slots)
    d = _Descs(k, v, slots)
    _call(lib.fq_kv_write, "fq_kv_write", cache.device, *d.ptrs, clip_ratio, dst_type_max, *cache._args(), _stream(stream, cache.device))


def kv_read(cache: KVCache, block_table, cu_seqlens, total: int, dtype, k_out=None, v_out=None, stream=None):
    """The cached tokens of every sequence as values: (k, v) [total, Hkv, D] of ``dtype``,
    sequence b in rows cu_seqlens[b] .. cu_seqlens[b+1]-1 (int32 [B+1]); block_table int32
    [B, pages per sequence]."""
    torch = _torch()
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    _same_gpu(stream, cache.k, block_table, cu_seqlens, k_out, v_out)
    held = cache._args()
    if k_out is None:
        make = lambda: torch.empty((total, cache.heads, cache.head_dim), dtype=dtype, device=cache.device)  # noqa: E731
        k_out, v_out = (make(), make()) if stream is None else (_new(stream, make), _new(stream, make))
    elif k_out.dtype != dtype or v_out.dtype != dtype or k_out.shape[0] != total or v_out.shape[0] != total:
        raise ValueError("k_out and v_out are [total, Hkv, D] of dtype")
    d = _Descs(block_table, cu_seqlens, k_out, v_out)
    _call(lib.fq_kv_read, "fq_kv_read", cache.device, *held, *d.ptrs, _stream(stream, cache.device))
    return k_out, v_out


def qk_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False, axes=None,
            q_out=None, k_out=None, stream=None):
    """Queries q [T, Hq, D] and keys k [T, Hkv, D] (one 16-bit dtype; either may be None), each row divided by its root
    mean square where its side has a weight [D] (float32 or 16-bit), then the pairs of its first 2 * len(inv_freq) elements
    turned by positions * inv_freq: pairs (i, i + R/2), or (2i, 2i + 1) interleaved.  positions int32 [T]; with ``axes``
    (int32 [R/2]: the axis of each pair) int32 [A, T].  inv_freq float32 [R/2].  Returns (q_out, k_out); an output may be
    its own input."""
    torch = _torch()
    if q is None and k is None:
        raise ValueError("neither queries nor keys")
    first = q if q is not None else k
    _same_gpu(stream, first, k, positions, inv_freq, q_weight, k_weight, axes, q_out, k_out)
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("an output without its input")

    def result(x, out):
        if x is None or out is not None:
            return out
        make = lambda: torch.empty_like(x, memory_format=torch.contiguous_format)  # noqa: E731
        return make() if stream is None else _new(stream, make)

    q_out, k_out = result(q, q_out), result(k, k_out)
    d = _Descs(q, k, q_weight, k_weight, positions, inv_freq, axes, q_out, k_out)
    p = d.ptrs
    _call(lib.fq_qk_rope, "fq_qk_rope", first.device, *p[:4], eps, *p[4:7], 1 if interleaved else 0, *p[7:], _stream(stream, first.device))
    return q_out, k_out


def kv_append(cache: KVCache, q, k, v, slots, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
              interleaved: bool = False, axes=None, clip_ratio: float = 1.0, dst_type_max: float = 0.0, q_out=None, stream=None):
    """qk_rope on q (may be None) and k, and kv_write of the turned keys and of v at slots [T], in one launch; the keys are
    quantized from unrounded rows.  Returns q_out."""
    torch = _torch()
    _same_gpu(stream, cache.k, q, k, v, slots, positions, inv_freq, q_weight, k_weight, axes, q_out)
    if q is None and q_out is not None:
        raise ValueError("an output without its input")
    if q is not None and q_out is None:
        make = lambda: torch.empty_like(q, memory_format=torch.contiguous_format)  # noqa: E731
        q_out = make() if stream is None else _new(stream, make)
    d = _Descs(q, k, v, slots, q_weight, k_weight, positions, inv_freq, axes, q_out)
    p = d.ptrs
    _call(lib.fq_kv_append, "fq_kv_append", cache.device, *p[:6], eps, *p[6:9], 1 if interleaved else 0, clip_ratio, dst_type_max,
          *cache._args(), p[9], _stream(stream, cache.device))
    return q_out


def _workspace(fn, name, device, stream, given, *args):
    """(tensor, pointer, bytes) of the workspace that `fn` asks for; `given` if the caller has one."""
    size = ctypes.c_uint64(0)
    st = fn(*args, ctypes.byref(size))
    if st != FQ_SUCCESS:
        raise FqError(st, name)
    if given is not None:
        if not given.is_contiguous():
            raise ValueError("a workspace is contiguous memory")
        return given, given.data_ptr(), given.numel() * given.element_size()
    if size.value == 0:
        return None, None, 0
    torch = _torch()
    ws = _new(stream, lambda: torch.empty((size.value,), dtype=torch.uint8, device=device), result=False)
    return ws, ws.data_ptr(), size.value


def attn_decode(q, cache: KVCache, block_table, lengths, scale: float = 0.0, out=None, lse=None, workspace=None,
                stream=None):
    """Attention of one new token per sequence: q [B, Hq, D] over the first lengths[b] (int32
    [B]) cached tokens of sequence b; Hq a multiple of the cache's heads.  scale 0 means
    1/sqrt(D).  ``lse`` (float32 [B, Hq]), when given, receives the log of the softmax's sum.
    ``workspace`` (uint8, at least attn_decode_workspace_size) may be passed to reuse one."""
    torch = _torch()
    _same_gpu(stream, cache.k, q, block_table, lengths, out, lse, workspace)
    if out is None:
        make = lambda: torch.empty_like(q, memory_format=torch.contiguous_format)  # noqa: E731
        out = make() if stream is None else _new(stream, make)
    d = _Descs(q, block_table, lengths, out, lse)
    qp, bp, lp, op, sp = d.ptrs
    held = cache._args()
    ws, ptr, size = _workspace(lib.fq_attn_decode_get_workspace_size, "fq_attn_decode_get_workspace_size", cache.device, stream,
                               workspace, qp, held[0], bp)
    _call(lib.fq_attn_decode, "fq_attn_decode", cache.device, qp, *held, bp, lp, scale, op, sp, ptr, size,
          _stream(stream, cache.device))
    return out


def attn_decode_workspace_size(q, cache: KVCache, block_table) -> int:
    size = ctypes.c_uint64(0)
    d = _Descs(q, block_table)
    st = lib.fq_attn_decode_get_workspace_size(d.ptrs[0], cache._args()[0], d.ptrs[1], ctypes.byref(size))
    if st != FQ_SUCCESS:
        raise FqError(st, "fq_attn_decode_get_workspace_size")
    return size.value


def attn_prefill_workspace_size(q, k, cu_q, causal: bool = True) -> int:
    size = ctypes.c_uint64(0)
    d = _Descs(q, k, cu_q)
    st = lib.fq_attn_prefill_get_workspace_size(*d.ptrs, 1 if causal else 0, ctypes.byref(size))
    if st != FQ_SUCCESS:
        raise FqError(st, "fq_attn_prefill_get_workspace_size")
    return size.value


def attn_prefill(q, k, v, cu_q, cu_k=None, causal: bool = True, scale: float = 0.0, out=None, lse=None, workspace=None,
                 stream=None):
    """Attention over packed sequences: q [Tq, Hq, D], k, v [Tk, Hkv, D] (one 16-bit dtype),
    sequence b in rows cu_q[b] .. cu_q[b+1]-1 of q and cu_k[b] .. cu_k[b+1]-1 of k and v (int32
    [B+1]; cu_k defaults to cu_q).  Causal: row i sees keys up to (Lk - Lq) + i.  scale 0 means
    1/sqrt(D).  ``lse``: float32 [Tq, Hq].  ``workspace`` (uint8, at least
    attn_prefill_workspace_size) may be passed to reuse one."""
    torch = _torch()
    if cu_k is None:
        cu_k = cu_q
    _same_gpu(stream, q, k, v, cu_q, cu_k, out, lse, workspace)
    if out is None:
        make = lambda: torch.empty_like(q, memory_format=torch.contiguous_format)  # noqa: E731
        out = make() if stream is None else _new(stream, make)
    d = _Descs(q, k, v, cu_q, cu_k, out, lse)
    qp, kp, vp, ap, bp, op, sp = d.ptrs
    causal = 1 if causal else 0
    ws, ptr, size = _workspace(lib.fq_attn_prefill_get_workspace_size, "fq_attn_prefill_get_workspace_size", q.device, stream,
                               workspace, qp, kp, ap, causal)
    _call(lib.fq_attn_prefill, "fq_attn_prefill", q.device, qp, kp, vp, ap, bp, causal, scale, op, sp, ptr, size,
          _stream(stream, q.device))
    return out


def _int32(n) -> int:
    """n, held to what an int32 can say of a length (ctypes keeps the low bits of any other)."""
    return max(-1, min(int(n), 2 ** 31 - 1))


def attn_chunk_workspace_size(q, cache: KVCache, block_table, cu_q, window: int = 0, sinks: int = 0) -> int:
    size = ctypes.c_uint64(0)
    d = _Descs(q, block_table, cu_q)
    st = lib.fq_attn_chunk_get_workspace_size(d.ptrs[0], cache._args()[0], d.ptrs[1], d.ptrs[2], _int32(window), _int32(sinks),
                                                ctypes.byref(size))
    if st != FQ_SUCCESS:
        raise FqError(st, "fq_attn_chunk_get_workspace_size")
    return size.value


def attn_chunk(q, cache: KVCache, block_table, cu_q, lengths, window: int = 0, sinks: int = 0, scale: float = 0.0, out=None,
               lse=None, workspace=None, stream=None):
    """Attention of new tokens over the cache, which holds their keys and values already: q [Tq, Hq, D], sequence b in rows
    cu_q[b] .. cu_q[b+1]-1 (int32 [B+1]), its last row at the last of its lengths[b] tokens (int32 [B]).  A row sees the keys up to its
    own position; with ``window`` only the last ``window`` of them and the first ``sinks`` tokens.  scale 0 means 1/sqrt(D).
    ``lse``: float32 [Tq, Hq].  ``workspace`` (uint8, at least attn_chunk_workspace_size) may be passed to reuse one.  Long chunks and
    single tokens can share a call, and take less time in calls of their own."""
    torch = _torch()
    window, sinks = _int32(window), _int32(sinks)
    _same_gpu(stream, cache.k, q, block_table, cu_q, lengths, out, lse, workspace)
    if out is None:
        make = lambda: torch.empty_like(q, memory_format=torch.contiguous_format)  # noqa: E731
        out = make() if stream is None else _new(stream, make)
    d = _Descs(q, block_table, cu_q, lengths, out, lse)
    qp, bp, ap, lp, op, sp = d.ptrs
    held = cache._args()
    ws, ptr, size = _workspace(lib.fq_attn_chunk_get_workspace_size, "fq_attn_chunk_get_workspace_size", cache.device, stream, workspace,
                               qp, held[0], bp, ap, window, sinks)
    _call(lib.fq_attn_chunk, "fq_attn_chunk", cache.device, qp, *held, bp, ap, lp, window, sinks, scale, op, sp, ptr, size,
          _stream(stream, cache.device))
    return out
