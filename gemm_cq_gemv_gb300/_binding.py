"""ctypes binding of ``libcqgemv.so`` (argument marshalling only).

Every function here has the name of the C entry point it calls (``include/cqgemv.h``),
takes CUDA tensors, checks dtype / device / contiguity / shape, passes raw device
pointers and sizes across the C ABI and raises ``CQError`` on a non-OK status.  All
arithmetic runs in the library's CUDA kernels; there is no fallback of any kind: if
the shared library is missing or does not load, every call raises.

``stream`` (a ``torch.cuda.Stream`` or a raw handle) is where a call launches, the current
stream by default.  Outputs and workspaces that the call allocates come from that stream's
memory, as if it were the current one.
"""

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcqgemv.so")

CQ_OK = 0
_STATUS = {0: "CQ_OK", 1: "CQ_ERR_INVALID_ARG", 2: "CQ_ERR_ALIGNMENT", 3: "CQ_ERR_UNSUPPORTED",
           4: "CQ_ERR_CUDA", 5: "CQ_ERR_DEVICE_TIMEOUT", 6: "CQ_ERR_WORKSPACE"}


class CQError(RuntimeError):
    def __init__(self, fn, status, cuda_err=0):
        name = _STATUS.get(status, f"status {status}")
        msg = f"{fn} failed: {name}"
        if status == 4:
            msg += f" (cudaError {cuda_err})"
        super().__init__(msg)
        self.status = status


class cq_codebook(ctypes.Structure):
    _fields_ = [("cb", ctypes.c_float * 28)]


class cq_gemm_problem(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("norms", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("Xq", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("Y", ctypes.c_void_p)]


class cq_gemv_problem(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("norms", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("X", ctypes.c_void_p), ("Y", ctypes.c_void_p)]


class q4_0_gemv_problem(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("X", ctypes.c_void_p), ("Y", ctypes.c_void_p)]


LAYER_MAX_PROBLEMS = 16   # CQ_LAYER_MAX_PROBLEMS
LAYER_MAX_K = 8192        # CQ_LAYER_MAX_K

F8_GROUP = 128            # values per F8 scale
MOE_MAX_EXPERTS = 1024    # CQ_MOE_MAX_EXPERTS
MOE_MAX_K = 32            # CQ_MOE_MAX_K
MOE_ONE_LAUNCH = 512      # CQ_MOE_ONE_LAUNCH

_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_SZ = ctypes.c_size_t

# name -> (restype, argtypes)
SIGNATURES = {
    "cq_status_string": (ctypes.c_char_p, [_INT]),
    "cq_last_cuda_error": (_INT, []),
    "cq_abi_version": (_INT, []),
    "cq_levels": (_INT, [_INT, ctypes.POINTER(cq_codebook), _P]),
    "cq_codebook_fit": (_INT, [_P, _I64, _INT, _INT, _P, _P]),
    "cq_encode": (_INT, [_P, _I64, _I64, _INT, _INT, ctypes.POINTER(cq_codebook), _P, _P, _P]),
    "a8_quantize": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "a8_quantize_groups": (_INT, [_P, _I64, _I64, _INT, _P, _P, _P]),
    "a8_fake_quant_groups": (_INT, [_P, _I64, _I64, _INT, _P, _P]),
    "cq_gemv_workspace_bytes": (_SZ, [_I64, _I64]),
    "cq_gemv": (_INT, [_P, _P, _I64, _I64, _INT, _INT, ctypes.POINTER(cq_codebook), _P, _P, _I64,
                       _P, _P, _SZ, _P]),
    "cq_gemv_noalloc": (_INT, [_P, _P, _I64, _I64, _INT, _INT, ctypes.POINTER(cq_codebook), _P,
                               _P, _I64, _P, _P]),
    "cq_gemv_lut": (_INT, [_P, _P, _I64, _I64, _INT, _INT, ctypes.POINTER(cq_codebook), _P, _P,
                           _I64, _P, _P]),
    "cq_gemm_workspace_bytes": (_SZ, [_I64, _I64]),
    "cq_gemm": (_INT, [_P, _P, _I64, _I64, _INT, _INT, ctypes.POINTER(cq_codebook), _P, _P, _I64,
                       _P, _P, _SZ, _P]),
    "cq_gemm_grouped_workspace_bytes": (_SZ, [ctypes.POINTER(cq_gemm_problem), _INT, _I64]),
    "cq_gemm_grouped": (_INT, [ctypes.POINTER(cq_gemm_problem), _INT, _I64, _INT, _INT,
                               ctypes.POINTER(cq_codebook), _P, _SZ, _P]),
    "cq_device_error": (_INT, [_P]),
    "cq_probe_bounded_wait": (_INT, [ctypes.c_uint64, _P]),
    "q4_0_quantize": (_INT, [_P, _I64, _I64, _P, _P]),
    "q4_0_gemv": (_INT, [_P, _I64, _I64, _P, _I64, _P, _P]),
    "q4_0_gemm_workspace_bytes": (_SZ, [_I64, _I64]),
    "q4_0_gemm": (_INT, [_P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P]),
    "cq_gemv_layer": (_INT, [ctypes.POINTER(cq_gemv_problem), _INT, _INT, _INT,
                             ctypes.POINTER(cq_codebook), _I64, _P]),
    "q4_0_gemv_layer": (_INT, [ctypes.POINTER(q4_0_gemv_problem), _INT, _I64, _P]),
    "f8_quantize_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "f8_quantize": (_INT, [_P, _INT, _I64, _I64, _P, _I64, _P, _P, _P, _SZ, _P]),
    "f8_quantize_weights": (_INT, [_P, _INT, _I64, _I64, _I64, _P, _P, _P]),
    "f8_gemm": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _INT, _P, _INT, _P]),
    "f8_gemm_experts": (_INT, [_P, _P, _I64, _I64, _I64, _P, _P, _P, _I64, _INT, _P, _INT, _P]),
    "f8_gemm_plan": (_INT, [_I64, _I64, _I64, _I64, _INT, _INT, _P]),
    "moe_route_workspace_bytes": (_SZ, [_I64, _I64]),
    "moe_route": (_INT, [_P, _I64, _I64, _INT, _INT, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_combine": (_INT, [_P, _INT, _I64, _I64, _P, _P, _I64, _INT, _P, _INT, _P]),
}


def lib():
    """Load ``libcqgemv.so`` (once).  Raises if it is missing: nothing runs without it."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; "
                "g.build()\"` (nvcc, sm_103a). There is no fallback implementation.")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _on(stream, device):
    """The context in which what a call launched on ``stream`` allocates is that stream's memory.
    Memory of the current stream's pool would not do for another one: work queued there may
    still use the block, and a workspace dropped on return would be handed out again before
    the kernels have run."""
    if not isinstance(stream, torch.cuda.Stream):
        # ExternalStream(0) would be a new stream
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    """``torch.empty`` for a call launched on ``stream``."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _ptr(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    return ctypes.c_void_p(t.data_ptr())


def _check(fn, status):
    if status != CQ_OK:
        raise CQError(fn, status, lib().cq_last_cuda_error())


def make_codebook(cb28):
    """Build the C ``cq_codebook`` from 28 floats (``cb2 | cb3 | cb4``)."""
    vals = [float(v) for v in (cb28.tolist() if hasattr(cb28, "tolist") else cb28)]
    if len(vals) != 28:
        raise ValueError("codebook needs 28 floats (cb2[4] | cb3[8] | cb4[16])")
    c = cq_codebook()
    for i, v in enumerate(vals):
        c.cb[i] = v
    return c


def _cbk(cb):
    return cb if isinstance(cb, cq_codebook) else make_codebook(cb)


def cq_status_string(status: int) -> str:
    return lib().cq_status_string(status).decode()


def cq_abi_version() -> int:
    return lib().cq_abi_version()


def cq_levels(b, cb=None):
    """The 16-entry float32 level table the CQ kernels use for code ``b`` (host only), as a
    list of 16 Python floats (each exactly a float32 value)."""
    out = (ctypes.c_float * 16)()
    c = ctypes.byref(_cbk(cb)) if cb is not None else None
    _check("cq_levels", lib().cq_levels(b, c, ctypes.cast(out, ctypes.c_void_p)))
    return list(out)


def cq_codebook_fit(samples, L, iters=200, levels_out=None, stream=None):
    """A1: Lloyd-Max levels (float32 [L]) from float64 samples on the GPU."""
    s = _ptr(samples, torch.float64, "samples")
    if levels_out is None:
        levels_out = _empty(L, torch.float32, samples.device, stream)
    _check("cq_codebook_fit", lib().cq_codebook_fit(s, samples.numel(), L, iters,
                                                     _ptr(levels_out, torch.float32, "levels_out"),
                                                     _stream(stream)))
    return levels_out


# CQ_TERNARY of the C header: bits = 5 selects the fixed codebook {-c, 0, +c}, whose
# indices are stored in 2-bit fields.
CQ_TERNARY = 5


def cq_field_bits(b: int) -> int:
    """Bits of one packed index field of code ``b`` (a group holds ``16 * field`` bytes)."""
    return 2 if b == CQ_TERNARY else b


def cq_encode(W, b, cb, packed=None, norms=None, g=128, stream=None):
    """A2: CQ-encode W [N, K] float32 -> (packed uint8 [N, K/128, 16 f], norms int16 [N, K/128]),
    f = ``cq_field_bits(b)``."""
    N, K = W.shape
    wp = _ptr(W, torch.float32, "W", 2)
    if packed is None:
        packed = _empty((N, K // 128, 16 * cq_field_bits(b)), torch.uint8, W.device, stream)
    if norms is None:
        norms = _empty((N, K // 128), torch.int16, W.device, stream)
    c = _cbk(cb)
    _check("cq_encode", lib().cq_encode(wp, N, K, g, b, ctypes.byref(c),
                                        _ptr(packed, torch.uint8, "packed"),
                                        _ptr(norms, torch.int16, "norms"), _stream(stream)))
    return packed, norms


def a8_quantize(X, Xq=None, scale=None, stream=None):
    """A3: X [B, K] float32 -> (Xq int8 [B, K], scale float32 [B])."""
    B, K = X.shape
    xp = _ptr(X, torch.float32, "X", 2)
    if Xq is None:
        Xq = _empty((B, K), torch.int8, X.device, stream)
    if scale is None:
        scale = _empty((B,), torch.float32, X.device, stream)
    _check("a8_quantize", lib().a8_quantize(xp, B, K, _ptr(Xq, torch.int8, "Xq"),
                                            _ptr(scale, torch.float32, "scale"), _stream(stream)))
    return Xq, scale


def a8_quantize_groups(X, G, codes=None, scales=None, stream=None):
    """Grouped A8: X [T, D] float32 -> (codes int8 [T, D], scales float32 [T, D/G])."""
    T, D = X.shape
    if codes is None:
        codes = _empty((T, D), torch.int8, X.device, stream)
    if scales is None:
        scales = _empty((T, D // G), torch.float32, X.device, stream)
    _check("a8_quantize_groups", lib().a8_quantize_groups(_ptr(X, torch.float32, "X", 2), T, D, G,
                                                          _ptr(codes, torch.int8, "codes"),
                                                          _ptr(scales, torch.float32, "scales"),
                                                          _stream(stream)))
    return codes, scales


def a8_fake_quant_groups(X, G, Y=None, stream=None):
    """Grouped A8 fake-quant: Y [T, D] float32 = q * s per group of G features."""
    T, D = X.shape
    if Y is None:
        Y = _empty((T, D), torch.float32, X.device, stream)
    _check("a8_fake_quant_groups", lib().a8_fake_quant_groups(_ptr(X, torch.float32, "X", 2), T, D, G,
                                                              _ptr(Y, torch.float32, "Y"), _stream(stream)))
    return Y


def cq_gemv_workspace_bytes(B, K) -> int:
    return int(lib().cq_gemv_workspace_bytes(B, K))


def cq_gemv(packed, norms, N, K, b, cb, Xq, scale, Y=None, workspace=None, g=128, stream=None):
    """A4+A5: Y [B, N] float32 = decode GEMV of CQ weights with int8 activations."""
    B = Xq.shape[0]
    if Y is None:
        Y = _empty((B, N), torch.float32, Xq.device, stream)
    need = cq_gemv_workspace_bytes(B, K)
    if workspace is None:
        workspace = _empty((max(need, 16),), torch.uint8, Xq.device, stream)
    c = _cbk(cb)
    _check("cq_gemv", lib().cq_gemv(_ptr(packed, torch.uint8, "packed"),
                                    _ptr(norms, torch.int16, "norms"), N, K, g, b, ctypes.byref(c),
                                    _ptr(Xq, torch.int8, "Xq"), _ptr(scale, torch.float32, "scale"),
                                    B, _ptr(Y, torch.float32, "Y"),
                                    _ptr(workspace, torch.uint8, "workspace"),
                                    workspace.numel(), _stream(stream)))
    return Y


def cq_gemv_lut(packed, norms, N, K, b, cb, Xq, scale, Y=None, g=128, stream=None):
    """A4+A5 by table lookup (b = 1, 2 or ternary): Y [B, N] float32, no workspace."""
    B = Xq.shape[0]
    if Y is None:
        Y = _empty((B, N), torch.float32, Xq.device, stream)
    c = _cbk(cb)
    _check("cq_gemv_lut", lib().cq_gemv_lut(_ptr(packed, torch.uint8, "packed"),
                                            _ptr(norms, torch.int16, "norms"), N, K, g, b,
                                            ctypes.byref(c), _ptr(Xq, torch.int8, "Xq"),
                                            _ptr(scale, torch.float32, "scale"), B,
                                            _ptr(Y, torch.float32, "Y"), _stream(stream)))
    return Y


def cq_gemm_workspace_bytes(M, K) -> int:
    return int(lib().cq_gemm_workspace_bytes(M, K))


def cq_gemm(packed, norms, N, K, b, cb, Xq, scale, Y=None, workspace=None, g=128, stream=None):
    """A4+A6: Y [M, N] bfloat16 = prefill GEMM of CQ weights with int8 activations."""
    M = Xq.shape[0]
    if Y is None:
        Y = _empty((M, N), torch.bfloat16, Xq.device, stream)
    need = cq_gemm_workspace_bytes(M, K)
    if workspace is None:
        workspace = _empty((max(need, 256),), torch.uint8, Xq.device, stream)
    c = _cbk(cb)
    _check("cq_gemm", lib().cq_gemm(_ptr(packed, torch.uint8, "packed"),
                                    _ptr(norms, torch.int16, "norms"), N, K, g, b, ctypes.byref(c),
                                    _ptr(Xq, torch.int8, "Xq"), _ptr(scale, torch.float32, "scale"),
                                    M, _ptr(Y, torch.bfloat16, "Y"),
                                    _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                                    _stream(stream)))
    return Y


def make_gemm_problems(items):
    """``items``: sequence of (packed, norms, N, K, Xq, scale, Y) tensors / ints."""
    arr = (cq_gemm_problem * len(items))()
    for i, (packed, norms, N, K, Xq, scale, Y) in enumerate(items):
        arr[i].packed = _ptr(packed, torch.uint8, "packed").value
        arr[i].norms = _ptr(norms, torch.int16, "norms").value
        arr[i].N, arr[i].K = N, K
        arr[i].Xq = _ptr(Xq, torch.int8, "Xq").value
        arr[i].scale = _ptr(scale, torch.float32, "scale").value
        arr[i].Y = _ptr(Y, torch.bfloat16, "Y").value
    return arr


def make_gemv_layer(items):
    """CQ layer problems from (packed, norms, N, K, X, Y) tuples: X [B][K] float32 and
    Y [B][N] float32 CUDA tensors.  The array keeps the tensors alive."""
    arr = (cq_gemv_problem * len(items))()
    for i, (packed, norms, N, K, X, Y) in enumerate(items):
        arr[i].packed = _ptr(packed, torch.uint8, "packed").value
        arr[i].norms = _ptr(norms, torch.int16, "norms").value
        arr[i].N, arr[i].K = N, K
        arr[i].X = _ptr(X, torch.float32, "X", 2).value
        arr[i].Y = _ptr(Y, torch.float32, "Y", 2).value
        if X.shape[1] != K or Y.shape != (X.shape[0], N):
            raise ValueError(f"problem {i}: X must be [B, {K}] and Y [B, {N}]")
    arr._keep = [t for it in items for t in it if isinstance(t, torch.Tensor)]
    arr._batch = items[0][4].shape[0]
    return arr


def make_q4_0_layer(items):
    """Q4_0 layer problems from (blocks, N, K, X, Y) tuples (X, Y as for make_gemv_layer)."""
    arr = (q4_0_gemv_problem * len(items))()
    for i, (blocks, N, K, X, Y) in enumerate(items):
        arr[i].blocks = _ptr(blocks, torch.uint8, "blocks").value
        arr[i].N, arr[i].K = N, K
        arr[i].X = _ptr(X, torch.float32, "X", 2).value
        arr[i].Y = _ptr(Y, torch.float32, "Y", 2).value
        if X.shape[1] != K or Y.shape != (X.shape[0], N):
            raise ValueError(f"problem {i}: X must be [B, {K}] and Y [B, {N}]")
    arr._keep = [t for it in items for t in it if isinstance(t, torch.Tensor)]
    arr._batch = items[0][3].shape[0]
    return arr


def cq_gemv_layer(problems, b, cb, g=128, stream=None):
    """Fused decode chain: a8 quantization, rotation and the CQ GEMV of every problem of a
    layer (an array from ``make_gemv_layer``) in one launch."""
    c = _cbk(cb)
    _check("cq_gemv_layer", lib().cq_gemv_layer(problems, len(problems), g, b, ctypes.byref(c),
                                                problems._batch, _stream(stream)))


def q4_0_gemv_layer(problems, stream=None):
    """Fused decode chain: the Q4_0 GEMV of every problem of a layer (an array from
    ``make_q4_0_layer``) in one launch."""
    _check("q4_0_gemv_layer", lib().q4_0_gemv_layer(problems, len(problems), problems._batch,
                                                    _stream(stream)))


def cq_gemm_grouped_workspace_bytes(problems, M) -> int:
    return int(lib().cq_gemm_grouped_workspace_bytes(problems, len(problems), M))


def cq_gemm_grouped(problems, M, b, cb, workspace=None, g=128, stream=None, device=None):
    """A6 grouped: every problem (a ``cq_gemm_problem`` array) in persistent launches."""
    need = cq_gemm_grouped_workspace_bytes(problems, M)
    if workspace is None:
        workspace = _empty((max(need, 256),), torch.uint8, device or torch.device("cuda"), stream)
    c = _cbk(cb)
    _check("cq_gemm_grouped", lib().cq_gemm_grouped(problems, len(problems), M, g, b,
                                                    ctypes.byref(c),
                                                    _ptr(workspace, torch.uint8, "workspace"),
                                                    workspace.numel(), _stream(stream)))
    return workspace


def cq_device_error(stream=None):
    """Raise CQError(CQ_ERR_DEVICE_TIMEOUT) if a bounded device wait gave up (clears it)."""
    _check("cq_device_error", lib().cq_device_error(_stream(stream)))


def cq_probe_bounded_wait(timeout_ns=20_000_000, stream=None):
    """Enqueue the failure-detection probe (bounded waits that nothing completes)."""
    _check("cq_probe_bounded_wait", lib().cq_probe_bounded_wait(int(timeout_ns), _stream(stream)))


NOALLOC_MAX_ELEMS = 1 << 20   # CQ_GEMV_NOALLOC_MAX_ELEMS


def cq_gemv_noalloc(packed, norms, N, K, b, cb, Xq, scale, Y=None, g=128, stream=None):
    """``cq_gemv`` for callers that cannot allocate a workspace: the library's fixed
    4 MiB scratch holds the rotated activations (B * K <= 2**20).  Calls that overlap on
    the GPU share that scratch and race; the first call on a device must precede any
    stream capture.  ``Y`` may be passed preallocated."""
    B = Xq.shape[0]
    if Y is None:
        Y = _empty((B, N), torch.float32, Xq.device, stream)
    c = _cbk(cb)
    _check("cq_gemv_noalloc", lib().cq_gemv_noalloc(
        _ptr(packed, torch.uint8, "packed"), _ptr(norms, torch.int16, "norms"), N, K, g, b,
        ctypes.byref(c), _ptr(Xq, torch.int8, "Xq"), _ptr(scale, torch.float32, "scale"), B,
        _ptr(Y, torch.float32, "Y"), _stream(stream)))
    return Y


def q4_0_quantize(W, blocks=None, stream=None):
    """A7: W [N, K] float32 -> Q4_0 blocks uint8 [N, ceil(K/32)*18]."""
    N, K = W.shape
    if blocks is None:
        blocks = _empty((N, ((K + 31) // 32) * 18), torch.uint8, W.device, stream)
    _check("q4_0_quantize", lib().q4_0_quantize(_ptr(W, torch.float32, "W", 2), N, K,
                                                _ptr(blocks, torch.uint8, "blocks"), _stream(stream)))
    return blocks


def q4_0_gemv(blocks, N, K, X, Y=None, stream=None):
    """A8: Y [B, N] float32 = Q4_0 decode GEMV with float32 activations X [B, K]."""
    B = X.shape[0]
    if Y is None:
        Y = _empty((B, N), torch.float32, X.device, stream)
    _check("q4_0_gemv", lib().q4_0_gemv(_ptr(blocks, torch.uint8, "blocks"), N, K,
                                        _ptr(X, torch.float32, "X"), B, _ptr(Y, torch.float32, "Y"),
                                        _stream(stream)))
    return Y


def q4_0_gemm_workspace_bytes(M, K) -> int:
    return int(lib().q4_0_gemm_workspace_bytes(M, K))


def q4_0_gemm(blocks, N, K, X, Y=None, workspace=None, stream=None):
    """Q4_0 GEMM on the tensor cores: Y [M, N] float32 for float32 activations X [M, K]
    (ceil(K/32) a multiple of 8)."""
    M = X.shape[0]
    if Y is None:
        Y = _empty((M, N), torch.float32, X.device, stream)
    need = q4_0_gemm_workspace_bytes(M, K)
    if workspace is None:
        workspace = _empty((max(need, 256),), torch.uint8, X.device, stream)
    _check("q4_0_gemm", lib().q4_0_gemm(_ptr(blocks, torch.uint8, "blocks"), N, K,
                                        _ptr(X, torch.float32, "X"), M, _ptr(Y, torch.float32, "Y"),
                                        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                                        _stream(stream)))
    return Y


# ---- F8 (e4m3 codes, one power-of-two scale per block of 128) and the expert layer ----------
# These calls serve single tokens, where a launch takes about 3 us and every check shows in the
# time of a step: one look at each tensor, addresses as plain integers, the stream's address
# without a Stream object, shapes worked out in place.

# absent from builds of torch without CUDA, where the package still imports
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def f8_row_bytes(K) -> int:
    """Code bytes of a row of K values: whole groups of 128."""
    return (K + F8_GROUP - 1) // F8_GROUP * F8_GROUP


def f8_scale_bytes(K) -> int:
    """Scale bytes of a row of K values: one per group, in whole words."""
    return (K + 4 * F8_GROUP - 1) // (4 * F8_GROUP) * 4


def _checked_stream(device):
    """Address of the current stream of the device, which has to be the current one: the library
    launches there."""
    if _current_device() != device:
        raise ValueError(f"the tensors are on CUDA device {device}, which is not the current one")
    return _current_stream(device)


def _raw_stream(device):
    """``_checked_stream``; where there is a single device, without the call that the check takes."""
    global _raw_stream
    _raw_stream = _current_stream if torch.cuda.device_count() == 1 else _checked_stream
    return _raw_stream(device)


def _device(t, name):
    """Device of a tensor, which the call's other tensors have to share; raises for one of the host."""
    device = t.get_device()
    if device < 0:
        _ptr(t, t.dtype, name)
    return device


def _at(t, dtype, shape, name, device):
    """Address of a contiguous tensor of this dtype and shape on this device; raises for any other."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _ptr(t, dtype, name)
    if t.get_device() != device:
        raise ValueError(f"{name} must be on CUDA device {device} like the call's other tensors, got {t.get_device()}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _float(t, name):
    """cq_dtype of a float32 or bfloat16 tensor; raises for anything else."""
    if isinstance(t, torch.Tensor):
        if t.dtype is _BF16:
            return 1
        if t.dtype is _F32:
            return 0
    raise TypeError(f"{name} must be a float32 or bfloat16 torch.Tensor")


def _dims(t, name, *ndims):
    """Shape of a tensor that must have one of these numbers of dims."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) not in ndims:
        raise ValueError(f"{name} must have {' or '.join(map(str, ndims))} dims")
    return shape


def f8_quantize_workspace_bytes(M, K, R) -> int:
    return int(lib().f8_quantize_workspace_bytes(M, K, R))


def f8_quantize(X, rows=None, codes=None, scales=None, workspace=None, stream=None):
    """X [M, K] float32 or bfloat16 -> (codes uint8 [R, Kp], scales uint8 [R, Ks]): e4m3 codes
    with one power-of-two scale per 128 values.  ``rows`` (int32 [R]) gathers: output row r
    comes from X[rows[r]]."""
    xt = _float(X, "X")
    M, K = shape = _dims(X, "X", 2)
    dev = _device(X, "X")
    xp = _at(X, X.dtype, shape, "X", dev)
    R, rp, wp, wn = M, None, None, 0
    if rows is not None:
        R, = shape = _dims(rows, "rows", 1)
        rp = _at(rows, _I32, shape, "rows", dev)
        if workspace is None and R * K >= 1 << 20:   # smaller gathers take none
            need = f8_quantize_workspace_bytes(M, K, R)
            workspace = _empty((need,), _U8, X.device, stream) if need else None
        if workspace is not None:
            wp, wn = _at(workspace, _U8, _dims(workspace, "workspace", 1), "workspace", dev), workspace.numel()
    cs, ss = (R, (K + 127) // 128 * 128), (R, (K + 511) // 512 * 4)
    if codes is None:
        codes = _empty(cs, _U8, X.device, stream)
    if scales is None:
        scales = _empty(ss, _U8, X.device, stream)
    status = (_lib or lib()).f8_quantize(
        xp, xt, M, K, rp, R, _at(codes, _U8, cs, "codes", dev), _at(scales, _U8, ss, "scales", dev), wp, wn,
        _raw_stream(dev) if stream is None else _stream(stream))
    if status:
        _check("f8_quantize", status)
    return codes, scales


def f8_quantize_weights(W, codes=None, scales=None, stream=None):
    """W [N, K] or [E, N, K] float32 or bfloat16 -> (codes uint8 [.., N, Kp], scales uint8
    [.., ceil(N / 128), Ks]): e4m3 codes with one power-of-two scale per 128 x 128 block."""
    wt = _float(W, "W")
    shape = _dims(W, "W", 2, 3)
    dev = _device(W, "W")
    wp = _at(W, W.dtype, shape, "W", dev)
    *lead, N, K = shape
    cs = (*lead, N, f8_row_bytes(K))
    ss = (*lead, (N + F8_GROUP - 1) // F8_GROUP, f8_scale_bytes(K))
    if codes is None:
        codes = _empty(cs, _U8, W.device, stream)
    if scales is None:
        scales = _empty(ss, _U8, W.device, stream)
    _check("f8_quantize_weights", lib().f8_quantize_weights(
        wp, wt, lead[0] if lead else 1, N, K, _at(codes, _U8, cs, "codes", dev), _at(scales, _U8, ss, "scales", dev),
        _raw_stream(dev) if stream is None else _stream(stream)))
    return codes, scales


def _gated(act):
    """cq_act of a name; raises for an unknown one."""
    if act == "none":
        return 0
    if act == "swiglu":
        return 1
    raise ValueError("act must be 'none' or 'swiglu'")


def f8_gemm(wcodes, wscales, N, K, xcodes, xscales, act="none", Y=None, stream=None):
    """Y [M, N] = x w^T of F8 rows and F8 weights (bfloat16 unless a float32 ``Y`` is passed).
    ``act="swiglu"``: Y [M, N / 2] = silu(gate) * up over interleaved weight rows (gate 2 j,
    up 2 j + 1)."""
    a, M, dev = _gated(act), _dims(xcodes, "xcodes", 2)[0], _device(xcodes, "xcodes")
    Kp, Ks, shape = (K + 127) // 128 * 128, (K + 511) // 512 * 4, (M, N >> a)
    if Y is None:
        Y = _empty(shape, _BF16, xcodes.device, stream)
    yt = _float(Y, "Y")
    status = (_lib or lib()).f8_gemm(
        _at(wcodes, _U8, (N, Kp), "wcodes", dev), _at(wscales, _U8, ((N + 127) // 128, Ks), "wscales", dev), N, K,
        _at(xcodes, _U8, (M, Kp), "xcodes", dev), _at(xscales, _U8, (M, Ks), "xscales", dev), M, a,
        _at(Y, Y.dtype, shape, "Y", dev), yt, _raw_stream(dev) if stream is None else _stream(stream))
    if status:
        _check("f8_gemm", status)
    return Y


def f8_gemm_experts(wcodes, wscales, N, K, offsets, xcodes, xscales, act="none", Y=None, stream=None):
    """``f8_gemm`` for rows sorted by expert: rows offsets[e] .. offsets[e + 1] - 1 (int32
    [E + 1], on the device) times matrix e of wcodes [E, N, Kp]; Y [R, N] or [R, N / 2]."""
    a, R, dev = _gated(act), _dims(xcodes, "xcodes", 2)[0], _device(xcodes, "xcodes")
    E = _dims(offsets, "offsets", 1)[0] - 1
    Kp, Ks, shape = (K + 127) // 128 * 128, (K + 511) // 512 * 4, (R, N >> a)
    if Y is None:
        Y = _empty(shape, _BF16, xcodes.device, stream)
    yt = _float(Y, "Y")
    status = (_lib or lib()).f8_gemm_experts(
        _at(wcodes, _U8, (E, N, Kp), "wcodes", dev), _at(wscales, _U8, (E, (N + 127) // 128, Ks), "wscales", dev), E, N, K,
        _at(offsets, _I32, (E + 1,), "offsets", dev), _at(xcodes, _U8, (R, Kp), "xcodes", dev),
        _at(xscales, _U8, (R, Ks), "xscales", dev), R, a, _at(Y, Y.dtype, shape, "Y", dev), yt, _raw_stream(dev) if stream is None else _stream(stream))
    if status:
        _check("f8_gemm_experts", status)
    return Y


def f8_gemm_plan(N, K, R, experts=0, act="none", dtype=torch.bfloat16):
    """How ``f8_gemm`` (or ``f8_gemm_experts`` with this many experts) cuts a call of R rows: (tokens of
    a tile at most, CTAs that share its weight rows, CTAs that share it along K)."""
    plan = (ctypes.c_int32 * 3)()
    _check("f8_gemm_plan", lib().f8_gemm_plan(experts, N, K, R, _gated(act), {_F32: 0, _BF16: 1}[dtype], plan))
    return tuple(plan)


def moe_route_workspace_bytes(T, E) -> int:
    return int(lib().moe_route_workspace_bytes(T, E))


def moe_route(logits, k, normalize=True, workspace=None, stream=None):
    """Softmax top-k of logits [T, E] float32: (ids int32 [T, k], weights float32 [T, k],
    offsets int32 [E + 1], rows int32 [T k], pos int32 [T, k]).  ``rows`` holds the token of
    every row in expert order (for ``f8_quantize``), ``pos`` the row of every choice (for
    ``moe_combine``).  ``normalize``: the weights sum to 1 over the k chosen, else over E."""
    T, E = shape = _dims(logits, "logits", 2)
    dev = _device(logits, "logits")
    lp = _at(logits, _F32, shape, "logits", dev)
    if stream is not None:
        with _on(stream, logits.device):
            return moe_route(logits, k, normalize, workspace)
    device, empty, l = logits.device, torch.empty, _lib or lib()
    wp, wn = None, 0
    if workspace is not None:
        wp, wn = _at(workspace, _U8, _dims(workspace, "workspace", 1), "workspace", dev), workspace.numel()
    elif T > MOE_ONE_LAUNCH:
        wn = l.moe_route_workspace_bytes(T, E)
        workspace = empty((wn,), dtype=_U8, device=device)
        wp = workspace.data_ptr()
    ids, weights = empty((T, k), dtype=_I32, device=device), empty((T, k), dtype=_F32, device=device)
    rows, offsets = empty((T * k,), dtype=_I32, device=device), empty((E + 1,), dtype=_I32, device=device)
    pos = empty((T, k), dtype=_I32, device=device)
    status = l.moe_route(lp, T, E, k, 1 if normalize else 0, ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(),
                         rows.data_ptr(), pos.data_ptr(), wp, wn, _raw_stream(dev))
    if status:
        _check("moe_route", status)
    return ids, weights, offsets, rows, pos


def moe_combine(Y, pos, weights, out=None, stream=None):
    """out [T, N] = sum over j of weights[:, j] * Y[pos[:, j]], Y [R, N] float32 or bfloat16,
    pos int32 [T, k], weights float32 [T, k] (out has Y's type unless it is passed)."""
    yt = _float(Y, "Y")
    R, N = ys = _dims(Y, "Y", 2)
    T, k = ps = _dims(pos, "pos", 2)
    dev = _device(Y, "Y")
    if out is None:
        out = _empty((T, N), Y.dtype, Y.device, stream)
    ot = _float(out, "out")
    status = (_lib or lib()).moe_combine(
        _at(Y, Y.dtype, ys, "Y", dev), yt, R, N, _at(pos, _I32, ps, "pos", dev), _at(weights, _F32, ps, "weights", dev), T, k,
        _at(out, out.dtype, (T, N), "out", dev), ot, _raw_stream(dev) if stream is None else _stream(stream))
    if status:
        _check("moe_combine", status)
    return out
