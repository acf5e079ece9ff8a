"""ctypes binding of the SALR C ABI (include/salr.h).  Argument marshalling only: every
step of the layer runs in the CUDA library; there is no fallback path.

Tensors are torch tensors (device memory and streams come from torch); bf16 tensors are
passed as raw pointers to their 16-bit patterns.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
# The built library; SALR_LIBRARY names another build of it (the bounds-checked debug
# build, libsalr_checks.so) to load instead.
LIB_PATH = os.environ.get("SALR_LIBRARY") or os.path.join(HERE, "libsalr.so")

SALR_OK = 0
SALR_ERR_INVALID = 1
SALR_ERR_UNSUPPORTED = 2
SALR_ERR_CUDA = 3
SALR_ERR_OOM = 4
SALR_ERR_TIMEOUT = 5

# name -> (restype, argtypes) for every entry point declared in include/salr.h
_P, _I64, _F, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int


class SalrPlan(ctypes.Structure):
    """salr_plan of include/salr.h (field order and types as declared there)."""
    _fields_ = [("path", ctypes.c_int32), ("kernels", ctypes.c_int32),
                ("token_tile", ctypes.c_int32), ("tile_rows", ctypes.c_int32),
                ("grid", ctypes.c_int32),
                ("units", ctypes.c_int32), ("tiles", ctypes.c_int32),
                ("whole_tiles", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("split_sum_bytes", ctypes.c_int64), ("dense_scratch_bytes", ctypes.c_int64),
                ("group_rows", ctypes.c_int32)]


class AdamwTensor(ctypes.Structure):
    """salr_adamw_tensor of include/salr.h."""
    _fields_ = [("param", _P), ("grad", _P), ("master", _P), ("exp_avg", _P), ("exp_avg_sq", _P),
                ("exp_avg_scale", _P), ("exp_avg_sq_scale", _P), ("n", _I64)]


class AdamwConfig(ctypes.Structure):
    """salr_adamw_config of include/salr.h."""
    _fields_ = ([(f, ctypes.c_double) for f in ("lr", "beta1", "beta2", "eps", "weight_decay")] +
                [(f, _P) for f in ("lr_dev", "grad_scale", "step")] +
                [(f, ctypes.c_int32) for f in ("param_type", "grad_type", "state_bits", "master")])


SIGNATURES = {
    "salr_encode": (_I, [_P, _I64, _I64, _F, _P, ctypes.POINTER(_P)]),
    "salr_decode": (_I, [_P, _P, _P]),
    "salr_linear": (_I, [_P, _I64, _P, _P, _P, _I64, _P, _P]),
    "salr_linear_host": (_I, [_P, _I64, _P, _P, _P, _I64, _P, _P]),
    "salr_linear_noalloc": (_I, [_P, _I64, _P, _P, _P, _I64, _P, _P]),
    "salr_free": (_I, [_P]),
    "salr_info": (_I, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I64),
                       ctypes.POINTER(_I64)]),
    "salr_format_view": (_I, [_P, ctypes.POINTER(_P), ctypes.POINTER(_I64), ctypes.POINTER(_P),
                              ctypes.POINTER(_I64)]),
    "salr_save_size": (_I, [_P, ctypes.POINTER(_I64)]),
    "salr_save": (_I, [_P, _P, _I64, _P]),
    "salr_load": (_I, [_P, _I64, _P, ctypes.POINTER(_P)]),
    "salr_residual_adapter": (_I, [_P, _P, _I64, _P, _I64, _I, _P, _P, _P, _P]),
    "salr_linear_plan": (_I, [_I64, _I64, _I64, _I64, ctypes.c_int32, ctypes.POINTER(SalrPlan)]),
    "salr_q4_pack": (_I, [_P, _P, _P, _I64, _I64, _I64, _P, ctypes.POINTER(_P)]),
    "salr_q4_encode": (_I, [_P, _I64, _I64, _I64, _I, _P, ctypes.POINTER(_P)]),
    "salr_linear_backward": (_I, [_P, _P, _I64, _P, _P, _P, _I64, _P, _P, _P, _P]),
    "salr_adamw": (_I, [ctypes.POINTER(AdamwTensor), _I64, ctypes.POINTER(AdamwConfig), _P]),
    "salr_sync_status": (_I, [_P, _P]),
    "salr_status_string": (ctypes.c_char_p, [_I]),
}

_lib = None


class SalrError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {status_string(code)} ({code})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library; raises if it has not been built (no silent fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"SALR CUDA library not built: {path} is missing "
                           "(run python -m sparse_rank_linear_b200.build)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().salr_status_string(int(code)).decode()


def _check(fn: str, code: int):
    if code != SALR_OK:
        raise SalrError(fn, code)


def _stream_ptr(stream=None):
    """The stream's handle; by default the current stream of the current device (looked up
    without building a Stream object, which takes longer than queueing a kernel)."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _on_device(t):
    """Context in which the device of CUDA tensor ``t`` is the current one."""
    import torch
    if t.get_device() == torch._C._cuda_getDevice():
        return _HERE
    return torch.cuda.device(t.device)


_HERE = contextlib.nullcontext()


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _require(t, name, shape=None, device=True, beside=None):
    """Checks of a bf16 tensor; ``beside``: a CUDA tensor on whose device it has to be."""
    import torch
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if beside is not None and t.get_device() != beside.get_device():
        raise ValueError(f"{name} must be on {beside.device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _written(tensors):
    """Tell autograd that the library wrote into tensors of the caller's: a graph that saved one
    of them then refuses its backward pass, as after torch's own in-place operations."""
    import torch
    torch.autograd.graph.increment_version(tensors)


def _ranks(A_cat, B_cat):
    """The adapters' rank, 0 without."""
    if (A_cat is None) != (B_cat is None):
        raise ValueError("A_cat and B_cat must be given together")
    return 0 if A_cat is None else A_cat.shape[1]


class Weight:
    """An encoded weight (pruned and bitmap-stored, or 4-bit codes with group scales): owns
    a ``salr_handle``."""

    def __init__(self, handle: ctypes.c_void_p):
        self._h = handle
        self._nk = None

    def _shape(self):
        """(N, K), which never change, looked up once."""
        if self._nk is None:
            inf = self.info()
            self._nk = (inf["N"], inf["K"])
        return self._nk

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("weight has been freed")
        return self._h

    def info(self):
        n, k, nnz, nbytes = _I64(), _I64(), _I64(), _I64()
        _check("salr_info", load_library().salr_info(self.handle, ctypes.byref(n), ctypes.byref(k),
                                                     ctypes.byref(nnz), ctypes.byref(nbytes)))
        return {"N": n.value, "K": k.value, "nnz": nnz.value, "bytes": nbytes.value}

    def format_view(self):
        """(blob_ptr, blob_bytes, offsets_ptr, n_offsets): device pointers, read only."""
        b, bb, o, no = _P(), _I64(), _P(), _I64()
        _check("salr_format_view", load_library().salr_format_view(
            self.handle, ctypes.byref(b), ctypes.byref(bb), ctypes.byref(o), ctypes.byref(no)))
        return b.value, bb.value, o.value, no.value

    def format_tensors(self):
        """Copies of the encoded blob (uint8) and offset table (int32 holding the uint32
        entries), made by torch from views of the handle's device memory."""
        b, bb, o, no = self.format_view()
        return (_device_view(b, bb, "|u1").clone(), _device_view(o, no, "<i4").clone())

    def decode(self, out=None, stream=None):
        import torch
        inf = self.info()
        given = out is not None
        if not given:
            out = torch.empty(inf["N"], inf["K"], dtype=torch.bfloat16, device="cuda")
        _require(out, "W_out", (inf["N"], inf["K"]))
        _check("salr_decode", load_library().salr_decode(self.handle, _ptr(out), _stream_ptr(stream)))
        if given:
            _written((out,))
        return out

    def to_bytes(self, stream=None) -> bytes:
        """salr_save: the serialised image of this weight (layout in include/salr.h)."""
        lib = load_library()
        n = _I64()
        _check("salr_save_size", lib.salr_save_size(self.handle, ctypes.byref(n)))
        buf = ctypes.create_string_buffer(n.value)
        _check("salr_save", lib.salr_save(self.handle, ctypes.cast(buf, _P), n.value,
                                          _stream_ptr(stream)))
        return buf.raw

    def sync_status(self, stream=None) -> int:
        return load_library().salr_sync_status(self.handle, _stream_ptr(stream))

    def free(self):
        if self._h is not None:
            _check("salr_free", load_library().salr_free(self._h))
            self._h = None

    def __del__(self):
        try:
            if self._h is not None and _lib is not None:
                _lib.salr_free(self._h)
                self._h = None
        except Exception:
            pass


class _DevArray:
    """Minimal __cuda_array_interface__ exporter of a device range (only ever cloned)."""

    def __init__(self, ptr: int, n: int, typestr: str):
        self.__cuda_array_interface__ = {"shape": (n,), "typestr": typestr,
                                         "data": (ptr, False), "version": 2, "strides": None}


def _device_view(ptr: int, n: int, typestr: str):
    import torch
    return torch.as_tensor(_DevArray(ptr, n, typestr), device="cuda")


def encode(W, sparsity: float = 0.5, stream=None) -> Weight:
    """salr_encode: prune ``W`` (N x K bf16, CUDA) per row and bitmap-encode it."""
    _require(W, "W")
    N, K = W.shape
    h = _P()
    _check("salr_encode", load_library().salr_encode(_ptr(W), N, K, float(sparsity),
                                                     _stream_ptr(stream), ctypes.byref(h)))
    return Weight(h)


def pack_q4(codes, scales, zeros=None, stream=None) -> Weight:
    """salr_q4_pack: a weight from 4-bit codes (N x K/2 uint8, even column in the low
    nibble), bf16 scales and optional uint8 zero points (both N x K/group); CUDA tensors."""
    import torch
    for t, name, kind in ((codes, "codes", torch.uint8), (scales, "scales", torch.bfloat16),
                          (zeros, "zeros", torch.uint8)):
        if t is None and name == "zeros":
            continue
        if t.dtype != kind:
            raise TypeError(f"{name} must be {str(kind)[6:]}")
        if t.dim() != 2 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous 2-D CUDA tensor")
        if t.device != codes.device or t.shape[0] != codes.shape[0]:
            raise ValueError(f"{name} must have codes' rows and device")
    N, K = codes.shape[0], 2 * codes.shape[1]
    if zeros is not None and zeros.shape != scales.shape:
        raise ValueError("zeros must have the shape of scales")
    if not scales.shape[1] or K % scales.shape[1]:
        raise ValueError("scales must have one column per group of equal size")
    h = _P()
    with _on_device(codes):
        _check("salr_q4_pack", load_library().salr_q4_pack(
            _ptr(codes), _ptr(scales), _ptr(zeros), N, K, K // scales.shape[1],
            _stream_ptr(stream), ctypes.byref(h)))
    return Weight(h)


def encode_q4(W, group: int = 64, symmetric: bool = True, stream=None) -> Weight:
    """salr_q4_encode: round ``W`` (N x K bf16, CUDA) to 4-bit codes with a bf16 scale, and a
    zero point unless ``symmetric``, per ``group`` columns of a row."""
    _require(W, "W")
    N, K = W.shape
    h = _P()
    with _on_device(W):
        _check("salr_q4_encode", load_library().salr_q4_encode(
            _ptr(W), N, K, int(group), 1 if symmetric else 0, _stream_ptr(stream),
            ctypes.byref(h)))
    return Weight(h)


def load(image: bytes, stream=None) -> Weight:
    """salr_load: a weight on the current CUDA device from a serialised image."""
    data = bytes(image)
    h = _P()
    _check("salr_load", load_library().salr_load(ctypes.cast(ctypes.c_char_p(data), _P),
                                                 len(data), _stream_ptr(stream),
                                                 ctypes.byref(h)))
    return Weight(h)


def residual_adapter(W, weight: Weight, r: int, q: int = 2, oversample: int = 16, omega=None,
                     seed: int = 0, stream=None):
    """salr_residual_adapter: the rank-r adapter (A' K x r, B' r x N, bf16) of W minus its
    pruned form, and the estimated singular values (r, fp32).  ``omega`` (K x l fp32,
    CUDA) is the random test matrix; by default a seeded standard normal one with
    l = r + oversample columns (capped at 160 and at min(N, K))."""
    import torch
    inf = weight.info()
    N, K = inf["N"], inf["K"]
    _require(W, "W", (N, K))
    if omega is None:
        l = min(r + oversample, 160, N, K)
        g = torch.Generator(device=W.device)
        g.manual_seed(seed)
        omega = torch.randn(K, l, generator=g, device=W.device, dtype=torch.float32)
    if omega.dtype != torch.float32 or not omega.is_contiguous() or omega.shape[0] != K:
        raise ValueError("omega must be a contiguous K x l float32 tensor")
    A = torch.empty(K, r, dtype=torch.bfloat16, device=W.device)
    B = torch.empty(r, N, dtype=torch.bfloat16, device=W.device)
    sigma = torch.empty(r, dtype=torch.float32, device=W.device)
    _check("salr_residual_adapter", load_library().salr_residual_adapter(
        _ptr(W), weight.handle, r, _ptr(omega), omega.shape[1], q, _ptr(A), _ptr(B),
        _ptr(sigma), _stream_ptr(stream)))
    return A, B, sigma


def linear(X, weight: Weight, A_cat=None, B_cat=None, Y=None, stream=None):
    """salr_linear: Y = X (M.W)^T + (X A_cat) B_cat; returns Y (M x N bf16).  Calls on one
    bitmap weight share workspace that it holds, so they must not run at the same time on
    different streams; calls on one 4-bit weight may.  No call of this module is recorded for
    autograd: ``linear_backward`` gives the gradients."""
    N, K = weight._shape()
    _require(X, "X")
    M = X.shape[0]
    if X.shape[1] != K:
        raise ValueError("X has the wrong number of columns")
    R = _ranks(A_cat, B_cat)
    if A_cat is not None:
        _require(A_cat, "A_cat", (K, R), beside=X)
        _require(B_cat, "B_cat", (R, N), beside=X)
    given = Y is not None
    if not given:
        Y = X.new_empty((M, N))
    else:
        _require(Y, "Y", (M, N), beside=X)
    with _on_device(X):
        _check("salr_linear", load_library().salr_linear(
            _ptr(X), M, weight.handle, _ptr(A_cat), _ptr(B_cat), R, _ptr(Y), _stream_ptr(stream)))
    if given:
        _written((Y,))
    return Y


def linear_backward(dY, X, weight: Weight, A_cat=None, B_cat=None, dX=None, dA=None, dB=None,
                    needs=(True, True, True), stream=None):
    """salr_linear_backward: the gradients (dX, dA, dB) of ``linear`` for the gradient ``dY``
    of its result (M x N bf16).  ``needs`` says which are wanted; the others, and dA and dB
    without adapters, come back as None.  ``X`` may be None if only dX is wanted."""
    N, K = weight._shape()
    _require(dY, "dY")
    if dY.dim() != 2 or dY.shape[1] != N:
        raise ValueError("dY has the wrong number of columns")
    M = dY.shape[0]
    R = _ranks(A_cat, B_cat)
    if A_cat is not None:
        _require(A_cat, "A_cat", (K, R), beside=dY)
        _require(B_cat, "B_cat", (R, N), beside=dY)
    want_x, want_a, want_b = bool(needs[0]), bool(needs[1]) and R > 0, bool(needs[2]) and R > 0
    if not (want_x or want_a or want_b):
        raise ValueError("no gradient is wanted")
    if want_a or want_b:
        if X is None:
            raise ValueError("X is needed for dA and dB")
        _require(X, "X", (M, K), beside=dY)
    else:
        X = None
    out, given = [], []
    for want, t, name, shape in ((want_x, dX, "dX", (M, K)), (want_a, dA, "dA", (K, R)),
                                 (want_b, dB, "dB", (R, N))):
        if not want:
            t = None
        elif t is None:
            t = dY.new_empty(shape)
        else:
            _require(t, name, shape, beside=dY)
            given.append(t)
        out.append(t)
    dX, dA, dB = out
    with _on_device(dY):
        _check("salr_linear_backward", load_library().salr_linear_backward(
            _ptr(dY), _ptr(X), M, weight.handle, _ptr(A_cat), _ptr(B_cat), R, _ptr(dX), _ptr(dA),
            _ptr(dB), _stream_ptr(stream)))
    if given:
        _written(given)
    return dX, dA, dB


def linear_host(X_host, weight: Weight, A_cat, B_cat, Y_host, stream=None):
    """salr_linear_host: X_host / Y_host are pinned CPU bf16 tensors; adapters on device."""
    inf = weight.info()
    _require(X_host, "X_host", device=False)
    _require(Y_host, "Y_host", (X_host.shape[0], inf["N"]), device=False)
    R = _ranks(A_cat, B_cat)
    _check("salr_linear_host", load_library().salr_linear_host(
        _ptr(X_host), X_host.shape[0], weight.handle, _ptr(A_cat), _ptr(B_cat), R, _ptr(Y_host),
        _stream_ptr(stream)))
    _written((Y_host,))
    return Y_host


def plan(N: int, K: int, M: int, R: int = 0, sms: int = 0) -> dict:
    """salr_linear_plan: the kernels, tiles, work split and extra device memory that
    salr_linear uses for M tokens on an N x K weight (sms = 0: the current device's)."""
    out = SalrPlan()
    _check("salr_linear_plan", load_library().salr_linear_plan(N, K, M, R, sms, ctypes.byref(out)))
    return {name: getattr(out, name) for name, _ in SalrPlan._fields_}
