"""Thin Python binding over the libgq4 C ABI (``include/gq4.h``).

Argument marshalling only: each function checks that the torch tensors it is
given are CUDA, contiguous and of the right dtype and shape, then passes their
device pointers and the current CUDA stream to the C entry point of the same
name.  Every step of the computation runs in the library's sm_103a kernels.
There is no CPU fallback: importing this module raises if ``libgq4.so`` has
not been built (``python -m int4_group_quantized_quant_gb300.build``).
"""

from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgq4.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first "
        "(python -m int4_group_quantized_quant_gb300.build)")

lib = ctypes.CDLL(LIB_PATH)

MAX_LANES = 32

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_ALIAS = 3
ERR_CUDA = 4
ERR_MISALIGNED = 5

_vp = ctypes.c_void_p
_i = ctypes.c_int


class Norm(ctypes.Structure):
    """``gq4_norm``: the optional residual + RMSNorm prologue."""
    _fields_ = [("A_b", _vp), ("W_norm", _vp), ("eps", ctypes.c_float),
                ("residual_out", _vp), ("norm_out", _vp)]


_NormP = ctypes.POINTER(Norm)

OP_MATVEC, OP_QUAD, OP_NORM, OP_GATED = 0, 1, 2, 3


class Call(ctypes.Structure):
    """``gq4_call``: one one-lane call of a sequence (``gq4_run_sequence``)."""
    _fields_ = [("op", _i), ("K", _i), ("N", _i), ("group_size", _i),
                ("n0", _i), ("n1", _i), ("n2", _i),
                ("A", _vp), ("Bq", _vp * 2), ("scales", _vp * 2), ("zeros", _vp * 2),
                ("out", _vp * 4), ("has_norm", _i), ("norm", Norm)]


class Rope(ctypes.Structure):
    """``gq4_rope``: the per-head norm and the rotation."""
    _fields_ = [("q_gain", _vp), ("k_gain", _vp), ("eps", ctypes.c_float), ("rot_dim", _i),
                ("interleaved", _i), ("inv_freq", _vp)]


class KVCache(ctypes.Structure):
    """``gq4_kv_cache``: the paged 4-bit key/value cache."""
    _fields_ = [("n_pages", _i), ("page_size", _i), ("kv_heads", _i), ("head_dim", _i),
                ("group_size", _i), ("Kq", _vp), ("K_sz", _vp), ("Vq", _vp), ("V_sz", _vp)]


_RopeP = ctypes.POINTER(Rope)
_CacheP = ctypes.POINTER(KVCache)

_SIGS = {
    "gq4_matvec": [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp],
    "gq4_quad_matvec": [_i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                        _vp, _vp],
    "gq4_norm_matvec": [_i, _i, _i, _i, _NormP, _vp, _vp, _vp, _vp, _vp, _vp],
    "gq4_gated_matvec": [_i, _i, _i, _i, _NormP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                         _vp],
    "gq4_dual_matvec": [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "gq4_sigmoid_gated_matvec": [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "gq4_swiglu_gated_matvec": [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "gq4_run_sequence": [ctypes.POINTER(Call), _i, _vp, _vp],
    "gq4_run_sequence_static": [ctypes.POINTER(Call), _i, _vp],
    "gq4_sequence_launches": [ctypes.POINTER(Call), _i, ctypes.POINTER(_i)],
    "gq4_gemm": [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "gq4_quantize": [_i, _i, _i, _vp, _vp, _vp, _vp, _vp],
    "gq4_from_mlx": [_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "gq4_embedding": [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp],
    "gq4_head_norm_rope": [_i, _i, _i, _i, _RopeP, _vp, _vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp],
    "gq4_kv_append": [_i, _CacheP, _vp, _i, _vp, _i, _vp, _vp],
    "gq4_kv_gather": [_i, _CacheP, _vp, _vp, _vp, _vp],
    "gq4_kv_plan": [_i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "gq4_kv_attention": [_i, _i, _i, _i, _i, _i, _CacheP, _vp, _i, _vp, _vp, _vp, ctypes.c_float, _i,
                         _vp, _i, _vp, ctypes.c_size_t, _vp],
    "gq4_unpack": [_i, _i, _vp, _vp, _vp],
    "gq4_dequant": [_i, _i, _i, _vp, _vp, _vp, _vp, _vp],
}
for _name, _args in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _i
    _fn.argtypes = _args
lib.gq4_status_string.restype = ctypes.c_char_p
lib.gq4_status_string.argtypes = [_i]
lib.gq4_version.restype = _i
lib.gq4_version.argtypes = []
lib.gq4_device_error.restype = _i
lib.gq4_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), _i]
lib.gq4_sequence_workspace_bytes.restype = ctypes.c_size_t
lib.gq4_sequence_workspace_bytes.argtypes = []
lib.gq4_gemm_workspace_bytes.restype = ctypes.c_size_t
lib.gq4_gemm_workspace_bytes.argtypes = [_i, _i]
lib.gq4_kv_attention_workspace_bytes.restype = ctypes.c_size_t
lib.gq4_kv_attention_workspace_bytes.argtypes = [_i, _i, _i, _i]

EXPORTED = list(_SIGS) + ["gq4_status_string", "gq4_version", "gq4_device_error",
                          "gq4_sequence_workspace_bytes", "gq4_gemm_workspace_bytes",
                          "gq4_kv_attention_workspace_bytes"]


class GQ4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.gq4_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


def _check(status: int, where: str):
    if status != OK:
        raise GQ4Error(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtypes, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")


_F32 = (torch.float32,)
_WORDS = (torch.int32,) + ((torch.uint32,) if hasattr(torch, "uint32") else ())


def _weights(Bq, scales, zeros, K, group_size, tag=""):
    N = Bq.shape[0]
    _need(Bq, "Bq" + tag, _WORDS, (N, K // 8))
    _need(scales, "scales" + tag, _F32, (N, K // group_size))
    _need(zeros, "zeros" + tag, _F32, (N, K // group_size))
    return N


def _lanes(A):
    _need(A, "A", _F32)
    if A.dim() != 2:
        raise ValueError("A must be [M, K]")
    return A.shape


def matvec(A, Bq, scales, zeros, group_size, C=None, stream=None):
    """C [M, N] = A [M, K] times the int4 matrix (Bq [N, K/8], scales/zeros [N, K/gs])."""
    M, K = _lanes(A)
    N = _weights(Bq, scales, zeros, K, group_size)
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _need(C, "C", _F32, (M, N))
    _check(lib.gq4_matvec(M, K, N, group_size, _ptr(A), _ptr(Bq), _ptr(scales), _ptr(zeros),
                          _ptr(C), _stream(stream)), "gq4_matvec")
    return C


def gemm_workspace_bytes(M, K) -> int:
    return int(lib.gq4_gemm_workspace_bytes(M, K))


def gemm(A, Bq, scales, zeros, group_size, C=None, workspace=None, stream=None):
    """C [M, N] = A [M, K] times the int4 matrix, any M >= 1 (gq4_gemm; bf16 tensor cores).
    ``workspace`` (a CUDA tensor of at least gemm_workspace_bytes(M, K) bytes) enables the
    GEMM kernel for M > 32; ``workspace=False`` runs the row chunks without one."""
    _need(A, "A", _F32)
    if A.dim() != 2:
        raise ValueError("A must be [M, K]")
    M, K = A.shape
    N = _weights(Bq, scales, zeros, K, group_size)
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _need(C, "C", _F32, (M, N))
    if workspace is None:
        workspace = torch.empty(gemm_workspace_bytes(M, K), dtype=torch.uint8, device=A.device)
    ws_ptr, ws_bytes = None, 0
    if workspace is not False:
        if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda and workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    _check(lib.gq4_gemm(M, K, N, group_size, _ptr(A), _ptr(Bq), _ptr(scales), _ptr(zeros),
                        _ptr(C), ws_ptr, ws_bytes, _stream(stream)), "gq4_gemm")
    return C


def quad_matvec(A, Bq, scales, zeros, group_size, n0, n1, n2, outs=None, stream=None):
    """Quad-output matvec; returns the four segment outputs [M, len_i] (empty ones have 0 columns)."""
    M, K = _lanes(A)
    N = _weights(Bq, scales, zeros, K, group_size)
    lens = [n0, n1 - n0, n2 - n1, N - n2]
    if outs is None:
        outs = [torch.empty((M, max(n, 0)), dtype=torch.float32, device=A.device) for n in lens]
    ptrs = []
    for i, (o, n) in enumerate(zip(outs, lens)):
        if o is None:
            ptrs.append(None)
            continue
        _need(o, f"out{i}", _F32, (M, n) if n >= 0 else None)
        ptrs.append(_ptr(o) if o.numel() else None)
    _check(lib.gq4_quad_matvec(M, K, N, group_size, n0, n1, n2, _ptr(A), _ptr(Bq), _ptr(scales),
                               _ptr(zeros), *ptrs, _stream(stream)), "gq4_quad_matvec")
    return outs


def _norm_struct(M, K, W_norm, eps, A_b, residual_out, norm_out):
    _need(W_norm, "W_norm", _F32, (K,))
    for name, t in (("A_b", A_b), ("residual_out", residual_out), ("norm_out", norm_out)):
        if t is not None:
            _need(t, name, _F32, (M, K))
    return Norm(_ptr(A_b), _ptr(W_norm), float(eps), _ptr(residual_out), _ptr(norm_out))


def norm_matvec(A, Bq, scales, zeros, group_size, W_norm, eps=1e-6, A_b=None,
                residual_out=None, norm_out=None, C=None, stream=None):
    """C = matvec of RMSNorm(A + A_b) * W_norm; optionally writes residual_out / norm_out."""
    M, K = _lanes(A)
    N = _weights(Bq, scales, zeros, K, group_size)
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _need(C, "C", _F32, (M, N))
    nrm = _norm_struct(M, K, W_norm, eps, A_b, residual_out, norm_out)
    _check(lib.gq4_norm_matvec(M, K, N, group_size, ctypes.byref(nrm), _ptr(A), _ptr(Bq),
                               _ptr(scales), _ptr(zeros), _ptr(C), _stream(stream)),
           "gq4_norm_matvec")
    return C


def gated_matvec(A, Bq_gate, scales_gate, zeros_gate, Bq_up, scales_up, zeros_up, group_size,
                 W_norm=None, eps=1e-6, A_b=None, residual_out=None, norm_out=None, out=None,
                 stream=None):
    """out = silu(a . Wg) * (a . Wu), a = A or RMSNorm(A + A_b) * W_norm when W_norm is given."""
    M, K = _lanes(A)
    N = _weights(Bq_gate, scales_gate, zeros_gate, K, group_size, "_gate")
    if _weights(Bq_up, scales_up, zeros_up, K, group_size, "_up") != N:
        raise ValueError("gate and up must have the same N")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _need(out, "out", _F32, (M, N))
    nrm = None
    if W_norm is not None:
        nrm = _norm_struct(M, K, W_norm, eps, A_b, residual_out, norm_out)
    elif A_b is not None or residual_out is not None or norm_out is not None:
        raise ValueError("A_b / residual_out / norm_out need W_norm")
    _check(lib.gq4_gated_matvec(M, K, N, group_size, ctypes.byref(nrm) if nrm else None,
                                _ptr(A), _ptr(Bq_gate), _ptr(scales_gate), _ptr(zeros_gate),
                                _ptr(Bq_up), _ptr(scales_up), _ptr(zeros_up), _ptr(out),
                                _stream(stream)), "gq4_gated_matvec")
    return out


def dual_matvec(A, Bq0, scales0, zeros0, Bq1, scales1, zeros1, group_size, C0=None, C1=None,
                stream=None):
    """(C0, C1) = (A . W0, A . W1): two projections sharing the input (gq4_dual_matvec)."""
    M, K = _lanes(A)
    N = _weights(Bq0, scales0, zeros0, K, group_size, "0")
    if _weights(Bq1, scales1, zeros1, K, group_size, "1") != N:
        raise ValueError("both matrices must have the same N")
    if C0 is None:
        C0 = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if C1 is None:
        C1 = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _need(C0, "C0", _F32, (M, N))
    _need(C1, "C1", _F32, (M, N))
    _check(lib.gq4_dual_matvec(M, K, N, group_size, _ptr(A), _ptr(Bq0), _ptr(scales0),
                               _ptr(zeros0), _ptr(Bq1), _ptr(scales1), _ptr(zeros1), _ptr(C0),
                               _ptr(C1), _stream(stream)), "gq4_dual_matvec")
    return C0, C1


def _gated_input(fn, name, X, G, Bq, scales, zeros, group_size, C, stream):
    M, K = _lanes(X)
    _need(G, "G", _F32, (M, K))
    N = _weights(Bq, scales, zeros, K, group_size)
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=X.device)
    _need(C, "C", _F32, (M, N))
    _check(fn(M, K, N, group_size, _ptr(X), _ptr(G), _ptr(Bq), _ptr(scales), _ptr(zeros), _ptr(C),
              _stream(stream)), name)
    return C


def sigmoid_gated_matvec(X, G, Bq, scales, zeros, group_size, C=None, stream=None):
    """C = (X * sigmoid(G)) . W (gq4_sigmoid_gated_matvec)."""
    return _gated_input(lib.gq4_sigmoid_gated_matvec, "gq4_sigmoid_gated_matvec", X, G, Bq, scales,
                        zeros, group_size, C, stream)


def swiglu_gated_matvec(X, G, Bq, scales, zeros, group_size, C=None, stream=None):
    """C = (silu(G) * X) . W (gq4_swiglu_gated_matvec)."""
    return _gated_input(lib.gq4_swiglu_gated_matvec, "gq4_swiglu_gated_matvec", X, G, Bq, scales,
                        zeros, group_size, C, stream)


# ---------------------------------------------------------------------------
# Producing the format
# ---------------------------------------------------------------------------

def _format_outputs(N, K, group_size, device, Bq, scales, zeros):
    G = K // group_size
    if Bq is None:
        Bq = torch.empty((N, K // 8), dtype=torch.int32, device=device)
    if scales is None:
        scales = torch.empty((N, G), dtype=torch.float32, device=device)
    if zeros is None:
        zeros = torch.empty((N, G), dtype=torch.float32, device=device)
    _need(Bq, "Bq", _WORDS, (N, K // 8))
    _need(scales, "scales", _F32, (N, G))
    _need(zeros, "zeros", _F32, (N, G))
    return Bq, scales, zeros


def quantize(W, group_size, Bq=None, scales=None, zeros=None, stream=None):
    """(Bq, scales, zeros) of W f32 [N, K] (gq4_quantize: min/max asymmetric per group)."""
    _need(W, "W", _F32)
    if W.dim() != 2:
        raise ValueError("W must be [N, K]")
    N, K = W.shape
    if K % 8 != 0 or group_size <= 0:
        raise ValueError("K must be a multiple of 8 and group_size positive")
    Bq, scales, zeros = _format_outputs(N, K, group_size, W.device, Bq, scales, zeros)
    _check(lib.gq4_quantize(K, N, group_size, _ptr(W), _ptr(Bq), _ptr(scales), _ptr(zeros),
                            _stream(stream)), "gq4_quantize")
    return Bq, scales, zeros


def from_mlx(packed, mlx_scales, mlx_biases, group_size, Bq=None, scales=None, zeros=None,
             stream=None):
    """(Bq, scales, zeros) of an MLX affine int4 matrix (gq4_from_mlx); pass Bq=packed to
    convert the words in place."""
    _need(packed, "packed", _WORDS)
    if packed.dim() != 2:
        raise ValueError("packed must be [N, K/8]")
    N, K = packed.shape[0], packed.shape[1] * 8
    if group_size <= 0 or K % group_size != 0:
        raise ValueError("K must be a multiple of group_size")
    G = K // group_size
    _need(mlx_scales, "mlx_scales", _F32, (N, G))
    _need(mlx_biases, "mlx_biases", _F32, (N, G))
    Bq, scales, zeros = _format_outputs(N, K, group_size, packed.device, Bq, scales, zeros)
    _check(lib.gq4_from_mlx(K, N, group_size, _ptr(packed), _ptr(mlx_scales), _ptr(mlx_biases),
                            _ptr(Bq), _ptr(scales), _ptr(zeros), _stream(stream)),
           "gq4_from_mlx")
    return Bq, scales, zeros


def embedding(ids, Bq, scales, zeros, group_size, out=None, stream=None):
    """out [T, K] = the int4 table's rows ids dequantized (gq4_embedding)."""
    _need(ids, "ids", (torch.int32,))
    if ids.dim() != 1:
        raise ValueError("ids must be [T]")
    V, K = Bq.shape[0], Bq.shape[1] * 8
    _weights(Bq, scales, zeros, K, group_size)
    T = ids.shape[0]
    if out is None:
        out = torch.empty((T, K), dtype=torch.float32, device=Bq.device)
    _need(out, "out", _F32, (T, K))
    _check(lib.gq4_embedding(T, K, V, group_size, _ptr(ids), _ptr(Bq), _ptr(scales),
                             _ptr(zeros), _ptr(out), _stream(stream)), "gq4_embedding")
    return out


# ---------------------------------------------------------------------------
# Between the QKV product and the output projection
# ---------------------------------------------------------------------------

_f32, _i32 = torch.float32, torch.int32
# the current device, and its current stream's handle without a Stream object around it, where torch has them
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, name, index, stream, *args):
    """fn(*args, stream) on device `index`, on the given stream or that device's current one."""
    if index != _current_device():
        with torch.cuda.device(index):
            return _call(fn, name, index, stream, *args)
    status = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if status != OK:
        raise GQ4Error(status, name)


def _lend(stream, index, *made):
    """Tensors that a call allocated (on the current stream) for use on another: that stream first waits for
    what their memory was last used for here, and they are not handed out again while it uses them."""
    if stream is None or not made or stream.cuda_stream == _raw_stream(index):
        return
    here = torch.cuda.current_stream(index)
    capturing = torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        capturing = capturing or torch.cuda.is_current_stream_capturing()
    if not capturing:       # (a captured graph's memory is its own)
        stream.wait_stream(here)
    for t in made:
        t.record_stream(stream)


def _at(t, name, dtype, shape, index):
    """t's address; _need's checks (its errors) and the device's, the common case in one expression."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        _need(t, name, (dtype,), shape)
        raise ValueError(f"{name} is on {t.device}, the others on cuda:{index}")
    return t.data_ptr()


def _device(t, name):
    """The CUDA device that a call's first tensor names."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    return index


def _width(t):
    """Columns of a matrix (-1: not one, which no shape matches)."""
    return t.shape[1] if isinstance(t, torch.Tensor) and t.dim() == 2 else -1


def _rows(t, name, index=None, heads_dim=None):
    """[T, heads, D] with dense rows (any row distance): (T, heads, D, row distance)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype is not _f32:
        raise TypeError(f"{name}: dtype {t.dtype} is not torch.float32")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, head_dim]")
    T, H, D = t.shape
    if heads_dim is not None and (T, H, D) != heads_dim:
        raise ValueError(f"{name}: shape {(T, H, D)} != {heads_dim}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the others on cuda:{index}")
    ld, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}: the heads of a row must be dense")
    return T, H, D, (H * D if T <= 1 else ld)


def _rope_side(x, y, gain, name, T, D, index):
    """One side's heads, tensors and row distances; its output is made where none is given."""
    if x is None:
        if y is not None or gain is not None:
            raise ValueError(f"{name}_out and {name}_gain need {name}")
        return None, None, (0, None, 0, None, 0)
    Tx, H, Dx, ld = _rows(x, name, index)
    if (Tx, Dx) != (T, D):
        raise ValueError(f"{name}: {Tx} rows of {Dx} != {T} rows of {D}")
    if y is None:
        y, ldy = torch.empty((T, H, D), dtype=_f32, device=x.device), H * D
    else:
        ldy = _rows(y, name + "_out", index, (T, H, D))[3]
    at_gain = None if gain is None else _at(gain, name + "_gain", _f32, (D,), index)
    return y, at_gain, (H, x.data_ptr(), ld, y.data_ptr(), ldy)


def head_norm_rope(q, k, positions, inv_freq, q_gain=None, k_gain=None, eps=1e-6, interleaved=False,
                   q_out=None, k_out=None, stream=None):
    """(q, k) with every head normalised (where a gain is given) and rotated by position
    (gq4_head_norm_rope).  q [T, heads, D] and k [T, kv_heads, D], either may be None; rows may be
    columns of a wider matrix.  inv_freq f32 [rot_dim / 2], or None for no rotation.  q_out / k_out
    may be q / k themselves."""
    first = k if q is None else q
    if first is None:
        raise ValueError("q or k must be given")
    T, _, D, _ = _rows(first, "k" if q is None else "q")
    index = first.get_device()
    given = q_out, k_out
    q_out, q_gain_at, (QH, xq, ldq, yq, ldqo) = _rope_side(q, q_out, q_gain, "q", T, D, index)
    k_out, k_gain_at, (KH, xk, ldk, yk, ldko) = _rope_side(k, k_out, k_gain, "k", T, D, index)
    rot, at_pos, at_inv = 0, None, None
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        at_inv = _at(inv_freq, "inv_freq", _f32, (rot // 2,), index)
        at_pos = _at(positions, "positions", _i32, (T,), index)
    if stream is not None:
        _lend(stream, index, *[y for y, was in zip((q_out, k_out), given) if was is None and y is not None])
    _call(lib.gq4_head_norm_rope, "gq4_head_norm_rope", index, stream, T, QH, KH, D,
          Rope(q_gain_at, k_gain_at, eps, rot, 1 if interleaved else 0, at_inv), at_pos, xq, ldq, xk, ldk,
          yq, ldqo, yk, ldko)
    return q_out, k_out


def kv_cache(n_pages, kv_heads, page_size, head_dim, group_size, device=None):
    """An empty cache: (Kq, K_sz, Vq, V_sz), the tensors the kv_* calls take (codes int32
    [n_pages, kv_heads, page_size, head_dim/8], scale and zero f32 [..., head_dim/group_size, 2])."""
    if group_size <= 0 or head_dim % group_size != 0 or head_dim % 8 != 0:
        raise ValueError("head_dim must be a multiple of 8 and of group_size")
    w, s = (n_pages, kv_heads, page_size, head_dim // 8), (n_pages, kv_heads, page_size, head_dim // group_size, 2)
    device = "cuda" if device is None else device
    return tuple(torch.zeros(x, dtype=d, device=device)
                 for x, d in ((w, torch.int32), (s, torch.float32), (w, torch.int32), (s, torch.float32)))


def _cache(Kq, K_sz, Vq, V_sz, group_size):
    """The cache's descriptor and device."""
    index, dtype = _device(Kq, "Kq"), Kq.dtype
    if Kq.dim() != 4:
        raise ValueError("Kq must be [n_pages, kv_heads, page_size, head_dim/8]")
    if dtype is not _i32:
        _need(Kq, "Kq", _WORDS)
    shape = P, H, S, W = Kq.shape
    if group_size <= 0 or (8 * W) % group_size != 0:
        raise ValueError("head_dim must be a multiple of group_size")
    sz = (P, H, S, 8 * W // group_size, 2)
    return KVCache(P, S, H, 8 * W, group_size, _at(Kq, "Kq", dtype, shape, index), _at(K_sz, "K_sz", _f32, sz, index),
                   _at(Vq, "Vq", dtype, shape, index), _at(V_sz, "V_sz", _f32, sz, index)), index


def kv_append(k, v, slots, Kq, K_sz, Vq, V_sz, group_size, stream=None):
    """Quantise rows k, v [T, kv_heads, D] into the cache at slots int32 [T] (gq4_kv_append;
    negative slots are skipped)."""
    c, index = _cache(Kq, K_sz, Vq, V_sz, group_size)
    T, H, D, ldk = _rows(k, "k", index)
    if (H, D) != (c.kv_heads, c.head_dim):
        raise ValueError(f"k: {H} heads of {D} != {c.kv_heads} heads of {c.head_dim}")
    ldv = _rows(v, "v", index, (T, H, D))[3]
    at_slots = _at(slots, "slots", _i32, (T,), index)
    _call(lib.gq4_kv_append, "gq4_kv_append", index, stream, T, c, k.data_ptr(), ldk, v.data_ptr(), ldv, at_slots)


def kv_gather(slots, Kq, K_sz, Vq, V_sz, group_size, k_out=None, v_out=None, stream=None):
    """(k, v) f32 [T, kv_heads, D] of the cache rows at slots (gq4_kv_gather; rows of negative slots
    are left as they were, so pass k_out and v_out where there are some)."""
    c, index = _cache(Kq, K_sz, Vq, V_sz, group_size)
    _device(slots, "slots")
    T = slots.numel()
    at_slots, shape = _at(slots, "slots", _i32, (T,), index), (T, c.kv_heads, c.head_dim)
    given = k_out, v_out
    if k_out is None:
        k_out = torch.empty(shape, dtype=_f32, device=Kq.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=_f32, device=Kq.device)
    if stream is not None:
        _lend(stream, index, *[y for y, was in zip((k_out, v_out), given) if was is None])
    _call(lib.gq4_kv_gather, "gq4_kv_gather", index, stream, T, c, at_slots,
          _at(k_out, "k_out", _f32, shape, index), _at(v_out, "v_out", _f32, shape, index))
    return k_out, v_out


def kv_plan(past_lens, new_lens, page_table, free_pages, free_count, n_tokens, page_size, seq_lens=None,
            query_start=None, positions=None, slots=None, free_count_out=None, stream=None):
    """A step's pages, positions and slots from the requests' lengths (gq4_kv_plan); page_table int32
    [B, max_pages] is extended in place.  Returns (seq_lens, query_start, positions, slots,
    free_count_out); pass seq_lens=past_lens and free_count_out=free_count to advance them in place."""
    index, B = _device(past_lens, "past_lens"), past_lens.numel()
    if n_tokens < 0:
        raise ValueError("n_tokens must not be negative")
    width, n_free = _width(page_table), free_pages.numel()
    at_past, at_new = _at(past_lens, "past_lens", _i32, (B,), index), _at(new_lens, "new_lens", _i32, (B,), index)
    at_table = _at(page_table, "page_table", _i32, (B, width), index)
    at_free, at_count = _at(free_pages, "free_pages", _i32, (n_free,), index), \
        _at(free_count, "free_count", _i32, (1,), index)
    sizes = (B, B + 1, n_tokens, n_tokens, 1)
    outs = [seq_lens, query_start, positions, slots, free_count_out]
    ptrs = [None if t is None else _at(t, name, _i32, (n,), index) for t, name, n in
            zip(outs, ("seq_lens", "query_start", "positions", "slots", "free_count_out"), sizes)]
    # what is not given is a stretch of one allocation
    missing = [i for i in range(5) if outs[i] is None]
    if missing:
        lens = [sizes[i] for i in missing]
        spare = torch.empty(sum(lens), dtype=_i32, device=past_lens.device)
        at = spare.data_ptr()
        for i, part in zip(missing, spare.split_with_sizes(lens)):
            outs[i], ptrs[i] = part, at
            at += 4 * sizes[i]
        if stream is not None:
            _lend(stream, index, spare)
    lens, starts, pos, slt, left = ptrs
    _call(lib.gq4_kv_plan, "gq4_kv_plan", index, stream, B, n_tokens, page_size, width, n_free, at_past, at_new,
          at_table, at_free, at_count, left, lens, starts, pos, slt)
    return tuple(outs)


def kv_attention_workspace_bytes(T, heads, kv_heads, head_dim) -> int:
    return lib.gq4_kv_attention_workspace_bytes(T, heads, kv_heads, head_dim)


def kv_attention(q, query_start, seq_lens, page_table, Kq, K_sz, Vq, V_sz, group_size, scale, max_query,
                 max_len=0, window=0, out=None, workspace=None, stream=None):
    """Causal attention of q [T, heads, D] over the cache (gq4_kv_attention): request b's queries are
    rows query_start[b]..query_start[b+1], its seq_lens[b] keys are in the pages of page_table row b.
    ``workspace``: a CUDA tensor of at least kv_attention_workspace_bytes(T, heads, kv_heads, D) bytes
    (allocated when None).  ``out`` rows of no request are left as they were."""
    c, index = _cache(Kq, K_sz, Vq, V_sz, group_size)
    T, H, D, ldq = _rows(q, "q", index)
    if D != c.head_dim:
        raise ValueError(f"q: head_dim {D} != {c.head_dim}")
    _device(seq_lens, "seq_lens")
    B, width = seq_lens.numel(), _width(page_table)
    at_lens, at_start = _at(seq_lens, "seq_lens", _i32, (B,), index), \
        _at(query_start, "query_start", _i32, (B + 1,), index)
    at_table = _at(page_table, "page_table", _i32, (B, width), index)
    made = []
    if out is None:
        out, ldo = torch.empty((T, H, D), dtype=_f32, device=q.device), H * D
        made.append(out)
    else:
        ldo = _rows(out, "out", index, (T, H, D))[3]
    if workspace is None:
        workspace = torch.empty(lib.gq4_kv_attention_workspace_bytes(T, H, c.kv_heads, D), dtype=torch.uint8,
                                device=q.device)
        made.append(workspace)
    elif not (isinstance(workspace, torch.Tensor) and workspace.get_device() == index and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor on the others' device")
    if stream is not None:
        _lend(stream, index, *made)
    _call(lib.gq4_kv_attention, "gq4_kv_attention", index, stream, B, T, H, width, max_query, max_len, c,
          q.data_ptr(), ldq, at_start, at_lens, at_table, scale, window, out.data_ptr(), ldo,
          workspace.data_ptr(), workspace.nbytes)
    return out


# ---------------------------------------------------------------------------
# Call sequences (one lane)
# ---------------------------------------------------------------------------

class SeqCall:
    """One call of a sequence: the C descriptor plus the tensors it points to
    (kept alive while the descriptor is in use)."""

    def __init__(self, desc: Call, tensors):
        self.desc = desc
        self.tensors = tensors


def _one_lane(A):
    M, K = _lanes(A)
    if M != 1:
        raise ValueError("sequence calls take one lane (A of shape [1, K])")
    return K


def _seq_norm(desc, K, W_norm, eps, A_b, residual_out, norm_out):
    desc.has_norm = 1
    desc.norm = _norm_struct(1, K, W_norm, eps, A_b, residual_out, norm_out)


def seq_matvec(A, Bq, scales, zeros, group_size, C):
    """Sequence entry of gq4_matvec (C [1, N] must be given)."""
    K = _one_lane(A)
    N = _weights(Bq, scales, zeros, K, group_size)
    _need(C, "C", _F32, (1, N))
    d = Call(op=OP_MATVEC, K=K, N=N, group_size=group_size, A=_ptr(A))
    d.Bq[0], d.scales[0], d.zeros[0], d.out[0] = _ptr(Bq), _ptr(scales), _ptr(zeros), _ptr(C)
    return SeqCall(d, (A, Bq, scales, zeros, C))


def seq_quad(A, Bq, scales, zeros, group_size, n0, n1, n2, outs):
    """Sequence entry of gq4_quad_matvec (outs: four [1, len] tensors or None for empty ones)."""
    K = _one_lane(A)
    N = _weights(Bq, scales, zeros, K, group_size)
    lens = [n0, n1 - n0, n2 - n1, N - n2]
    d = Call(op=OP_QUAD, K=K, N=N, group_size=group_size, n0=n0, n1=n1, n2=n2, A=_ptr(A))
    d.Bq[0], d.scales[0], d.zeros[0] = _ptr(Bq), _ptr(scales), _ptr(zeros)
    for i, (o, n) in enumerate(zip(outs, lens)):
        if o is not None:
            _need(o, f"out{i}", _F32, (1, n))
        d.out[i] = _ptr(o)
    return SeqCall(d, (A, Bq, scales, zeros, *outs))


def seq_norm(A, Bq, scales, zeros, group_size, W_norm, C, eps=1e-6, A_b=None,
             residual_out=None, norm_out=None):
    """Sequence entry of gq4_norm_matvec."""
    K = _one_lane(A)
    N = _weights(Bq, scales, zeros, K, group_size)
    _need(C, "C", _F32, (1, N))
    d = Call(op=OP_NORM, K=K, N=N, group_size=group_size, A=_ptr(A))
    d.Bq[0], d.scales[0], d.zeros[0], d.out[0] = _ptr(Bq), _ptr(scales), _ptr(zeros), _ptr(C)
    _seq_norm(d, K, W_norm, eps, A_b, residual_out, norm_out)
    return SeqCall(d, (A, Bq, scales, zeros, C, W_norm, A_b, residual_out, norm_out))


def seq_gated(A, Bq_gate, scales_gate, zeros_gate, Bq_up, scales_up, zeros_up, group_size, out,
              W_norm=None, eps=1e-6, A_b=None, residual_out=None, norm_out=None):
    """Sequence entry of gq4_gated_matvec."""
    K = _one_lane(A)
    N = _weights(Bq_gate, scales_gate, zeros_gate, K, group_size, "_gate")
    if _weights(Bq_up, scales_up, zeros_up, K, group_size, "_up") != N:
        raise ValueError("gate and up must have the same N")
    _need(out, "out", _F32, (1, N))
    d = Call(op=OP_GATED, K=K, N=N, group_size=group_size, A=_ptr(A))
    d.Bq[0], d.scales[0], d.zeros[0] = _ptr(Bq_gate), _ptr(scales_gate), _ptr(zeros_gate)
    d.Bq[1], d.scales[1], d.zeros[1] = _ptr(Bq_up), _ptr(scales_up), _ptr(zeros_up)
    d.out[0] = _ptr(out)
    if W_norm is not None:
        _seq_norm(d, K, W_norm, eps, A_b, residual_out, norm_out)
    elif A_b is not None or residual_out is not None or norm_out is not None:
        raise ValueError("A_b / residual_out / norm_out need W_norm")
    return SeqCall(d, (A, Bq_gate, scales_gate, zeros_gate, Bq_up, scales_up, zeros_up, out,
                       W_norm, A_b, residual_out, norm_out))


def sequence_workspace(device=None):
    """A zero-filled workspace for run_sequence (reusable on one stream)."""
    n = int(lib.gq4_sequence_workspace_bytes())
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def run_sequence(calls, workspace, stream=None):
    """Run the calls in order as one persistent launch (gq4_run_sequence)."""
    _need(workspace, "workspace", (torch.uint8,), (int(lib.gq4_sequence_workspace_bytes()),))
    arr = (Call * max(len(calls), 1))(*[c.desc for c in calls])
    _check(lib.gq4_run_sequence(arr, len(calls), _ptr(workspace), _stream(stream)),
           "gq4_run_sequence")


def sequence_launches(calls) -> int:
    """Persistent launches the calls would take (gq4_sequence_launches; 0 = run call by call)."""
    arr = (Call * max(len(calls), 1))(*[c.desc for c in calls])
    n = _i(0)
    _check(lib.gq4_sequence_launches(arr, len(calls), ctypes.byref(n)), "gq4_sequence_launches")
    return int(n.value)


def run_sequence_static(calls, stream=None):
    """Run the calls in order with the library's fixed scratch (gq4_run_sequence_static)."""
    arr = (Call * max(len(calls), 1))(*[c.desc for c in calls])
    _check(lib.gq4_run_sequence_static(arr, len(calls), _stream(stream)), "gq4_run_sequence_static")


def unpack(Bq, K, q=None, stream=None):
    """Integer unpack test kernel: codes [N, K] uint8."""
    N = Bq.shape[0]
    _need(Bq, "Bq", _WORDS, (N, K // 8))
    if q is None:
        q = torch.empty((N, K), dtype=torch.uint8, device=Bq.device)
    _need(q, "q", (torch.uint8,), (N, K))
    _check(lib.gq4_unpack(K, N, _ptr(Bq), _ptr(q), _stream(stream)), "gq4_unpack")
    return q


def dequant(Bq, scales, zeros, K, group_size, W=None, stream=None):
    """Dequant test kernel: W [N, K] = fl32(fl32(q - zero) * scale)."""
    N = _weights(Bq, scales, zeros, K, group_size)
    if W is None:
        W = torch.empty((N, K), dtype=torch.float32, device=Bq.device)
    _need(W, "W", _F32, (N, K))
    _check(lib.gq4_dequant(K, N, group_size, _ptr(Bq), _ptr(scales), _ptr(zeros), _ptr(W),
                           _stream(stream)), "gq4_dequant")
    return W


def device_error(clear: bool = True) -> int:
    """The library's sticky device error bits (bit 0: the one-lane kernel, bit 1: the
    tensor-core kernel, bit 2: a call sequence gave up a bounded wait; bit 3: the
    quantizer or the cache's writer met a non-finite group; bit 4: the embedding
    gather met an id outside its table; bit 6: a cache slot outside the pool; bit 7:
    kv_plan refused a request; bit 8: kv_attention met a request outside its bounds or
    a page outside the pool; bit 9: its prompt kernel gave up a bounded wait)."""
    bits = ctypes.c_uint(0)
    _check(lib.gq4_device_error(ctypes.byref(bits), int(clear)), "gq4_device_error")
    return int(bits.value)


def version() -> int:
    return int(lib.gq4_version())
