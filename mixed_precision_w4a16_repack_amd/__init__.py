"""Python binding of libw4a16.so: the fused W4A16 linear layer on MI355X.

Argument marshalling only. Every step of the path (repack, dequantisation,
products, reductions, bias, rounding) runs in the HIP kernels of the C
library; this module passes torch tensors' device pointers and the current
stream, allocates outputs with torch, and raises ``RuntimeError`` with the
library's message on any non-zero status. It never falls back to another
implementation: without the built library every call raises.

Names follow the C ABI (include/w4a16.h): ``packed_size``, ``repack``,
``unpack``, ``workspace_size``, ``select_path``, ``gemm``, the dense
prefill variant ``dequant`` and ``gemm_dense``, and the operators between a
decoder layer's GEMMs: ``rmsnorm``, ``silu_mul`` (and their int8 forms
``rmsnorm_a8``, ``silu_mul_a8``), ``kv_cache_size``, ``kv_write``,
``kv_read`` and ``attention``.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a16.so")

UINT4B8 = 0
UINT4 = 1
F16 = 0
BF16 = 1
PATH_AUTO = 0
PATH_SKINNY = 1
PATH_MFMA = 2

KV_ACT = 0
KV_INT8 = 1

_DTYPE_CODE = {torch.float16: F16, torch.bfloat16: BF16}

# C ABI function signatures: name -> (restype, argtypes)
_P, _I64, _I32, _SZ, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "w4a16_abi_version": (_I32, []),
    "w4a16_last_error": (ctypes.c_char_p, []),
    "w4a16_packed_size": (ctypes.c_int, [_I64, _I64, _I32, _I32, ctypes.POINTER(_SZ)]),
    "w4a16_repack": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I32, _I32, _P, _SZ, _P]),
    "w4a16_repack_layout": (ctypes.c_int, [_P, _I32, _I32, _P, _I32, _P, _I32, _I64, _I64, _I32, _I32, _P, _SZ, _P]),
    "w4a16_unpack": (ctypes.c_int, [_P, _I64, _I64, _I32, _I32, _P, _P, _P, _P]),
    "w4a16_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, _I32, _I32, _I32, ctypes.POINTER(_SZ)]),
    "w4a16_workspace_counter_bytes": (_SZ, []),
    "w4a16_select_path": (_I32, [_I64, _I32, _I32]),
    "w4a16_gemm": (
        ctypes.c_int,
        [_P, _I64, _I64, _P, _I64, _I64, _I32, _I32, _I32, _P, _P, _I64, _I32, _I32, _P, _SZ, _P],
    ),
    "w4a16_gemm_noalloc": (
        ctypes.c_int,
        [_P, _I64, _I64, _P, _I64, _I64, _I32, _I32, _I32, _P, _P, _I64, _I32, _I32, _P],
    ),
    "w4a16_dequant": (ctypes.c_int, [_P, _I64, _I64, _I32, _I32, _I32, _P, _I64, _P]),
    "w4a8_quantize": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _I64, _P, _P]),
    "w4a8_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, _I32, ctypes.POINTER(_SZ)]),
    "w4a8_gemm": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _I64, _I64, _I32, _I32, _P, _P, _I64, _P, _SZ, _P]),
    "w4a16_gemm_dense": (
        ctypes.c_int,
        [_P, _I64, _I64, _P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _SZ, _P],
    ),
    "w4a16_rmsnorm": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _F32, _P, _I64, _P, _I64, _P, _I64, _P]),
    "w4a8_rmsnorm": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _F32, _P, _I64, _P, _I64, _P, _I64, _P, _P]),
    "w4a16_silu_mul": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _I64, _P]),
    "w4a8_silu_mul": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _I64, _P, _P]),
    "w4a16_kv_cache_size": (ctypes.c_int, [_I64, _I32, _I32, _I32, _I32, ctypes.POINTER(_SZ)]),
    "w4a16_kv_write": (
        ctypes.c_int,
        [_P, _I64, _I64, _P, _I64, _I64, _I64, _P, _P, _SZ, _I64, _I32, _I32, _I32, _I32, _I32, _P],
    ),
    "w4a16_kv_read": (
        ctypes.c_int,
        [_P, _I64, _P, _SZ, _I64, _I32, _I32, _I32, _I32, _I32, _P, _I64, _I64, _P, _I64, _I64, _P],
    ),
    "w4a16_attention_workspace_size": (
        ctypes.c_int, [_I64, _I32, _I32, _I32, _I32, _I64, _I64, _I32, ctypes.POINTER(_SZ)]),
    "w4a16_attention": (
        ctypes.c_int,
        [_P, _I64, _I64, _I64, _I32, _P, _SZ, _I64, _I32, _I32, _I32, _I32, _I32, _P, _I64, _I64, _P, _I64, _F32,
         _P, _I64, _I64, _P, _SZ, _P],
    ),
}

_lib = None
_lock = threading.Lock()


def load_library(path: str = LIB_PATH):
    """Load libw4a16.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with `python -m mixed_precision_w4a16_repack_amd.build` "
                    "(there is no fallback implementation)"
                )
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def abi_version() -> int:
    return int(load_library().w4a16_abi_version())


def last_error() -> str:
    return load_library().w4a16_last_error().decode()


def _check(status: int):
    if status != 0:
        raise RuntimeError(f"w4a16 status {status}: {last_error()}")


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The same without building the object, where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _stream(t: torch.Tensor):
    return _raw_stream(t.get_device())


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _need_cuda(name: str, t: torch.Tensor | None, dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def packed_size(N: int, K: int, group_size: int, qtype: int) -> int:
    out = _SZ(0)
    _check(load_library().w4a16_packed_size(N, K, group_size, qtype, ctypes.byref(out)))
    return int(out.value)


def repack(weight_packed: torch.Tensor, weight_scale: torch.Tensor, weight_zero_point: torch.Tensor | None,
           group_size: int, qtype: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Checkpoint tensors (GPU) -> packed uint8 buffer (GPU)."""
    _need_cuda("weight_packed", weight_packed, torch.int32)
    _need_cuda("weight_scale", weight_scale, (torch.float16, torch.bfloat16))
    _need_cuda("weight_zero_point", weight_zero_point, torch.int32)
    N, K8 = weight_packed.shape
    K = K8 * 8
    for name, t in (("weight_packed", weight_packed), ("weight_scale", weight_scale),
                    ("weight_zero_point", weight_zero_point)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    nbytes = packed_size(N, K, group_size, qtype)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=weight_packed.device)
    _check(load_library().w4a16_repack(
        _ptr(weight_packed), _ptr(weight_scale), _ptr(weight_zero_point), N, K, group_size, qtype,
        _ptr(out), out.numel() * out.element_size(), _stream(weight_packed)))
    return out


def repack_layout(weight: torch.Tensor, weight_output_dim: int, weight_packed_dim: int, weight_scale: torch.Tensor,
                  scale_output_dim: int, weight_zero_point: torch.Tensor | None, zero_output_dim: int,
                  group_size: int, qtype: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Checkpoint tensors in any orientation w4a16_repack_layout accepts -> packed buffer.

    N and K follow from the weight's shape and dims (the packed dimension holds
    a word per eight entries); the scale and zero-point shapes are checked
    against them before the call.
    """
    _need_cuda("weight", weight, torch.int32)
    _need_cuda("weight_scale", weight_scale, (torch.float16, torch.bfloat16))
    _need_cuda("weight_zero_point", weight_zero_point, torch.int32)
    for name, d in (("weight_output_dim", weight_output_dim), ("weight_packed_dim", weight_packed_dim),
                    ("scale_output_dim", scale_output_dim), ("zero_output_dim", zero_output_dim)):
        if d not in (0, 1):
            raise ValueError(f"{name} must be 0 or 1")
    if weight.dim() != 2:
        raise ValueError("weight must be 2-D")
    dims = list(weight.shape)
    dims[weight_packed_dim] *= 8
    N, K = dims[weight_output_dim], dims[1 - weight_output_dim]
    Kg = 1 if group_size == -1 else (K // group_size if group_size > 0 else 0)
    want_s = (N, Kg) if scale_output_dim == 0 else (Kg, N)
    if tuple(weight_scale.shape) != want_s:
        raise ValueError(f"weight_scale must be {list(want_s)}, got {list(weight_scale.shape)}")
    if weight_zero_point is not None:
        want_z = (N // 8, Kg) if zero_output_dim == 0 else (Kg, N // 8)
        if tuple(weight_zero_point.shape) != want_z:
            raise ValueError(f"weight_zero_point must be {list(want_z)}, got {list(weight_zero_point.shape)}")
    for name, t in (("weight", weight), ("weight_scale", weight_scale), ("weight_zero_point", weight_zero_point)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    nbytes = packed_size(N, K, group_size, qtype)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=weight.device)
    _check(load_library().w4a16_repack_layout(
        _ptr(weight), weight_output_dim, weight_packed_dim, _ptr(weight_scale), scale_output_dim,
        _ptr(weight_zero_point), zero_output_dim, N, K, group_size, qtype,
        _ptr(out), out.numel() * out.element_size(), _stream(weight)))
    return out


def unpack(packed: torch.Tensor, N: int, K: int, group_size: int, qtype: int):
    """Packed buffer -> (codes [N,K] uint8, scale bits [N,Kg] int16, zeros [N,Kg] uint8 or None)."""
    _need_cuda("packed", packed)
    Kg = 1 if group_size == -1 else K // group_size
    dev = packed.device
    codes = torch.empty((N, K), dtype=torch.uint8, device=dev)
    sbits = torch.empty((N, Kg), dtype=torch.int16, device=dev)
    zeros = torch.empty((N, Kg), dtype=torch.uint8, device=dev) if qtype == UINT4 else None
    _check(load_library().w4a16_unpack(_ptr(packed), N, K, group_size, qtype, _ptr(codes), _ptr(sbits),
                                       _ptr(zeros), _stream(packed)))
    return codes, sbits, zeros


def workspace_size(M: int, N: int, K: int, group_size: int, path: int = PATH_AUTO, skinny_max_m: int = 0) -> int:
    out = _SZ(0)
    _check(load_library().w4a16_workspace_size(M, N, K, group_size, path, skinny_max_m, ctypes.byref(out)))
    return int(out.value)


def workspace_counter_bytes() -> int:
    return int(load_library().w4a16_workspace_counter_bytes())


def select_path(M: int, path: int = PATH_AUTO, skinny_max_m: int = 0) -> int:
    r = int(load_library().w4a16_select_path(M, path, skinny_max_m))
    if r < 0:
        raise RuntimeError(f"w4a16 status {r}: {last_error()}")
    return r


class Workspace:
    """A zero-initialised device workspace that grows on demand.

    The library returns the counter region to zero after every call, so one
    workspace serves every shape; calls that share it must be stream-ordered,
    replays of graphs that were captured with it among them.

    For calls that are captured into a graph, size the workspace first, by one
    call of the same sizes before the capture, and keep it as long as the graph.
    Former buffers stay allocated when it grows, since a graph may hold their
    address (it at least doubles, so they are never more than the present one).
    A captured call that needs more than the buffer holds, or that is given no
    workspace, takes memory of the graph's own, whose counter region is cleared
    at each replay (one fill kernel more).
    """

    def __init__(self, device, default: bool = False):
        self.device = torch.device(device)
        self.buf: torch.Tensor | None = None
        # A default workspace belongs to one stream's eager calls: a graph may
        # be replayed beside them, on any stream.
        self._eager_only = default
        self._former: list[torch.Tensor] = []

    def get(self, nbytes: int) -> torch.Tensor | None:
        if nbytes == 0:
            return self.buf
        fits = self.buf is not None and self.buf.numel() >= nbytes
        if fits and not self._eager_only:
            return self.buf
        if torch.cuda.is_current_stream_capturing():
            # Not kept as buf: what is captured clears it at replays only.
            buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            buf[: min(nbytes, workspace_counter_bytes())].zero_()
            return buf
        if not fits:
            if self.buf is not None and not self._eager_only:
                self._former.append(self.buf)
                nbytes = max(nbytes, 2 * self.buf.numel())
            self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        return self.buf


_workspaces: dict = {}


def _default_workspace(device, kind: str = "w4a16") -> Workspace:
    """The default workspace of one kind of call on a device and stream.
    w4a16_gemm and w4a8_gemm get separate ones: w4a16_gemm needs the counter
    region at the start of its workspace to be zero, and w4a8_gemm writes its
    partial results from the start of its own."""
    index = (device if isinstance(device, torch.device) else torch.device(device)).index
    key = (kind, index, _raw_stream(torch.cuda.current_device() if index is None else index))
    ws = _workspaces.get(key)
    if ws is None:
        ws = _workspaces[key] = Workspace(device, default=True)
    return ws


def gemm(A: torch.Tensor, packed: torch.Tensor, N: int, K: int, group_size: int, qtype: int,
         bias: torch.Tensor | None = None, out: torch.Tensor | None = None, path: int = PATH_AUTO,
         skinny_max_m: int = 0, workspace: Workspace | None = None) -> torch.Tensor:
    """C[M, N] = A[M, K] @ dequant(W)^T (+ bias), on the current stream."""
    _need_cuda("A", A, (torch.float16, torch.bfloat16))
    _need_cuda("packed", packed)
    _need_cuda("bias", bias, A.dtype)
    if A.dim() != 2 or A.shape[1] != K or A.stride(1) != 1:
        raise ValueError(f"A must be [M, K={K}] with unit column stride, got {tuple(A.shape)} {A.stride()}")
    M = A.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=A.dtype, device=A.device)
    _need_cuda("out", out, A.dtype)
    if out.dim() != 2 or tuple(out.shape) != (M, N) or out.stride(1) != 1:
        raise ValueError(f"out must be [M={M}, N={N}] with unit column stride")
    if bias is not None and (bias.dim() != 1 or bias.shape[0] != N or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous [N={N}] tensor")
    ws_bytes = workspace_size(M, N, K, group_size, path, skinny_max_m) if M > 0 else 0
    ws = (workspace or _default_workspace(A.device)).get(ws_bytes)
    _check(load_library().w4a16_gemm(
        _ptr(A), M, A.stride(0), _ptr(packed), N, K, group_size, qtype, _DTYPE_CODE[A.dtype], _ptr(bias),
        _ptr(out), out.stride(0), path, skinny_max_m, _ptr(ws) if ws_bytes else None,
        ws.numel() if (ws is not None and ws_bytes) else 0, _stream(A)))
    return out


def gemm_noalloc(A: torch.Tensor, packed: torch.Tensor, N: int, K: int, group_size: int, qtype: int,
                 bias: torch.Tensor | None = None, out: torch.Tensor | None = None, path: int = PATH_AUTO,
                 skinny_max_m: int = 0) -> torch.Tensor:
    """``gemm`` through w4a16_gemm_noalloc: the split-K workspace is the
    library's static device scratch (no workspace argument). With ``out``
    given, the call allocates nothing, here or in the library."""
    _need_cuda("A", A, (torch.float16, torch.bfloat16))
    _need_cuda("packed", packed)
    _need_cuda("bias", bias, A.dtype)
    if A.dim() != 2 or A.shape[1] != K or A.stride(1) != 1:
        raise ValueError(f"A must be [M, K={K}] with unit column stride, got {tuple(A.shape)} {A.stride()}")
    M = A.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=A.dtype, device=A.device)
    _need_cuda("out", out, A.dtype)
    if out.dim() != 2 or tuple(out.shape) != (M, N) or out.stride(1) != 1:
        raise ValueError(f"out must be [M={M}, N={N}] with unit column stride")
    if bias is not None and (bias.dim() != 1 or bias.shape[0] != N or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous [N={N}] tensor")
    _check(load_library().w4a16_gemm_noalloc(
        _ptr(A), M, A.stride(0), _ptr(packed), N, K, group_size, qtype, _DTYPE_CODE[A.dtype], _ptr(bias),
        _ptr(out), out.stride(0), path, skinny_max_m, _stream(A)))
    return out


def dequant(packed: torch.Tensor, N: int, K: int, group_size: int, qtype: int, dtype: torch.dtype,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """Packed buffer -> dense [N, K] weight RN((q - z) * s) in ``dtype`` (fp16 or bf16)."""
    _need_cuda("packed", packed)
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"dtype {dtype} is not fp16 or bf16")
    if out is None:
        out = torch.empty((N, K), dtype=dtype, device=packed.device)
    _need_cuda("out", out, dtype)
    if out.dim() != 2 or tuple(out.shape) != (N, K) or out.stride(1) != 1:
        raise ValueError(f"out must be [N={N}, K={K}] with unit column stride")
    _check(load_library().w4a16_dequant(_ptr(packed), N, K, group_size, qtype, _DTYPE_CODE[dtype], _ptr(out),
                                        out.stride(0), _stream(packed)))
    return out


def quantize_a8(A: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """Per-token symmetric int8 quantisation: A [M, K] -> (qa [M, K] int8, xs [M] fp32).

    Each run of 8 codes of qa is stored in the order 0, 4, 1, 5, 2, 6, 3, 7
    (the packed weight's code order, which ``gemm_w4a8`` expects)."""
    _need_cuda("A", A, (torch.float16, torch.bfloat16))
    if A.dim() != 2 or A.stride(1) != 1:
        raise ValueError("A must be 2-D with unit column stride")
    M, K = A.shape
    if out is None:
        qa = torch.empty((M, K), dtype=torch.int8, device=A.device)
        xs = torch.empty((M,), dtype=torch.float32, device=A.device)
    else:
        qa, xs = out
        _need_cuda("qa", qa, torch.int8)
        _need_cuda("xs", xs, torch.float32)
        if qa.dim() != 2 or tuple(qa.shape) != (M, K) or qa.stride(1) != 1 or xs.shape != (M,):
            raise ValueError("out must be (qa [M, K] with unit column stride, xs [M])")
    _check(load_library().w4a8_quantize(_ptr(A), M, K, A.stride(0), _DTYPE_CODE[A.dtype], _ptr(qa), qa.stride(0),
                                        _ptr(xs), _stream(A)))
    return qa, xs


def w4a8_workspace_size(M: int, N: int, K: int, group_size: int) -> int:
    out = _SZ(0)
    _check(load_library().w4a8_workspace_size(M, N, K, group_size, ctypes.byref(out)))
    return int(out.value)


def gemm_w4a8(qa: torch.Tensor, xs: torch.Tensor, packed: torch.Tensor, N: int, K: int, group_size: int,
              dtype: torch.dtype, bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
              workspace: Workspace | None = None) -> torch.Tensor:
    """C[M, N] from int8 activations (quantize_a8) and a symmetric (uint4b8) packed weight."""
    _need_cuda("qa", qa, torch.int8)
    _need_cuda("xs", xs, torch.float32)
    _need_cuda("packed", packed)
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"dtype {dtype} is not fp16 or bf16")
    _need_cuda("bias", bias, dtype)
    if qa.dim() != 2 or qa.shape[1] != K or qa.stride(1) != 1:
        raise ValueError(f"qa must be [M, K={K}] with unit column stride")
    M = qa.shape[0]
    if xs.shape != (M,) or not xs.is_contiguous():
        raise ValueError(f"xs must be a contiguous [M={M}] tensor")
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=qa.device)
    _need_cuda("out", out, dtype)
    if out.dim() != 2 or tuple(out.shape) != (M, N) or out.stride(1) != 1:
        raise ValueError(f"out must be [M={M}, N={N}] with unit column stride")
    if bias is not None and (bias.dim() != 1 or bias.shape[0] != N or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous [N={N}] tensor")
    ws_bytes = w4a8_workspace_size(M, N, K, group_size) if M > 0 else 0
    ws = (workspace or _default_workspace(qa.device, "w4a8")).get(ws_bytes)
    _check(load_library().w4a8_gemm(
        _ptr(qa), _ptr(xs), M, qa.stride(0), _ptr(packed), N, K, group_size, _DTYPE_CODE[dtype], _ptr(bias),
        _ptr(out), out.stride(0), _ptr(ws) if ws_bytes else None, ws.numel() if (ws is not None and ws_bytes) else 0,
        _stream(qa)))
    return out


def gemm_dense(A: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C[M, N] = A[M, K] @ W[N, K]^T (+ bias) for a dense weight (e.g. from ``dequant``), via hipBLASLt."""
    _need_cuda("A", A, (torch.float16, torch.bfloat16))
    _need_cuda("W", W, A.dtype)
    _need_cuda("bias", bias, A.dtype)
    if A.dim() != 2 or A.stride(1) != 1 or W.dim() != 2 or W.stride(1) != 1 or W.shape[1] != A.shape[1]:
        raise ValueError(f"A [M, K] and W [N, K] need unit column strides and equal K, got {tuple(A.shape)}, {tuple(W.shape)}")
    M, K = A.shape
    N = W.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=A.dtype, device=A.device)
    _need_cuda("out", out, A.dtype)
    if out.dim() != 2 or tuple(out.shape) != (M, N) or out.stride(1) != 1:
        raise ValueError(f"out must be [M={M}, N={N}] with unit column stride")
    if bias is not None and (bias.dim() != 1 or bias.shape[0] != N or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous [N={N}] tensor")
    _need_cuda("workspace", workspace)
    _check(load_library().w4a16_gemm_dense(
        _ptr(A), M, A.stride(0), _ptr(W), N, K, W.stride(0), _DTYPE_CODE[A.dtype], _ptr(bias), _ptr(out),
        out.stride(0), _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(A)))
    return out


def _same_device(first: torch.Tensor, **others: torch.Tensor | None):
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")


# The operators between the GEMMs are often shorter than their checks, so each
# argument is first compared as a whole; only one that does not fit is looked
# at again, for the message.


def _fits(t: torch.Tensor, shape, dtype, device: int) -> bool:
    return t.dtype is dtype and t.shape == shape and t.get_device() == device and t.stride(-1) == 1


def _empty(like: torch.Tensor, shape) -> torch.Tensor:
    """A contiguous tensor of the shape, which is `like`'s."""
    return torch.empty_like(like) if like.is_contiguous() else torch.empty(shape, dtype=like.dtype, device=like.device)


def _rows(name: str, t: torch.Tensor, x: torch.Tensor, M: int, K: int):
    """t must be [M, K] rows of x's dtype on its device."""
    if _fits(t, (M, K), x.dtype, x.get_device()):
        return
    _need_cuda(name, t, x.dtype)
    if tuple(t.shape) != (M, K) or t.stride(1) != 1:
        raise ValueError(f"{name} must be [M={M}, K={K}] with unit column stride, got {tuple(t.shape)} {t.stride()}")
    _same_device(x, **{name: t})


def _ld(t: torch.Tensor | None, M: int, K: int) -> int:
    """Row stride of [M, K] rows (torch gives a single row any stride)."""
    return 0 if t is None else t.stride(0) if M > 1 else K


def _codes_out(out, x: torch.Tensor, M: int, K: int):
    device = x.device
    if out is None:
        return (torch.empty((M, K), dtype=torch.int8, device=device),
                torch.empty((M,), dtype=torch.float32, device=device))
    qa, xs = out
    _need_cuda("qa", qa, torch.int8)
    _need_cuda("xs", xs, torch.float32)
    if tuple(qa.shape) != (M, K) or qa.stride(1) != 1 or xs.shape != (M,) or not xs.is_contiguous():
        raise ValueError(f"out must be (qa [M={M}, K={K}] with unit column stride, contiguous xs [M={M}])")
    _same_device(x, qa=qa, xs=xs)
    return qa, xs


def _ld_codes(qa: torch.Tensor, M: int, K: int) -> int:
    return qa.stride(0) if M > 1 else (K + 7) // 8 * 8


def _norm_args(x, weight, residual, residual_out):
    if not x.is_cuda or x.dtype not in _DTYPE_CODE:
        _need_cuda("x", x, (torch.float16, torch.bfloat16))
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    if not _fits(weight, (K,), x.dtype, x.get_device()):
        _need_cuda("weight", weight, x.dtype)
        if tuple(weight.shape) != (K,) or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous [K={K}] tensor")
        _same_device(x, weight=weight)
    if residual is not None:
        _rows("residual", residual, x, M, K)
    if residual_out is not None and residual_out is not residual:
        _rows("residual_out", residual_out, x, M, K)
    return M, K


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, residual: torch.Tensor | None = None,
            residual_out: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = h / sqrt(mean(h^2) + eps) * weight per row of h = x (+ residual).

    ``residual_out`` (which may be ``residual`` itself) receives h."""
    M, K = _norm_args(x, weight, residual, residual_out)
    if out is None:
        out = _empty(x, (M, K))
    else:
        _rows("out", out, x, M, K)
    status = (_lib or load_library()).w4a16_rmsnorm(
        x.data_ptr(), M, K, x.stride(0) if M > 1 else K, _DTYPE_CODE[x.dtype], weight.data_ptr(), eps,
        _ptr(residual), _ld(residual, M, K), _ptr(residual_out), _ld(residual_out, M, K),
        out.data_ptr(), out.stride(0) if M > 1 else K, _raw_stream(x.get_device()))
    if status:
        _check(status)
    return out


def rmsnorm_a8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, residual: torch.Tensor | None = None,
               residual_out: torch.Tensor | None = None, out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """``rmsnorm`` as the input of ``gemm_w4a8``: (qa [M, K] int8, xs [M] fp32), as ``quantize_a8`` stores them."""
    M, K = _norm_args(x, weight, residual, residual_out)
    qa, xs = _codes_out(out, x, M, K)
    status = (_lib or load_library()).w4a8_rmsnorm(
        x.data_ptr(), M, K, x.stride(0) if M > 1 else K, _DTYPE_CODE[x.dtype], weight.data_ptr(), eps,
        _ptr(residual), _ld(residual, M, K), _ptr(residual_out), _ld(residual_out, M, K),
        qa.data_ptr(), _ld_codes(qa, M, K), xs.data_ptr(), _raw_stream(x.get_device()))
    if status:
        _check(status)
    return qa, xs


def _gate_args(x):
    if not x.is_cuda or x.dtype not in _DTYPE_CODE:
        _need_cuda("x", x, (torch.float16, torch.bfloat16))
    if x.dim() != 2 or x.stride(1) != 1 or x.shape[1] % 2:
        raise ValueError(f"x must be [M, 2*K] with unit column stride, got {tuple(x.shape)} {x.stride()}")
    return x.shape[0], x.shape[1] // 2


def silu_mul(x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """silu(g) * u of x [M, 2K] = [g | u] (a fused gate/up product)."""
    M, K = _gate_args(x)
    if out is None:
        out = torch.empty((M, K), dtype=x.dtype, device=x.device)
    else:
        _rows("out", out, x, M, K)
    status = (_lib or load_library()).w4a16_silu_mul(
        x.data_ptr(), M, K, x.stride(0) if M > 1 else 2 * K, _DTYPE_CODE[x.dtype], out.data_ptr(),
        out.stride(0) if M > 1 else K, _raw_stream(x.get_device()))
    if status:
        _check(status)
    return out


def silu_mul_a8(x: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """``silu_mul`` as the input of ``gemm_w4a8``: (qa [M, K] int8, xs [M] fp32)."""
    M, K = _gate_args(x)
    qa, xs = _codes_out(out, x, M, K)
    status = (_lib or load_library()).w4a8_silu_mul(
        x.data_ptr(), M, K, x.stride(0) if M > 1 else 2 * K, _DTYPE_CODE[x.dtype], qa.data_ptr(), _ld_codes(qa, M, K),
        xs.data_ptr(), _raw_stream(x.get_device()))
    if status:
        _check(status)
    return qa, xs


def kv_cache_size(pages: int, kv_heads: int, head_dim: int, page_size: int, kind: int) -> int:
    """Bytes of a paged key/value cache (allocate them as uint8)."""
    out = _SZ(0)
    _check(load_library().w4a16_kv_cache_size(pages, kv_heads, head_dim, page_size, kind, ctypes.byref(out)))
    return int(out.value)


def _heads(name: str, t: torch.Tensor, shape, dtype, device: int):
    if _fits(t, shape, dtype, device):
        return
    _need_cuda(name, t, dtype)
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if t.dim() != 3 or tuple(t.shape) != tuple(shape) or t.stride(2) != 1:
        raise ValueError(f"{name} must be {list(shape)} with unit stride in its last dimension, "
                         f"got {tuple(t.shape)} {t.stride()}")


def _cache_bytes(cache: torch.Tensor, device: int) -> int:
    if cache.get_device() != device:
        _need_cuda("cache", cache)
        raise ValueError(f"cache is on {cache.device}, expected cuda:{device}")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    return cache.numel() * cache.element_size()


def _slots(slots: torch.Tensor) -> int:
    if not slots.is_cuda or slots.dtype is not torch.int64:
        _need_cuda("slots", slots, torch.int64)
    if slots.dim() != 1 or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous [T] tensor")
    return slots.shape[0]


def kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor, pages: int, page_size: int,
             kind: int) -> None:
    """Writes keys and values [T, kv_heads, head_dim] to their slots (page * page_size + offset; -1: not written).

    Any token and head strides; ``kind`` is ``KV_ACT`` (values in k's dtype) or ``KV_INT8``."""
    if not k.is_cuda or k.dtype not in _DTYPE_CODE:
        _need_cuda("k", k, (torch.float16, torch.bfloat16))
    T = _slots(slots)
    if k.dim() != 3:
        raise ValueError("k must be [T, kv_heads, head_dim]")
    device, dtype = k.get_device(), k.dtype
    H, D = k.shape[1:]
    _heads("k", k, (T, H, D), dtype, device)
    _heads("v", v, (T, H, D), dtype, device)
    nbytes = _cache_bytes(cache, device)
    if slots.get_device() != device:
        _same_device(k, slots=slots)
    status = (_lib or load_library()).w4a16_kv_write(
        k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), T, slots.data_ptr(),
        cache.data_ptr(), nbytes, pages, H, D, page_size, kind, _DTYPE_CODE[dtype], _raw_stream(device))
    if status:
        _check(status)


def kv_read(slots: torch.Tensor, cache: torch.Tensor, pages: int, kv_heads: int, head_dim: int, page_size: int,
            kind: int, dtype: torch.dtype, out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """The keys and values [T, kv_heads, head_dim] of slots, in ``dtype`` (zeros for a slot outside the cache)."""
    T = _slots(slots)
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"dtype {dtype} is not fp16 or bf16")
    shape, device = (T, kv_heads, head_dim), slots.get_device()
    if out is None:
        k = torch.empty(shape, dtype=dtype, device=slots.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        _heads("k", k, shape, dtype, device)
        _heads("v", v, shape, dtype, device)
    nbytes = _cache_bytes(cache, device)
    status = (_lib or load_library()).w4a16_kv_read(
        slots.data_ptr(), T, cache.data_ptr(), nbytes, pages, kv_heads, head_dim, page_size, kind, _DTYPE_CODE[dtype],
        k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), _raw_stream(device))
    if status:
        _check(status)
    return k, v


@functools.lru_cache(maxsize=4096)
def attention_workspace_size(B: int, q_heads: int, kv_heads: int, head_dim: int, page_size: int, table_width: int,
                             window: int, kind: int) -> int:
    out = _SZ(0)
    _check(load_library().w4a16_attention_workspace_size(B, q_heads, kv_heads, head_dim, page_size, table_width,
                                                         window, kind, ctypes.byref(out)))
    return int(out.value)


def attention(q: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor, pages: int,
              kv_heads: int, page_size: int, kind: int, window: int = 0, scale: float | None = None,
              out: torch.Tensor | None = None, workspace: Workspace | None = None) -> torch.Tensor:
    """Attention of one new token per sequence over the cache: q [B, q_heads, head_dim] -> the same shape.

    ``table`` [B, width] int32 holds each sequence's pages, ``lengths`` [B] int32 its tokens (the new one
    included); ``window`` > 0 sees only the last tokens; ``scale`` defaults to head_dim ** -0.5. For calls that
    are captured into a graph see ``Workspace``."""
    if not q.is_cuda or q.dtype not in _DTYPE_CODE:
        _need_cuda("q", q, (torch.float16, torch.bfloat16))
    if q.dim() != 3:
        raise ValueError("q must be [B, q_heads, head_dim]")
    B, Hq, D = shape = q.shape
    device, dtype = q.get_device(), q.dtype
    _heads("q", q, shape, dtype, device)
    if out is None:
        out = _empty(q, shape)
    else:
        _heads("out", out, shape, dtype, device)
    if table.dtype is not torch.int32 or table.get_device() != device:
        _need_cuda("table", table, torch.int32)
        _same_device(q, table=table)
    if table.dim() != 2 or table.shape[0] != B or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"table must be [B={B}, width] with unit column stride")
    if lengths.dtype is not torch.int32 or lengths.get_device() != device:
        _need_cuda("lengths", lengths, torch.int32)
        _same_device(q, lengths=lengths)
    if lengths.shape != (B,) or not lengths.is_contiguous():
        raise ValueError(f"lengths must be a contiguous [B={B}] tensor")
    nbytes = _cache_bytes(cache, device)
    width = table.shape[1]
    stream = _raw_stream(device)
    ws_ptr, ws_bytes = None, 0
    if B > 0:
        need = attention_workspace_size(B, Hq, kv_heads, D, page_size, width, window, kind)
        # the first look is _default_workspace's own, without building the device object
        ws = (workspace or _workspaces.get(("attention", device, stream)) or _default_workspace(q.device, "attention")).get(need)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel()
    status = (_lib or load_library()).w4a16_attention(
        q.data_ptr(), q.stride(0), q.stride(1), B, Hq, cache.data_ptr(), nbytes, pages, kv_heads, D, page_size, kind,
        _DTYPE_CODE[dtype], table.data_ptr(), width, table.stride(0) if B > 1 else width, lengths.data_ptr(), window,
        D ** -0.5 if scale is None else scale, out.data_ptr(), out.stride(0), out.stride(1), ws_ptr, ws_bytes, stream)
    if status:
        _check(status)
    return out
