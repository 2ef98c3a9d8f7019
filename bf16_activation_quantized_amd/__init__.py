"""Python binding of the W4A16 GEMM library (libw4a16.so, C ABI in include/w4a16.h;
the kernel-forcing entry points used by tests and benchmarks are declared in
csrc/w4a16_internal.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of the library. PyTorch provides device memory and the current
stream. There is no fallback: if the library is not built, every call raises.

bf16 tensors are passed as torch.bfloat16 (their raw bits are what the
library reads); packed weights and nibbles are torch.uint8; group sizes are
torch.int32.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a16.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "w4a16.h")
INTERNAL_HEADER = os.path.join(_HERE, "csrc", "w4a16_internal.h")

GROUP_SIZE = 128
PATH_AUTO, PATH_GEMV, PATH_SKINNY, PATH_TILE = 0, 1, 2, 3

_STATUS_NAMES = {0: "W4A16_OK", 1: "W4A16_ERR_NULL", 2: "W4A16_ERR_SHAPE", 3: "W4A16_ERR_GROUP_SIZE",
                 4: "W4A16_ERR_SPLIT_K", 5: "W4A16_ERR_WORKSPACE", 6: "W4A16_ERR_ALIGN",
                 7: "W4A16_ERR_LAUNCH"}


class W4A16Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class _Config(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("variant", ctypes.c_int32)]


_lib_handle = None


def _lib():
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"W4A16 HIP library not built ({LIB_PATH} missing); run "
                           "python -m bf16_activation_quantized_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    sig = {
        "w4a16_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "w4a16_pack_int4": (ctypes.c_int, [P, P, I64, I64, P]),
        "w4a16_gemm_auto_split_k": (I32, [I64, I64, I64, I32]),
        "w4a16_gemm_workspace_bytes": (SZ, [I64, I64, I64, I32]),
        "w4a16_gemm_workspace_bytes_gs": (SZ, [I64, I64, I64, I32, I32]),
        "w4a16_gemm": (ctypes.c_int, [P, P, P, P, I64, I64, I64, I32, I32, P, SZ, P]),
        "w4a16_gemm_grouped": (ctypes.c_int, [P, P, P, P, P, I32, I64, I64, I64, I32, P]),
        "w4a16_gemm_batched_workspace_bytes": (SZ, [I32, I64, I64, I64, I32, I32]),
        "w4a16_gemm_batched": (ctypes.c_int, [P, P, P, P, I32, I64, I64, I64, I32, I32, P, SZ, P]),
        "w4a16_splitk_reduce": (ctypes.c_int, [P, P, I32, I64, I64, P]),
        "w4a16_gemm_noalloc": (ctypes.c_int, [P, P, P, P, I64, I64, I64, I32, I32, P]),
        "w4a16_gemm_lora_workspace_bytes": (SZ, [I64, I64, I64, I32, I32, I32, I32]),
        "w4a16_gemm_lora": (ctypes.c_int, [P, P, P, P, P, P, P, P, I64, I64, I64, I32, I32, I32, I32, P, SZ, P]),
        "w4a16_expert_sort_workspace_bytes": (SZ, [I64, I32, I32]),
        "w4a16_expert_sort": (ctypes.c_int, [P, P, P, P, I64, I32, I32, P, SZ, P]),
        "w4a16_expert_gather": (ctypes.c_int, [P, P, P, I64, I32, I64, I64, P]),
        "w4a16_expert_gather_grad": (ctypes.c_int, [P, P, P, I64, I32, I64, I64, P]),
        "w4a16_expert_combine": (ctypes.c_int, [P, P, P, P, I64, I32, I64, I64, P]),
        "w4a16_expert_combine_grad": (ctypes.c_int, [P, P, P, P, P, P, I64, I32, I64, I64, P]),
        "w4a16_fp8_quantize": (ctypes.c_int, [P, P, P, I64, I64, I32, P]),
        "w4a16_fp8_gemm_workspace_bytes": (SZ, [I64, I64, I64]),
        "w4a16_fp8_gemm": (ctypes.c_int, [P, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "w4a16_fp8_gemm_grouped": (ctypes.c_int, [P, P, P, P, P, P, I32, I64, I64, I64, P]),
        "w4a16_fp8_gemm_grad_workspace_bytes": (SZ, [I64, I64, I64]),
        "w4a16_fp8_gemm_grad": (ctypes.c_int, [P, P, P, P, P, P, I32, I64, I64, I64, P, SZ, P]),
        "w4a16_gemm_grad_workspace_bytes": (SZ, [I32, I64, I64, I64, I32]),
        "w4a16_gemm_grad": (ctypes.c_int, [P, P, P, P, P, I32, I64, I64, I64, I32, P, SZ, P]),
        # internal entry points that force a kernel (tests, benchmarks)
        "w4a16_gemm_auto_config": (ctypes.c_int, [I64, I64, I64, I32, P, P]),
        "w4a16_gemm_workspace_bytes_ex": (SZ, [I64, I64, I64, I32, I32, P]),
        "w4a16_gemm_ex": (ctypes.c_int, [P, P, P, P, I64, I64, I64, I32, I32, P, SZ, P, P]),
        "w4a16_gemm_grouped_ex": (ctypes.c_int, [P, P, P, P, P, I32, I64, I64, I64, I32, P, P]),
        "w4a16_gemm_batched_workspace_bytes_ex": (SZ, [I32, I64, I64, I64, I32, I32, P]),
        "w4a16_gemm_batched_ex": (ctypes.c_int, [P, P, P, P, I32, I64, I64, I64, I32, I32, P, SZ, P, P]),
    }
    sig.update({
        "w4a16_fp8_gemm_workspace_bytes_ex": (SZ, [I32, I64, I64, I64, I32, I32]),
        "w4a16_fp8_gemm_ex": (ctypes.c_int, [I32, P, P, P, P, P, P, I32, I64, I64, I64, I32, I32, P, SZ, P]),
        "w4a16_fp8_gemm_auto": (ctypes.c_int, [I32, I32, I32, I64, I64, I64, P, P]),
        "w4a16_gemm_grad_workspace_bytes_ex": (SZ, [I32, I64, I64, I64, I32, I32, I32]),
        "w4a16_gemm_grad_ex": (ctypes.c_int, [P, P, P, P, P, I32, I64, I64, I64, I32, I32, I32, P, SZ, P]),
        "w4a16_gemm_grad_auto": (ctypes.c_int, [I32, I32, I64, I64, I64, I32, P, P]),
    })
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib_handle = L
    return L


def header_functions(path: str = HEADER) -> list:
    """Names of the functions a header (default include/w4a16.h) declares."""
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(w4a16_[a-z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    try:
        return _lib().w4a16_status_string(int(status)).decode()
    except RuntimeError:
        return _STATUS_NAMES.get(int(status), "unknown")


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _cfg(path: Optional[int], variant: Optional[int]):
    if path is None and variant is None:
        return None
    return ctypes.byref(_Config(int(path or 0), int(-1 if variant is None else variant)))


def _raise(status: int, what: str):
    if status != 0:
        raise W4A16Error(status, what)


# ------------------------------------------------------------------ entry points

def w4a16_pack_int4(q: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """q [..., K] uint8 nibbles -> packed [..., K/2] (low nibble = even k)."""
    _check(q, "q", torch.uint8)
    K = q.shape[-1]
    rows = q.numel() // K if K else 0
    if out is None:
        out = torch.empty(q.shape[:-1] + (K // 2,), dtype=torch.uint8, device=q.device)
    _check(out, "out", torch.uint8, q.shape[:-1] + (K // 2,))
    _raise(_lib().w4a16_pack_int4(_ptr(q), _ptr(out), rows, K, _stream(stream)), "w4a16_pack_int4")
    return out


def w4a16_gemm_auto_split_k(M: int, N: int, K: int, group_size: int = GROUP_SIZE) -> int:
    return int(_lib().w4a16_gemm_auto_split_k(M, N, K, group_size))


def w4a16_gemm_auto_config(M: int, N: int, K: int, group_size: int = GROUP_SIZE) -> tuple:
    """The automatic choice of w4a16_gemm at these sizes (internal entry
    point): (path, variant, split_k); path 0 when nothing would run (M = 0)."""
    cfg, sk = _Config(), ctypes.c_int32(0)
    _raise(_lib().w4a16_gemm_auto_config(M, N, K, group_size, ctypes.byref(cfg), ctypes.byref(sk)),
           "w4a16_gemm_auto_config")
    return int(cfg.path), int(cfg.variant), int(sk.value)


def w4a16_gemm_workspace_bytes(M: int, N: int, K: int, split_k: int = 0,
                               path: Optional[int] = None, variant: Optional[int] = None,
                               group_size: int = GROUP_SIZE) -> int:
    """Workspace bytes of w4a16_gemm (0 when the effective split is 1)."""
    cfg = _cfg(path, variant)
    if cfg is not None:
        return int(_lib().w4a16_gemm_workspace_bytes_ex(M, N, K, group_size, split_k, cfg))
    if group_size != GROUP_SIZE:
        return int(_lib().w4a16_gemm_workspace_bytes_gs(M, N, K, group_size, split_k))
    return int(_lib().w4a16_gemm_workspace_bytes(M, N, K, split_k))


def _workspace(need: int, workspace: Optional[torch.Tensor], device) -> Optional[torch.Tensor]:
    if workspace is None and need > 0:
        workspace = torch.empty(need // 4 + 1, dtype=torch.float32, device=device)
    if workspace is not None:
        _check(workspace, "workspace", torch.float32)
    return workspace


def w4a16_gemm(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor,
               y: Optional[torch.Tensor] = None, split_k: int = 0,
               workspace: Optional[torch.Tensor] = None, path: Optional[int] = None,
               variant: Optional[int] = None, stream=None, group_size: int = GROUP_SIZE) -> torch.Tensor:
    """Y[M, N] = X[M, K] . dequant(W)[N, K]^T (bf16 out, fp32 accumulation).
    `path` / `variant` force a kernel (internal entry point w4a16_gemm_ex)."""
    _check(x, "x", torch.bfloat16)
    M, K = x.shape
    N = w_packed.shape[0]
    _check(w_packed, "w_packed", torch.uint8, (N, K // 2))
    _check(scales, "scales", torch.bfloat16, (N, K // group_size))
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check(y, "y", torch.bfloat16, (M, N))
    workspace = _workspace(w4a16_gemm_workspace_bytes(M, N, K, split_k, path, variant, group_size), workspace,
                           x.device)
    wbytes = 0 if workspace is None else workspace.numel() * 4
    cfg = _cfg(path, variant)
    L = _lib()
    if cfg is None:
        st = L.w4a16_gemm(_ptr(x), _ptr(w_packed), _ptr(scales), _ptr(y), M, N, K, group_size, split_k,
                          _ptr(workspace), wbytes, _stream(stream))
    else:
        st = L.w4a16_gemm_ex(_ptr(x), _ptr(w_packed), _ptr(scales), _ptr(y), M, N, K, group_size, split_k,
                             _ptr(workspace), wbytes, _stream(stream), cfg)
    _raise(st, "w4a16_gemm")
    return y


NOALLOC_SCRATCH_BYTES = 16 << 20


def w4a16_gemm_noalloc(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor, y: torch.Tensor,
                       split_k: int = 0, stream=None, group_size: int = GROUP_SIZE) -> torch.Tensor:
    """w4a16_gemm with the library's own device scratch in place of a
    workspace (the C entry point allocates nothing; y must be given)."""
    _check(x, "x", torch.bfloat16)
    M, K = x.shape
    N = w_packed.shape[0]
    _check(w_packed, "w_packed", torch.uint8, (N, K // 2))
    _check(scales, "scales", torch.bfloat16, (N, K // group_size))
    _check(y, "y", torch.bfloat16, (M, N))
    _raise(_lib().w4a16_gemm_noalloc(_ptr(x), _ptr(w_packed), _ptr(scales), _ptr(y), M, N, K, group_size, split_k,
                                     _stream(stream)), "w4a16_gemm_noalloc")
    return y


def w4a16_gemm_grouped(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor,
                       m_sizes: torch.Tensor, y: Optional[torch.Tensor] = None,
                       variant: Optional[int] = None, stream=None, group_size: int = GROUP_SIZE) -> torch.Tensor:
    """Grouped GEMM in one launch; m_sizes stays on the device. `variant`
    forces the tile height in rows (internal entry point)."""
    _check(x, "x", torch.bfloat16)
    M_total, K = x.shape
    G, N = w_packed.shape[0], w_packed.shape[1]
    _check(w_packed, "w_packed", torch.uint8, (G, N, K // 2))
    _check(scales, "scales", torch.bfloat16, (G, N, K // group_size))
    _check(m_sizes, "m_sizes", torch.int32, (G,))
    if y is None:
        y = torch.empty((M_total, N), dtype=torch.bfloat16, device=x.device)
    _check(y, "y", torch.bfloat16, (M_total, N))
    L = _lib()
    if variant is None:
        st = L.w4a16_gemm_grouped(_ptr(x), _ptr(w_packed), _ptr(scales), _ptr(m_sizes), _ptr(y), G, M_total, N, K,
                                  group_size, _stream(stream))
    else:
        st = L.w4a16_gemm_grouped_ex(_ptr(x), _ptr(w_packed), _ptr(scales), _ptr(m_sizes), _ptr(y), G, M_total, N,
                                     K, group_size, _stream(stream), _cfg(PATH_TILE, variant))
    _raise(st, "w4a16_gemm_grouped")
    return y


def w4a16_gemm_batched_workspace_bytes(B: int, M: int, N: int, K: int, split_k: int = 0,
                                       variant: Optional[int] = None, group_size: int = GROUP_SIZE) -> int:
    L = _lib()
    if variant is None:
        return int(L.w4a16_gemm_batched_workspace_bytes(B, M, N, K, group_size, split_k))
    return int(L.w4a16_gemm_batched_workspace_bytes_ex(B, M, N, K, group_size, split_k, _cfg(PATH_TILE, variant)))


def w4a16_gemm_batched(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor,
                       y: Optional[torch.Tensor] = None, split_k: int = 0,
                       workspace: Optional[torch.Tensor] = None, variant: Optional[int] = None,
                       stream=None, group_size: int = GROUP_SIZE) -> torch.Tensor:
    """Y[b] = X[b] . dequant(W[b])^T for B independent problems, one launch."""
    _check(x, "x", torch.bfloat16)
    B, M, K = x.shape
    N = w_packed.shape[1]
    _check(w_packed, "w_packed", torch.uint8, (B, N, K // 2))
    _check(scales, "scales", torch.bfloat16, (B, N, K // group_size))
    if y is None:
        y = torch.empty((B, M, N), dtype=torch.bfloat16, device=x.device)
    _check(y, "y", torch.bfloat16, (B, M, N))
    workspace = _workspace(w4a16_gemm_batched_workspace_bytes(B, M, N, K, split_k, variant, group_size), workspace,
                           x.device)
    wbytes = 0 if workspace is None else workspace.numel() * 4
    L = _lib()
    if variant is None:
        st = L.w4a16_gemm_batched(_ptr(x), _ptr(w_packed), _ptr(scales), _ptr(y), B, M, N, K, group_size, split_k,
                                  _ptr(workspace), wbytes, _stream(stream))
    else:
        st = L.w4a16_gemm_batched_ex(_ptr(x), _ptr(w_packed), _ptr(scales), _ptr(y), B, M, N, K, group_size,
                                     split_k, _ptr(workspace), wbytes, _stream(stream), _cfg(PATH_TILE, variant))
    _raise(st, "w4a16_gemm_batched")
    return y


def w4a16_splitk_reduce(workspace: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = bf16_rne(sum over slices of workspace[SK, M, N]) in slice order."""
    _check(workspace, "workspace", torch.float32)
    SK, M, N = workspace.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=workspace.device)
    _check(y, "y", torch.bfloat16, (M, N))
    _raise(_lib().w4a16_splitk_reduce(_ptr(workspace), _ptr(y), SK, M, N, _stream(stream)), "w4a16_splitk_reduce")
    return y


# ------------------------------------------------------------------ low-rank adapters, rows of a mixture of experts
# These calls are short (a few us on the GPU), so their checks are one pass
# over each tensor's own attributes.

def _in(t, name: str, dtype, shape, dev: int) -> int:
    """The address of a contiguous tensor of this type and shape on device
    `dev`; raises what `_check` raises, or ValueError for another device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev >= 0 and t.shape == shape and \
            t.is_contiguous():
        return t.data_ptr()
    _check(t, name, dtype, shape)
    raise ValueError(f"{name} is on device {t.get_device()}, the first argument on device {dev}")


def _rank(t, name: str, dtype, dims: int):
    """Shape of a tensor of `dims` dimensions (its other checks: `_in`)."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        _check(t, name, dtype)
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    return t.shape


def _out(t, name: str, dtype, shape, like: torch.Tensor, dev: int, stream) -> tuple:
    """An output and its address: the caller's, checked as `_in` does, or a new
    one from the memory pool of the stream that will write it."""
    if t is not None:
        return t, _in(t, name, dtype, shape, dev)
    if stream is None:
        t = like.new_empty(shape, dtype=dtype)
    else:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=like.device) if int(stream) else \
                torch.cuda.default_stream(like.device)
        with torch.cuda.stream(stream):
            t = like.new_empty(shape, dtype=dtype)
    return t, t.data_ptr()


# the current stream of a device as an address, without building a Stream object
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on(dev: int, f, *args):
    """f(*args) with device `dev` current (sizes and plans go by its compute units)."""
    if dev == torch.cuda.current_device():
        return f(*args)
    with torch.cuda.device(dev):
        return f(*args)


def _run(name: str, dev: int, stream, *args) -> None:
    """Calls a C entry point with device `dev` current, on `stream` or that
    device's current stream."""
    f = getattr(_lib_handle or _lib(), name)
    if stream is None:
        raw = _current_raw_stream(dev)
    elif isinstance(stream, torch.cuda.Stream) and stream.device.index != dev:
        raise ValueError(f"{name}: stream is on {stream.device}, the tensors on device {dev}")
    else:
        raw = _stream(stream)
    # (the usual case without a frame of its own: these calls last a few us)
    status = f(*args, raw) if dev == torch.cuda.current_device() else _on(dev, f, *args, raw)
    if status != 0:
        raise W4A16Error(status, name)


def w4a16_gemm_lora_workspace_bytes(M: int, N: int, K: int, L: int, R: int, split_k: int = 0,
                                    group_size: int = GROUP_SIZE) -> int:
    return int(_lib().w4a16_gemm_lora_workspace_bytes(M, N, K, group_size, L, R, split_k))


def w4a16_gemm_lora(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor, a: torch.Tensor,
                    b: torch.Tensor, adapter_ids: torch.Tensor, scaling: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None, split_k: int = 0,
                    workspace: Optional[torch.Tensor] = None, stream=None,
                    group_size: int = GROUP_SIZE) -> torch.Tensor:
    """w4a16_gemm with each row's own low-rank adapter added before the one
    rounding: Y[m] = X[m] . dequant(W)^T + scaling[l] (X[m] . A[l]^T) . B[l]^T,
    l = adapter_ids[m] (int32 [M]; outside [0, L): no adapter), a [L, R, K],
    b [L, N, R], scaling fp32 [L] or None (all 1)."""
    bf16 = torch.bfloat16
    M, K = _rank(x, "x", bf16, 2)
    N = _rank(w_packed, "w_packed", torch.uint8, 2)[0]
    L, R, _ = _rank(a, "a", bf16, 3)
    dev = x.get_device()
    px = _in(x, "x", bf16, (M, K), dev)
    pw = _in(w_packed, "w_packed", torch.uint8, (N, K // 2), dev)
    ps = _in(scales, "scales", bf16, (N, K // group_size), dev)
    pa = _in(a, "a", bf16, (L, R, K), dev)
    pb = _in(b, "b", bf16, (L, N, R), dev)
    pi = _in(adapter_ids, "adapter_ids", torch.int32, (M,), dev)
    pc = None if scaling is None else _in(scaling, "scaling", torch.float32, (L,), dev)
    y, py = _out(y, "y", bf16, (M, N), x, dev, stream)
    if workspace is None:
        nws = _on(dev, _lib().w4a16_gemm_lora_workspace_bytes, M, N, K, group_size, L, R, split_k) // 4
        workspace, pws = _out(None, "workspace", torch.float32, (nws,), x, dev, stream)
    else:
        pws = _in(workspace, "workspace", torch.float32, getattr(workspace, "shape", None), dev)
        nws = workspace.numel()
    _run("w4a16_gemm_lora", dev, stream, px, pw, ps, pa, pb, pi, pc, py, M, N, K, group_size, L, R, split_k, pws,
         nws * 4)
    return y


def w4a16_expert_sort_workspace_bytes(T: int, k: int, G: int) -> int:
    return int(_lib().w4a16_expert_sort_workspace_bytes(T, k, G))


def w4a16_expert_sort(ids: torch.Tensor, G: int, order: Optional[torch.Tensor] = None,
                      pos: Optional[torch.Tensor] = None, m_sizes: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """Slots of ids [T, k] (int32; outside [0, G): dropped) in expert order:
    (order [T k], pos [T, k], m_sizes [G]), all int32. m_sizes is the argument
    of w4a16_gemm_grouped, pos that of the gather and combine calls."""
    i32 = torch.int32
    T, k = _rank(ids, "ids", i32, 2)
    dev = ids.get_device()
    pi = _in(ids, "ids", i32, (T, k), dev)
    order, po = _out(order, "order", i32, (T * k,), ids, dev, stream)
    pos, pp = _out(pos, "pos", i32, (T, k), ids, dev, stream)
    m_sizes, pm = _out(m_sizes, "m_sizes", i32, (G,), ids, dev, stream)
    pws = None
    if workspace is None:
        nws = _lib().w4a16_expert_sort_workspace_bytes(T, k, G) // 4
        if nws > 0:
            workspace, pws = _out(None, "workspace", i32, (nws,), ids, dev, stream)
    else:
        pws = _in(workspace, "workspace", i32, getattr(workspace, "shape", None), dev)
        nws = workspace.numel()
    _run("w4a16_expert_sort", dev, stream, pi, po, pp, pm, T, k, G, pws, nws * 4)
    return order, pos, m_sizes


def w4a16_expert_gather(x: torch.Tensor, pos: torch.Tensor, xs: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """xs[pos[t, j]] = x[t] (rows that no slot names are left as they were)."""
    bf16 = torch.bfloat16
    T, k = _rank(pos, "pos", torch.int32, 2)
    width = _rank(x, "x", bf16, 2)[1]
    dev = x.get_device()
    px = _in(x, "x", bf16, (T, width), dev)
    pp = _in(pos, "pos", torch.int32, (T, k), dev)
    rows = T * k if xs is None else _rank(xs, "xs", bf16, 2)[0]
    xs, pxs = _out(xs, "xs", bf16, (rows, width), x, dev, stream)
    _run("w4a16_expert_gather", dev, stream, px, pp, pxs, T, k, rows, width)
    return xs


def w4a16_expert_gather_grad(dxs: torch.Tensor, pos: torch.Tensor, dx: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """dx[t] = sum_j dxs[pos[t, j]]: the gradient of w4a16_expert_gather."""
    bf16 = torch.bfloat16
    T, k = _rank(pos, "pos", torch.int32, 2)
    rows, width = _rank(dxs, "dxs", bf16, 2)
    dev = dxs.get_device()
    pd = _in(dxs, "dxs", bf16, (rows, width), dev)
    pp = _in(pos, "pos", torch.int32, (T, k), dev)
    dx, pdx = _out(dx, "dx", bf16, (T, width), dxs, dev, stream)
    _run("w4a16_expert_gather_grad", dev, stream, pd, pp, pdx, T, k, rows, width)
    return dx


def w4a16_expert_combine(z: torch.Tensor, pos: torch.Tensor, weights: Optional[torch.Tensor] = None,
                         y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] z[pos[t, j]] (weights fp32 [T, k], or None: all 1)."""
    bf16 = torch.bfloat16
    T, k = _rank(pos, "pos", torch.int32, 2)
    rows, width = _rank(z, "z", bf16, 2)
    dev = z.get_device()
    pz = _in(z, "z", bf16, (rows, width), dev)
    pp = _in(pos, "pos", torch.int32, (T, k), dev)
    pw = None if weights is None else _in(weights, "weights", torch.float32, (T, k), dev)
    y, py = _out(y, "y", bf16, (T, width), z, dev, stream)
    _run("w4a16_expert_combine", dev, stream, pz, pp, pw, py, T, k, rows, width)
    return y


def w4a16_expert_combine_grad(dy: torch.Tensor, z: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor,
                              dz: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None,
                              stream=None) -> tuple:
    """Gradients of w4a16_expert_combine: (dz, dweights). Rows of dz that no
    slot names are left as they were."""
    bf16, f32 = torch.bfloat16, torch.float32
    T, k = _rank(pos, "pos", torch.int32, 2)
    rows, width = _rank(z, "z", bf16, 2)
    dev = dy.get_device() if isinstance(dy, torch.Tensor) else -1
    pd = _in(dy, "dy", bf16, (T, width), dev)
    pz = _in(z, "z", bf16, (rows, width), dev)
    pp = _in(pos, "pos", torch.int32, (T, k), dev)
    pw = _in(weights, "weights", f32, (T, k), dev)
    dz, pdz = _out(dz, "dz", bf16, (rows, width), z, dev, stream)
    dweights, pdw = _out(dweights, "dweights", f32, (T, k), z, dev, stream)
    _run("w4a16_expert_combine_grad", dev, stream, pd, pz, pp, pw, pdz, pdw, T, k, rows, width)
    return dz, dweights


# ------------------------------------------------------------------ 8-bit products, input gradients

_E4M3 = torch.float8_e4m3fn


def _given_workspace(workspace, dtype, need: int, like: torch.Tensor, dev: int, stream) -> tuple:
    """(address, bytes) of the caller's workspace or a new one of `need` bytes, and the tensor."""
    if workspace is not None:
        p = _in(workspace, "workspace", dtype, getattr(workspace, "shape", None), dev)
        return workspace, p, workspace.numel() * workspace.element_size()
    if need == 0:
        return None, None, 0
    workspace, p = _out(None, "workspace", dtype, (-(-need // dtype.itemsize),), like, dev, stream)
    return workspace, p, need


def w4a16_fp8_quantize(x: torch.Tensor, q: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                       block_rows: int = 1, stream=None) -> tuple:
    """x [M, K] bf16 -> (q [M, K] e4m3, scales [ceil(M / block_rows), K / 128]
    fp32) in blocks of block_rows (1 or 128) x 128."""
    M, K = _rank(x, "x", torch.bfloat16, 2)
    dev = x.get_device()
    px = _in(x, "x", torch.bfloat16, (M, K), dev)
    q, pq = _out(q, "q", _E4M3, (M, K), x, dev, stream)
    scales, ps = _out(scales, "scales", torch.float32, (-(-M // max(block_rows, 1)), K // 128), x, dev, stream)
    _run("w4a16_fp8_quantize", dev, stream, px, pq, ps, M, K, block_rows)
    return q, scales


@functools.lru_cache(maxsize=4096)
def _bytes_of(name: str, dev: int, *args) -> int:
    """A workspace size, which depends on the sizes and the device's compute
    units only: kept, since asking takes a good part of a short call."""
    return int(_on(dev, getattr(_lib_handle or _lib(), name), *args))


def w4a16_fp8_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib().w4a16_fp8_gemm_workspace_bytes(M, N, K))


def w4a16_fp8_gemm_grad_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib().w4a16_fp8_gemm_grad_workspace_bytes(M, N, K))


def _fp8(name: str, grad: bool, x, x_scales, w, w_scales, m_sizes, y, workspace, stream, tile) -> torch.Tensor:
    """The three calls on e4m3 operands; `tile`: (rows per tile, split of the
    contraction), forced (internal entry point), or None."""
    f32 = torch.float32
    nx, ny = ("dy", "dx") if grad else ("x", "y")
    M, C = _rank(x, nx, _E4M3, 2)
    if m_sizes is None:
        G, (N, K) = 1, _rank(w, "w", _E4M3, 2)
        lead = ()
    else:
        G, N, K = _rank(w, "w", _E4M3, 3)
        lead = (G,)
    inner, outer = (N, K) if grad else (K, N)
    dev = x.get_device()
    px = _in(x, nx, _E4M3, (M, inner), dev)
    pxs = _in(x_scales, nx + "_scales", f32, (M, inner // 128), dev)
    pw = _in(w, "w", _E4M3, (*lead, N, K), dev)
    pws = _in(w_scales, "w_scales", f32, (*lead, -(-N // 128), K // 128), dev)
    pm = None if m_sizes is None else _in(m_sizes, "m_sizes", torch.int32, (G,), dev)
    y, py = _out(y, ny, torch.bfloat16, (M, outer), x, dev, stream)
    if tile is not None:
        need = 0 if pm else _bytes_of("w4a16_fp8_gemm_workspace_bytes_ex", dev, int(grad), M, N, K, *tile)
        workspace, pk, nk = _given_workspace(workspace, f32, need, x, dev, stream)
        _run("w4a16_fp8_gemm_ex", dev, stream, int(grad), px, pxs, pw, pws, pm, py, G, M, N, K, *tile, pk, nk)
    elif grad:
        need = 0 if pm else _bytes_of("w4a16_fp8_gemm_grad_workspace_bytes", dev, M, N, K)
        workspace, pk, nk = _given_workspace(workspace, f32, need, x, dev, stream)
        _run(name, dev, stream, px, pxs, pw, pws, pm, py, G, M, N, K, pk, nk)
    elif pm is None:
        need = _bytes_of("w4a16_fp8_gemm_workspace_bytes", dev, M, N, K)
        workspace, pk, nk = _given_workspace(workspace, f32, need, x, dev, stream)
        _run(name, dev, stream, px, pxs, pw, pws, py, M, N, K, pk, nk)
    else:
        _run(name, dev, stream, px, pxs, pw, pws, pm, py, G, M, N, K)
    return y


def w4a16_fp8_gemm(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                   y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
                   tile=None) -> torch.Tensor:
    """Y [M, N] bf16 = (x x_scales) . (w w_scales)^T: x [M, K] e4m3 with scales
    [M, K / 128], w [N, K] e4m3 with scales [ceil(N / 128), K / 128] (fp32)."""
    return _fp8("w4a16_fp8_gemm", False, x, x_scales, w, w_scales, None, y, workspace, stream, tile)


def w4a16_fp8_gemm_grouped(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                           m_sizes: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None,
                           tile=None) -> torch.Tensor:
    """w4a16_fp8_gemm for rows grouped by expert (w [G, N, K]); m_sizes [G]
    int32 stays on the device. Rows past the last expert's are left as they were."""
    return _fp8("w4a16_fp8_gemm_grouped", False, x, x_scales, w, w_scales, _sizes(m_sizes), y, None, stream, tile)


def w4a16_fp8_gemm_grad(dy: torch.Tensor, dy_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                        m_sizes: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None, tile=None) -> torch.Tensor:
    """dX [M, K] bf16 of w4a16_fp8_gemm (with m_sizes: of _grouped) from dy
    [M, N] e4m3 with scales [M, N / 128]; N a multiple of 128."""
    return _fp8("w4a16_fp8_gemm_grad", True, dy, dy_scales, w, w_scales, m_sizes, dx, workspace, stream, tile)


def _sizes(m_sizes):
    if m_sizes is None:
        raise TypeError("m_sizes must be a torch.Tensor")
    return m_sizes


def w4a16_gemm_grad_workspace_bytes(G: int, M: int, N: int, K: int, group_size: int = GROUP_SIZE) -> int:
    return int(_lib().w4a16_gemm_grad_workspace_bytes(G, M, N, K, group_size))


def w4a16_gemm_grad(dy: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor,
                    m_sizes: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None, group_size: int = GROUP_SIZE,
                    tile=None) -> torch.Tensor:
    """dX [M, K] = dY [M, N] . dequant(W): the gradient of w4a16_gemm with
    respect to x (with m_sizes and w_packed [G, N, K / 2]: of
    w4a16_gemm_grouped). N a multiple of 8; workspace uint8."""
    bf16, u8 = torch.bfloat16, torch.uint8
    M, N = _rank(dy, "dy", bf16, 2)
    shape = _rank(w_packed, "w_packed", u8, 2 if m_sizes is None else 3)
    lead, K = tuple(shape[:-2]), 2 * shape[-1]
    G = lead[0] if lead else 1
    dev = dy.get_device()
    pd = _in(dy, "dy", bf16, (M, N), dev)
    pw = _in(w_packed, "w_packed", u8, (*lead, N, K // 2), dev)
    ps = _in(scales, "scales", bf16, (*lead, N, K // group_size), dev)
    pm = None if m_sizes is None else _in(m_sizes, "m_sizes", torch.int32, (G,), dev)
    dx, px = _out(dx, "dx", bf16, (M, K), dy, dev, stream)
    if tile is None:
        need = _bytes_of("w4a16_gemm_grad_workspace_bytes", dev, G, M, N, K, group_size)
        workspace, pk, nk = _given_workspace(workspace, u8, need, dy, dev, stream)
        _run("w4a16_gemm_grad", dev, stream, pd, pw, ps, pm, px, G, M, N, K, group_size, pk, nk)
    else:
        need = _bytes_of("w4a16_gemm_grad_workspace_bytes_ex", dev, G, M, N, K, group_size, *tile)
        workspace, pk, nk = _given_workspace(workspace, u8, need, dy, dev, stream)
        _run("w4a16_gemm_grad_ex", dev, stream, pd, pw, ps, pm, px, G, M, N, K, group_size, *tile, pk, nk)
    return dx
