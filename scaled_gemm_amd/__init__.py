"""Python binding of libptpc, the PTPC-FP8 hot path for MI355X (gfx950).

Argument marshalling only: every step runs in the HIP kernels of
``libptpc.so`` behind the C ABI declared in ``include/ptpc.h``.  PyTorch
provides device memory and the current stream; nothing here computes.  If
the library has not been built, every call raises -- there is no fallback.

Tensors: bf16 inputs as ``torch.bfloat16``; E4M3 codes as ``torch.uint8``
(view as ``torch.float8_e4m3fn`` if wanted); scales ``torch.float32``.
"""
import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass

import torch  # must load before libptpc so both share torch's HIP runtime

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libptpc.so")

_STATUS = {
    0: "PTPC_OK", 1: "PTPC_ERR_NULL", 2: "PTPC_ERR_SHAPE", 3: "PTPC_ERR_UNSUPPORTED",
    4: "PTPC_ERR_ALIGN", 5: "PTPC_ERR_HIP",
}

# Every symbol include/ptpc.h declares.
EXPORTS = (
    "ptpc_status_string", "ptpc_abi_version", "ptpc_quant_act", "ptpc_weight_packed_bytes",
    "ptpc_quant_weight", "ptpc_unpack_weight", "ptpc_gemm",
    "ptpc_gemm_workspace_bytes", "ptpc_gemm_ws", "ptpc_gemm_noalloc",
    "ptpc_gemm_unfused_workspace_bytes", "ptpc_gemm_unfused",
    "ptpc_gemm_unfused_bf16_workspace_bytes", "ptpc_gemm_unfused_bf16", "ptpc_tensor_scale",
    "ptpc_quant_act_static", "ptpc_quant_weight_static", "ptpc_gemm_tensor",
    "ptpc_gemm_kernel", "ptpc_quant_act_kernel", "ptpc_gemm_ws_splits",
    "ptpc_rope_append", "ptpc_attn_paged_workspace_bytes", "ptpc_attn_paged", "ptpc_attn_prompt",
    "ptpc_quant_act_block", "ptpc_quant_weight_block", "ptpc_pack_weight_block", "ptpc_gemm_block",
    "ptpc_route_experts_workspace_bytes", "ptpc_route_experts", "ptpc_gemm_experts",
    "ptpc_combine_experts", "ptpc_gemm_block_kernel",
)

_lib = None


class _CacheStruct(ctypes.Structure):
    """ptpc_kv_cache of include/ptpc.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dk", ctypes.c_void_p),
                ("dv", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("fp8", ctypes.c_int32)]


class PtpcError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)}")


def lib():
    """The loaded libptpc.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m scaled_gemm_amd.build` (no fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        L.ptpc_status_string.restype = ctypes.c_char_p
        L.ptpc_status_string.argtypes = [ctypes.c_int]
        L.ptpc_abi_version.restype = ctypes.c_int
        L.ptpc_abi_version.argtypes = []
        L.ptpc_quant_act.restype = ctypes.c_int
        L.ptpc_quant_act.argtypes = [P, I, I, I, P, I, P, P]
        L.ptpc_weight_packed_bytes.restype = S
        L.ptpc_weight_packed_bytes.argtypes = [I, I]
        L.ptpc_quant_weight.restype = ctypes.c_int
        L.ptpc_quant_weight.argtypes = [P, I, I, I, P, P, P]
        L.ptpc_unpack_weight.restype = ctypes.c_int
        L.ptpc_unpack_weight.argtypes = [P, I, I, P, P]
        L.ptpc_gemm.restype = ctypes.c_int
        L.ptpc_gemm.argtypes = [P, I, P, P, P, I, I, I, P, I, P]
        L.ptpc_gemm_unfused_workspace_bytes.restype = S
        L.ptpc_gemm_unfused_workspace_bytes.argtypes = [I, I]
        L.ptpc_gemm_unfused.restype = ctypes.c_int
        L.ptpc_gemm_unfused.argtypes = [P, I, P, P, P, I, I, I, P, I, P, P]
        L.ptpc_gemm_workspace_bytes.restype = S
        L.ptpc_gemm_workspace_bytes.argtypes = [I, I, I]
        L.ptpc_gemm_ws.restype = ctypes.c_int
        L.ptpc_gemm_ws.argtypes = [P, I, P, P, P, I, I, I, P, I, P, S, P]
        L.ptpc_gemm_noalloc.restype = ctypes.c_int
        L.ptpc_gemm_noalloc.argtypes = [P, I, P, P, P, I, I, I, P, I, P]
        L.ptpc_gemm_unfused_bf16_workspace_bytes.restype = S
        L.ptpc_gemm_unfused_bf16_workspace_bytes.argtypes = [I, I]
        L.ptpc_gemm_unfused_bf16.restype = ctypes.c_int
        L.ptpc_gemm_unfused_bf16.argtypes = [P, I, P, P, P, I, I, I, P, I, P, P]
        L.ptpc_tensor_scale.restype = ctypes.c_int
        L.ptpc_tensor_scale.argtypes = [P, I, I, I, P, P]
        L.ptpc_quant_act_static.restype = ctypes.c_int
        L.ptpc_quant_act_static.argtypes = [P, I, I, I, P, P, I, P]
        L.ptpc_quant_weight_static.restype = ctypes.c_int
        L.ptpc_quant_weight_static.argtypes = [P, I, I, I, P, P, P]
        L.ptpc_gemm_tensor.restype = ctypes.c_int
        L.ptpc_gemm_tensor.argtypes = [P, I, P, P, P, I, I, I, P, I, P]
        L.ptpc_gemm_kernel.restype = ctypes.c_char_p
        L.ptpc_gemm_kernel.argtypes = [I, I, I]
        L.ptpc_quant_act_kernel.restype = ctypes.c_char_p
        L.ptpc_quant_act_kernel.argtypes = [I, I]
        L.ptpc_gemm_ws_splits.restype = ctypes.c_int
        L.ptpc_gemm_ws_splits.argtypes = [I, I, I]
        F, J, C = ctypes.c_float, ctypes.c_int, ctypes.POINTER(_CacheStruct)
        L.ptpc_rope_append.restype = ctypes.c_int
        L.ptpc_rope_append.argtypes = [P, I, P, I, P, I, P, I, I, J, P, P, I, I, C, P, I, P]
        L.ptpc_attn_paged_workspace_bytes.restype = S
        L.ptpc_attn_paged_workspace_bytes.argtypes = [I, I, I, I, I, C]
        L.ptpc_attn_paged.restype = ctypes.c_int
        L.ptpc_attn_paged.argtypes = [P, I, P, C, P, I, I, P, I, I, I, I, I, F, P, I, P, S, P]
        L.ptpc_attn_prompt.restype = ctypes.c_int
        L.ptpc_attn_prompt.argtypes = [P, I, P, I, P, I, P, I, I, I, I, I, F, P, I, P]
        L.ptpc_quant_act_block.restype = ctypes.c_int
        L.ptpc_quant_act_block.argtypes = [P, I, I, I, J, P, P, I, P, I, P]
        L.ptpc_quant_weight_block.restype = ctypes.c_int
        L.ptpc_quant_weight_block.argtypes = [P, I, I, I, I, I, P, P, P]
        L.ptpc_pack_weight_block.restype = ctypes.c_int
        L.ptpc_pack_weight_block.argtypes = [P, I, I, I, P, I, I, I, I, I, I, P, P, P]
        L.ptpc_gemm_block.restype = ctypes.c_int
        L.ptpc_gemm_block.argtypes = [P, I, P, I, P, P, I, I, I, P, I, P]
        L.ptpc_route_experts_workspace_bytes.restype = S
        L.ptpc_route_experts_workspace_bytes.argtypes = [I, I]
        L.ptpc_route_experts.restype = ctypes.c_int
        L.ptpc_route_experts.argtypes = [P, J, I, P, I, I, I, J, I, I, I, J, F, I, I, P, P, P, P, P,
                                         P, S, P]
        L.ptpc_gemm_experts.restype = ctypes.c_int
        L.ptpc_gemm_experts.argtypes = [P, I, P, I, P, P, P, P, I, I, I, I, I, I, P, I, P]
        L.ptpc_combine_experts.restype = ctypes.c_int
        L.ptpc_combine_experts.argtypes = [P, I, I, P, P, I, I, I, P, I, P]
        L.ptpc_gemm_block_kernel.restype = ctypes.c_char_p
        L.ptpc_gemm_block_kernel.argtypes = [I, I, I, I]
        _lib = L
    return _lib


def _stream(dev, stream):
    """Handle of the stream a call runs on: the current one of GPU dev, unless one is given."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream: expected a stream of GPU {dev}, got one of GPU "
                         f"{stream.device_index}")
    return stream.cuda_stream


def _call(fn, dev, *args):
    """One call of the library with GPU dev current: a launch takes its kernels, and the null
    stream, from the current device."""
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status != 0:
        raise PtpcError(fn.__name__, status)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() > 0 else None


# Every tensor handed to the library is checked here before the call: the
# kernels trust the extents they are given, so a buffer that is too small or
# not on the GPU would be read or written out of bounds on the device.
def _on_gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a tensor on the GPU, got one on {t.device}")


def _matrix(t, dtype, name, shape=None):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2 or (t.numel() > 0 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a 2-D tensor with unit column stride")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    _on_gpu(t, name)
    return t.shape[0], t.shape[1], max(t.stride(0), t.shape[1])


def _vector(t, n, dtype, name, exact=True):
    """A contiguous 1-D buffer of n (exact) or at least n elements."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous 1-D tensor")
    if (t.numel() != n) if exact else (t.numel() < n):
        want = f"{n}" if exact else f"at least {n}"
        raise ValueError(f"{name}: expected {want} elements, got {t.numel()}")
    _on_gpu(t, name)


def _scratch(t, nbytes, name):
    """A contiguous buffer of at least nbytes bytes, any dtype."""
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name}: expected at least {nbytes} bytes, got "
                         f"{t.numel() * t.element_size()}")
    _on_gpu(t, name)


def packed_bytes(Ci: int, Co: int) -> int:
    return int(lib().ptpc_weight_packed_bytes(Ci, Co))


def workspace_bytes(T: int, Co: int) -> int:
    return int(lib().ptpc_gemm_unfused_workspace_bytes(T, Co))


@dataclass
class PackedWeight:
    """A weight quantized once: packed E4M3 codes plus its scales -- one per
    output column (per-channel, from quant_weight) or, with per_tensor set,
    one for the whole matrix (from quant_weight_static)."""
    data: torch.Tensor     # uint8 [packed_bytes(Ci, Co)]
    dw: torch.Tensor       # float32 [Co], or [1] when per_tensor
    Ci: int
    Co: int
    per_tensor: bool = False


def _check_packed(pw: PackedWeight, name, per_tensor):
    if pw.per_tensor != per_tensor:
        kind = "per-tensor" if pw.per_tensor else "per-channel"
        raise ValueError(f"{name}: got a {kind} weight; this call needs "
                         f"{'a per-tensor' if per_tensor else 'a per-channel'} one")
    _vector(pw.data, packed_bytes(pw.Ci, pw.Co), torch.uint8, f"{name}.data", exact=False)
    _vector(pw.dw, 1 if per_tensor else pw.Co, torch.float32, f"{name}.dw")


def gemm_kernel(T: int, Ci: int, Co: int):
    """Name of the GEMM kernel ptpc_gemm launches for this shape (None if none)."""
    r = lib().ptpc_gemm_kernel(T, Ci, Co)
    return r.decode() if r is not None else None


def gemm_ws_splits(T: int, Ci: int, Co: int) -> int:
    """K ranges ptpc_gemm_ws / ptpc_gemm_noalloc use for this shape (1: no split)."""
    return int(lib().ptpc_gemm_ws_splits(T, Ci, Co))


def quant_act_kernel(T: int, Ci: int):
    """Name of the kernel ptpc_quant_act launches for T rows of Ci elements."""
    r = lib().ptpc_quant_act_kernel(T, Ci)
    return r.decode() if r is not None else None


def quant_act(x, qx=None, dx=None, stream=None):
    """Per-token FP8 quantization of bf16 X [T, Ci] -> (codes uint8 [T, Ci], dx fp32 [T])."""
    T, Ci, ldx = _matrix(x, torch.bfloat16, "x")
    if qx is None:
        qx = torch.empty((T, Ci), dtype=torch.uint8, device=x.device)
    if dx is None:
        dx = torch.empty((T,), dtype=torch.float32, device=x.device)
    _, _, ldq = _matrix(qx, torch.uint8, "qx", (T, Ci))
    _vector(dx, T, torch.float32, "dx")
    dev = x.get_device()
    _call(lib().ptpc_quant_act, dev, _ptr(x), T, Ci, ldx, _ptr(qx), ldq, _ptr(dx),
          _stream(dev, stream))
    return qx, dx


def quant_weight(w, out: PackedWeight = None, stream=None) -> PackedWeight:
    """Per-output-channel FP8 quantization + MFMA prepack of bf16 W [Ci, Co]."""
    Ci, Co, ldw = _matrix(w, torch.bfloat16, "w")
    if out is None:
        out = PackedWeight(torch.empty((packed_bytes(Ci, Co),), dtype=torch.uint8, device=w.device),
                           torch.empty((Co,), dtype=torch.float32, device=w.device), Ci, Co)
    if (out.Ci, out.Co) != (Ci, Co):
        raise ValueError(f"out: PackedWeight is {out.Ci}x{out.Co}, w is {Ci}x{Co}")
    _check_packed(out, "out", per_tensor=False)
    dev = w.get_device()
    _call(lib().ptpc_quant_weight, dev, _ptr(w), Ci, Co, ldw, _ptr(out.data), _ptr(out.dw),
          _stream(dev, stream))
    return out


def unpack_weight(pw: PackedWeight, stream=None):
    """E4M3 codes of the weight back in [Ci, Co] order (for tests)."""
    _vector(pw.data, packed_bytes(pw.Ci, pw.Co), torch.uint8, "pw.data", exact=False)
    qw = torch.empty((pw.Ci, pw.Co), dtype=torch.uint8, device=pw.data.device)
    dev = pw.data.get_device()
    _call(lib().ptpc_unpack_weight, dev, _ptr(pw.data), pw.Ci, pw.Co, _ptr(qw),
          _stream(dev, stream))
    return qw


def _gemm_args(qx, dx, pw: PackedWeight, out, per_tensor):
    T, Ci, ldq = _matrix(qx, torch.uint8, "qx")
    if Ci != pw.Ci:
        raise ValueError(f"qx has Ci={Ci}, weight has Ci={pw.Ci}")
    _check_packed(pw, "pw", per_tensor)
    if per_tensor:
        _vector(dx, 1, torch.float32, "dx")
    else:
        _vector(dx, T, torch.float32, "dx")
    if out is None:
        out = torch.empty((T, pw.Co), dtype=torch.bfloat16, device=qx.device)
    _matrix(out, torch.bfloat16, "out", (T, pw.Co))
    return T, Ci, ldq, out


def gemm(qx, dx, pw: PackedWeight, out=None, stream=None):
    """Fused PTPC GEMM: bf16 [T, Co] = ((qx @ qw) * dx[:, None]) * dw[None, :]."""
    T, Ci, ldq, out = _gemm_args(qx, dx, pw, out, per_tensor=False)
    ldo = max(out.stride(0), out.shape[1])
    dev = qx.get_device()
    _call(lib().ptpc_gemm, dev, _ptr(qx), ldq, _ptr(dx), _ptr(pw.data), _ptr(pw.dw), T, Ci, pw.Co,
          _ptr(out), ldo, _stream(dev, stream))
    return out


def gemm_workspace_bytes(T: int, Ci: int, Co: int) -> int:
    return int(lib().ptpc_gemm_workspace_bytes(T, Ci, Co))


def gemm_ws(qx, dx, pw: PackedWeight, out=None, workspace=None, stream=None):
    """ptpc_gemm_ws: the fused GEMM, splitting K across workgroups where the
    output tiles alone leave the GPU idle (workspace: uint8 tensor of at least
    gemm_workspace_bytes(T, Ci, Co) bytes; allocated here if not given)."""
    T, Ci, ldq, out = _gemm_args(qx, dx, pw, out, per_tensor=False)
    need = gemm_workspace_bytes(T, Ci, pw.Co)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=qx.device)
    if workspace is not None:
        _scratch(workspace, need, "workspace")
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    ldo = max(out.stride(0), out.shape[1])
    dev = qx.get_device()
    _call(lib().ptpc_gemm_ws, dev, _ptr(qx), ldq, _ptr(dx), _ptr(pw.data), _ptr(pw.dw), T, Ci,
          pw.Co, _ptr(out), ldo, _ptr(workspace), nbytes, _stream(dev, stream))
    return out


# Scratch bytes the library holds per GPU for gemm_noalloc (include/ptpc.h).
NOALLOC_SCRATCH_BYTES = 64 << 20


def gemm_noalloc(qx, dx, pw: PackedWeight, out=None, stream=None):
    """ptpc_gemm_noalloc: gemm_ws without a workspace -- the split-K partials
    go to the library's own per-GPU scratch, nothing is allocated (pass `out`
    to allocate nothing here either).  Calls overlapping on one GPU race."""
    T, Ci, ldq, out = _gemm_args(qx, dx, pw, out, per_tensor=False)
    ldo = max(out.stride(0), out.shape[1])
    dev = qx.get_device()
    _call(lib().ptpc_gemm_noalloc, dev, _ptr(qx), ldq, _ptr(dx), _ptr(pw.data), _ptr(pw.dw), T, Ci,
          pw.Co, _ptr(out), ldo, _stream(dev, stream))
    return out


def gemm_unfused(qx, dx, pw: PackedWeight, out=None, workspace=None, stream=None):
    """Two-step form: fp32 GEMM result to `workspace`, then a rescale pass."""
    T, Ci, ldq, out = _gemm_args(qx, dx, pw, out, per_tensor=False)
    if workspace is None:
        workspace = torch.empty((T, pw.Co), dtype=torch.float32, device=qx.device)
    if workspace.dtype != torch.float32:
        raise TypeError(f"workspace: expected torch.float32, got {workspace.dtype}")
    _scratch(workspace, workspace_bytes(T, pw.Co), "workspace")
    ldo = max(out.stride(0), out.shape[1])
    dev = qx.get_device()
    _call(lib().ptpc_gemm_unfused, dev, _ptr(qx), ldq, _ptr(dx), _ptr(pw.data), _ptr(pw.dw), T, Ci,
          pw.Co, _ptr(out), ldo, _ptr(workspace), _stream(dev, stream))
    return out


def gemm_unfused_bf16(qx, dx, pw: PackedWeight, out=None, workspace=None, stream=None):
    """Two-step form with a bf16 intermediate: bf16(acc) to `workspace`, then scaled."""
    T, Ci, ldq, out = _gemm_args(qx, dx, pw, out, per_tensor=False)
    if workspace is None:
        workspace = torch.empty((T, pw.Co), dtype=torch.bfloat16, device=qx.device)
    if workspace.dtype != torch.bfloat16:
        raise TypeError(f"workspace: expected torch.bfloat16, got {workspace.dtype}")
    _scratch(workspace, 2 * T * pw.Co, "workspace")
    ldo = max(out.stride(0), out.shape[1])
    dev = qx.get_device()
    _call(lib().ptpc_gemm_unfused_bf16, dev, _ptr(qx), ldq, _ptr(dx), _ptr(pw.data), _ptr(pw.dw), T,
          Ci, pw.Co, _ptr(out), ldo, _ptr(workspace), _stream(dev, stream))
    return out


def linear(x, pw: PackedWeight, stream=None):
    """Per-token quantization of X followed by the fused GEMM (one layer's forward)."""
    qx, dx = quant_act(x, stream=stream)
    return gemm(qx, dx, pw, stream=stream)


# -- per-tensor comparator ------------------------------------------------------
def tensor_scale(x, d=None, stream=None):
    """One scale for a whole bf16 matrix: d[0] = max|x| / 448 (1 if zero) -> fp32 [1]."""
    R, C, ld = _matrix(x, torch.bfloat16, "x")
    if d is None:
        d = torch.empty((1,), dtype=torch.float32, device=x.device)
    _vector(d, 1, torch.float32, "d")
    dev = x.get_device()
    _call(lib().ptpc_tensor_scale, dev, _ptr(x), R, C, ld, _ptr(d), _stream(dev, stream))
    return d


def quant_act_static(x, d, qx=None, stream=None):
    """Per-tensor FP8 codes of bf16 X [T, Ci] with the given scale d (fp32 [1])."""
    T, Ci, ldx = _matrix(x, torch.bfloat16, "x")
    if qx is None:
        qx = torch.empty((T, Ci), dtype=torch.uint8, device=x.device)
    _, _, ldq = _matrix(qx, torch.uint8, "qx", (T, Ci))
    _vector(d, 1, torch.float32, "d")
    dev = x.get_device()
    _call(lib().ptpc_quant_act_static, dev, _ptr(x), T, Ci, ldx, _ptr(d), _ptr(qx), ldq,
          _stream(dev, stream))
    return qx


def quant_weight_static(w, d, out: PackedWeight = None, stream=None) -> PackedWeight:
    """Per-tensor FP8 codes of bf16 W [Ci, Co] with the scale d (fp32 [1]), prepacked;
    the returned PackedWeight carries d as its (one-element) dw and is marked
    per_tensor (only gemm_tensor accepts it)."""
    Ci, Co, ldw = _matrix(w, torch.bfloat16, "w")
    _vector(d, 1, torch.float32, "d")
    if out is None:
        out = PackedWeight(torch.empty((packed_bytes(Ci, Co),), dtype=torch.uint8, device=w.device),
                           d, Ci, Co, per_tensor=True)
    if (out.Ci, out.Co) != (Ci, Co):
        raise ValueError(f"out: PackedWeight is {out.Ci}x{out.Co}, w is {Ci}x{Co}")
    _check_packed(out, "out", per_tensor=True)
    dev = w.get_device()
    _call(lib().ptpc_quant_weight_static, dev, _ptr(w), Ci, Co, ldw, _ptr(d), _ptr(out.data),
          _stream(dev, stream))
    return out


def gemm_tensor(qx, dx, pw: PackedWeight, out=None, stream=None):
    """Per-tensor FP8 GEMM: bf16 [T, Co] = ((qx @ qw) * dx[0]) * dw[0]."""
    T, Ci, ldq, out = _gemm_args(qx, dx, pw, out, per_tensor=True)
    ldo = max(out.stride(0), out.shape[1])
    dev = qx.get_device()
    _call(lib().ptpc_gemm_tensor, dev, _ptr(qx), ldq, _ptr(dx), _ptr(pw.data), _ptr(pw.dw), T, Ci,
          pw.Co, _ptr(out), ldo, _stream(dev, stream))
    return out


# -- attention of the decoder layer ---------------------------------------------
class KVCache:
    """A paged cache of keys and values: k, v [pages, kv_heads, page_size, head_dim],
    bf16, or uint8 E4M3 codes with fp32 scales dk, dv [pages, kv_heads, page_size].
    Token slot s is entry s % page_size of page s // page_size.  The tensors are the
    caller's; they are checked once, here, and cannot be exchanged afterwards."""
    __slots__ = ("_tensors", "_struct", "_pointer", "_extents", "_device", "_head_dim",
                 "_kv_heads", "_page_size")

    def __init__(self, k, v, dk=None, dv=None):
        fp8 = k.dtype == torch.uint8
        if not fp8 and k.dtype != torch.bfloat16:
            raise TypeError(f"k: expected torch.bfloat16 or torch.uint8, got {k.dtype}")
        if v.dtype != k.dtype:
            raise TypeError(f"v: expected {k.dtype}, got {v.dtype}")
        if k.dim() != 4:
            raise ValueError("k: expected [pages, kv_heads, page_size, head_dim]")
        if (dk is not None) != fp8 or (dv is not None) != fp8:
            raise ValueError("dk, dv: scales go with E4M3 codes (uint8), and only with them")
        want = [(v, "v", k.shape, k.dtype)]
        if fp8:
            want += [(dk, "dk", k.shape[:3], torch.float32), (dv, "dv", k.shape[:3], torch.float32)]
        for t, name, shape, dtype in [(k, "k", k.shape, k.dtype)] + want:
            if t.dtype != dtype:
                raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
            if t.shape != shape:
                raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous tensor")
            _on_gpu(t, name)
            if t.device != k.device:
                raise ValueError(f"{name}: expected a tensor on {k.device}, got one on {t.device}")
        self._tensors = (k, v, dk, dv)
        pages, heads, page, d = k.shape
        p = [t.data_ptr() if t is not None else None for t in self._tensors]
        self._struct = _CacheStruct(*p, pages, heads, page, d, int(fp8))

        self._pointer = ctypes.pointer(self._struct)
        self._extents = (pages, heads, page, d, int(fp8))
        self._device, self._head_dim, self._kv_heads, self._page_size = k.get_device(), d, heads, page

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    dk = property(lambda self: self._tensors[2])
    dv = property(lambda self: self._tensors[3])
    pages = property(lambda self: self._extents[0])
    kv_heads = property(lambda self: self._extents[1])
    page_size = property(lambda self: self._extents[2])
    head_dim = property(lambda self: self._extents[3])
    fp8 = property(lambda self: bool(self._extents[4]))


def kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, fp8: bool = False,
             device="cuda") -> KVCache:
    """A new cache, its entries unset until tokens are appended."""
    shape = (pages, kv_heads, page_size, head_dim)
    dtype = torch.uint8 if fp8 else torch.bfloat16
    k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
    dk, dv = (torch.empty(shape[:3], dtype=torch.float32, device=device) if fp8 else None
              for _ in range(2))
    return KVCache(k, v, dk, dv)


# The calls below are made once per layer and token, so their checks are written for few
# Python steps: what is right is seen in one or two comparisons, and the rest is sorted out
# afterwards, by _other_heads and _wrong_index.
_BF16, _I32, _I64, _F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
_U8 = torch.uint8


def _heads(t, name, dev, T, H, D):
    """Token pitch of a bf16 [T, H, D] tensor whose heads lie one after another."""
    if t.dtype is _BF16 and t.shape == (T, H, D) and t.get_device() == dev:
        s0, s1, s2 = t.stride()
        if s2 == 1 and s1 == D and s0 >= H * D and T > 1:
            return s0
    return _other_heads(t, name, dev, T, H, D)


def _other_heads(t, name, dev, T, H, D):
    if t.dtype is not _BF16:
        raise TypeError(f"{name}: expected {_BF16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name}: expected [tokens, heads, head_dim]")
    if tuple(t.shape) != (T, H, D):
        raise ValueError(f"{name}: expected shape {(T, H, D)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        _wrong_device(t, name, dev)
    s0, s1, s2 = t.stride()
    if (s2 != 1 or (s1 != D and H > 1) or (s0 < H * D and T > 1)) and T * H * D > 0:
        raise ValueError(f"{name}: expected a token's heads one after another and tokens apart")
    return s0 if T > 1 else H * D       # one token, one head or none: their strides say nothing


def _index(t, shape, dtype, name, dev):
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _wrong_index(t, shape, dtype, name, dev)


def _wrong_index(t, shape, dtype, name, dev):
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of shape {tuple(shape)}, got "
                         f"{tuple(t.shape)}")
    _wrong_device(t, name, dev)


def _wrong_device(t, name, dev):
    _on_gpu(t, name)
    raise ValueError(f"{name}: expected a tensor on GPU {dev}, got one on {t.device}")


def _three(t, name):
    """(tokens, heads, head_dim) of t."""
    if t.dim() != 3:
        raise ValueError(f"{name}: expected [tokens, heads, head_dim]")
    return t.shape


def _empty(like, shape, stream, dtype=None):
    """A new tensor that belongs to the stream it is used on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def rope_append(q, k, v, table, positions, slots, cache: KVCache, q_out=None,
                interleaved: bool = False, stream=None):
    """Rotate new tokens' queries and keys by their positions and append keys and values.

    q [T, q_heads, D], k, v [T, kv_heads, D] bf16 (slices of the QKV projection's output are
    fine); table fp32 [n_pos, rot_dim], cosines then sines; positions int32 [T]; slots int64
    [T], -1 for a token that is not stored.  Returns the rotated q (q_out; q itself rotates in
    place)."""
    dev, D, Hk = cache._device, cache._head_dim, cache._kv_heads
    T, Hq, _ = _three(q, "q")
    ldq = _heads(q, "q", dev, T, Hq, D)
    ldk, ldv = _heads(k, "k", dev, T, Hk, D), _heads(v, "v", dev, T, Hk, D)
    if table.dim() != 2:
        raise ValueError("table: expected [positions, rot_dim]")
    n_pos, rot = shape = table.shape
    _index(table, shape, _F32, "table", dev)
    _index(positions, (T,), _I32, "positions", dev)
    _index(slots, (T,), _I64, "slots", dev)
    if q_out is None:
        q_out = _empty(q, (T, Hq, D), stream)
        ldqo = Hq * D
    else:
        ldqo = _heads(q_out, "q_out", dev, T, Hq, D)
    _call(lib().ptpc_rope_append, dev, q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
          table.data_ptr(), n_pos, rot, int(interleaved), positions.data_ptr(), slots.data_ptr(), T,
          Hq, cache._pointer, q_out.data_ptr(), ldqo, _stream(dev, stream))
    return q_out


@functools.lru_cache(maxsize=4096)
def _paged_workspace(T, B, max_q, max_kv, q_heads, pages, kv_heads, page_size, head_dim, fp8):
    c = _CacheStruct(None, None, None, None, pages, kv_heads, page_size, head_dim, fp8)
    return int(lib().ptpc_attn_paged_workspace_bytes(T, B, max_q, max_kv, q_heads, c))


def attn_paged_workspace_bytes(T: int, B: int, max_q: int, max_kv: int, q_heads: int,
                               cache: KVCache) -> int:
    return _paged_workspace(T, B, max_q, max_kv, q_heads, *cache._extents)


def attn_paged(q, cu_q, cache: KVCache, page_table, kv_lens, max_q=None, max_kv=None, scale=None,
               out=None, workspace=None, stream=None):
    """Attention of new tokens over the paged cache: bf16 [T, q_heads, D].

    q [T, q_heads, D] bf16, sequence b's rows cu_q[b]:cu_q[b+1] (int32 [B+1]), the last of its
    kv_lens[b] cached tokens (int32 [B]); page_table int32 [B, pages per sequence].  max_q and
    max_kv bound the new tokens and cached tokens of a sequence and choose the kernel; scale
    defaults to D ** -0.5; workspace: uint8, attn_paged_workspace_bytes.

    The default bounds are the only safe ones, T and what the table holds: pass max_q=1 for a
    decode batch, which is laid out for sequences of up to T tokens without it (128 sequences of
    2048 E4M3 keys, 64 heads on 8: 101 us with it, 318 us without).  A bound that is too small
    costs far more (one sequence of 128 tokens under max_q=1: 9 ms instead of 0.2)."""
    dev, D = cache._device, cache._head_dim
    T, Hq, _ = _three(q, "q")
    ldq = _heads(q, "q", dev, T, Hq, D)
    if kv_lens.dim() != 1:
        raise ValueError("kv_lens: expected one length per sequence")
    B = kv_lens.shape[0]
    _index(kv_lens, (B,), _I32, "kv_lens", dev)
    _index(cu_q, (B + 1,), _I32, "cu_q", dev)
    if B == 0 and T > 0:
        raise ValueError("cu_q: the rows of q belong to no sequence")
    if page_table.dtype is not _I32:
        raise TypeError(f"page_table: expected {_I32}, got {page_table.dtype}")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table: expected {B} rows, got shape {tuple(page_table.shape)}")
    width = page_table.shape[1]
    ldt, step = page_table.stride()
    if B < 2 or width == 0:
        ldt = width
    if (step != 1 and B * width > 0 and width > 1) or ldt < width:
        raise ValueError("page_table: expected rows apart, with unit column stride")
    if page_table.get_device() != dev:
        _wrong_device(page_table, "page_table", dev)
    if out is None:
        out = _empty(q, (T, Hq, D), stream)
        ldo = Hq * D
    else:
        ldo = _heads(out, "out", dev, T, Hq, D)
    if max_q is None:
        max_q = T
    if max_kv is None:
        max_kv = width * cache._page_size
    need = _paged_workspace(T, B, max_q, max_kv, Hq, *cache._extents)
    ws, nbytes = None, 0
    if need > 0 or workspace is not None:
        if workspace is None:
            workspace = _empty(q, (need,), stream, torch.uint8)
        else:
            _scratch(workspace, need, "workspace")
            if workspace.get_device() != dev:
                _wrong_device(workspace, "workspace", dev)
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(lib().ptpc_attn_paged, dev, q.data_ptr(), ldq, cu_q.data_ptr(), cache._pointer,
          page_table.data_ptr(), ldt, width, kv_lens.data_ptr(), T, B, max_q, max_kv, Hq,
          D ** -0.5 if scale is None else scale, out.data_ptr(), ldo, ws, nbytes,
          _stream(dev, stream))
    return out


def attn_prompt(q, k, v, cu, scale=None, out=None, stream=None):
    """Causal attention over whole prompts packed one after another: bf16 [T, q_heads, D].

    q [T, q_heads, D], k, v [T, kv_heads, D] bf16; prompt b is rows cu[b]:cu[b+1] (int32
    [B+1]); scale defaults to D ** -0.5."""
    dev = q.get_device()
    if dev < 0:
        _on_gpu(q, "q")
    T, Hq, D = _three(q, "q")
    _, Hk, _ = _three(k, "k")
    ldq, ldk, ldv = (_heads(q, "q", dev, T, Hq, D), _heads(k, "k", dev, T, Hk, D),
                     _heads(v, "v", dev, T, Hk, D))
    if cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu: expected the B + 1 bounds of B prompts")
    _index(cu, cu.shape, _I32, "cu", dev)
    if cu.shape[0] == 1 and T > 0:
        raise ValueError("cu: the rows of q belong to no sequence")
    if out is None:
        out = _empty(q, (T, Hq, D), stream)
        ldo = Hq * D
    else:
        ldo = _heads(out, "out", dev, T, Hq, D)
    _call(lib().ptpc_attn_prompt, dev, q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
          cu.data_ptr(), T, cu.shape[0] - 1, Hq, Hk, D, D ** -0.5 if scale is None else scale,
          out.data_ptr(), ldo, _stream(dev, stream))
    return out


# -- block-scaled FP8 and experts -------------------------------------------------
def _blocks(n):
    return (n + 127) // 128


class _Checked:
    """Tensors that are checked once, when they are put together, and cannot be exchanged
    afterwards (their contents can change)."""
    __slots__ = ()

    def __setattr__(self, name, value):
        raise AttributeError(f"{type(self).__name__} cannot be changed: make a new one")

    def _put(self, **fields):
        for name, value in fields.items():
            object.__setattr__(self, name, value)

    def _moved(self):
        raise ValueError(f"{type(self).__name__}: its tensors lie elsewhere than when it was made: "
                         f"make a new one")


class BlockWeight(_Checked):
    """A weight with one scale per block of 128 x 128, packed for the GEMM: of one layer
    (experts None) or of `experts` experts of the same size.

    data: uint8 [experts * packed_bytes(Ci, Co)]; sw: float32 [experts, blocks of Co, blocks of
    Ci], without experts 2-D."""
    __slots__ = ("data", "sw", "Ci", "Co", "experts", "_device", "_args", "_kb")

    def __init__(self, data, sw, Ci: int, Co: int, experts: int = None):
        n = packed_bytes(Ci, Co) * (1 if experts is None else experts)
        if data.dtype is not torch.uint8:
            raise TypeError(f"data: expected torch.uint8, got {data.dtype}")
        if data.dim() != 1 or not data.is_contiguous():
            raise ValueError("data: expected a contiguous 1-D tensor")
        if data.shape[0] < n:
            raise ValueError(f"data: expected at least {n} bytes, got {data.shape[0]}")
        dev = _device(data, "data")
        shape = (_blocks(Co), _blocks(Ci))
        _index(sw, shape if experts is None else (experts,) + shape, _F32, "sw", dev)
        self._put(data=data, sw=sw, Ci=Ci, Co=Co, experts=experts, _device=dev,
                  _args=(data.data_ptr(), sw.data_ptr()), _kb=_blocks(Ci))


class Routing(_Checked):
    """What route_experts finds: ids, weights [T, top_k] (int32, float32), and the pairs
    (token, choice) sorted by expert: offsets int32 [experts + 1], rows int32 [T * top_k] (the
    pair t * top_k + k at each row, -1 past the last), slots int32 [T, top_k] (each pair's row,
    -1 if its expert is not laid out).  What a call does not need may be None: gemm_experts takes
    ids (for its shape), offsets and rows, combine_experts weights and slots."""
    __slots__ = ("ids", "weights", "offsets", "rows", "slots", "_device", "_shape", "_ptrs",
                 "_experts")

    def __init__(self, ids, weights, offsets, rows, slots):
        like = ids if ids is not None else slots
        if like is None or like.dim() != 2:
            raise ValueError("ids: expected [tokens, top_k]")
        dev, shape = _device(like, "ids"), tuple(like.shape)
        for t, size, dtype, name in ((ids, shape, _I32, "ids"), (weights, shape, _F32, "weights"),
                                     (offsets, None, _I32, "offsets"),
                                     (rows, (shape[0] * shape[1],), _I32, "rows"),
                                     (slots, shape, _I32, "slots")):
            if t is not None:
                if size is None and (t.dim() != 1 or t.shape[0] < 1):
                    raise ValueError(f"{name}: expected one bound more than experts")
                _index(t, t.shape if size is None else size, dtype, name, dev)
        self._fill(ids, weights, offsets, rows, slots, dev, shape,
                   None if offsets is None else offsets.shape[0] - 1,
                   tuple(None if t is None else t.data_ptr()
                         for t in (offsets, rows, slots, weights)))

    def _fill(self, ids, weights, offsets, rows, slots, dev, shape, experts, ptrs):
        put = object.__setattr__
        put(self, "ids", ids)
        put(self, "weights", weights)
        put(self, "offsets", offsets)
        put(self, "rows", rows)
        put(self, "slots", slots)
        put(self, "_device", dev)
        put(self, "_shape", shape)
        put(self, "_experts", experts)
        put(self, "_ptrs", ptrs)
        return self


def _pitch(t, dtype, name, dev, R=None, C=None):
    """Row pitch of a 2-D tensor [R, C] with unit column stride on GPU dev."""
    if t.dtype is dtype and t.get_device() == dev and t.dim() == 2:
        r, c = t.shape
        s0, s1 = t.stride()
        if (R is None or r == R) and (C is None or c == C) and s1 == 1 and s0 >= c and r > 1:
            return s0
    return _other_pitch(t, dtype, name, dev, R, C)


def _other_pitch(t, dtype, name, dev, R, C):
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor, got shape {tuple(t.shape)}")
    r, c = t.shape
    if (R is not None and r != R) or (C is not None and c != C):
        raise ValueError(f"{name}: expected shape {(r if R is None else R, c if C is None else C)}, "
                         f"got {(r, c)}")
    if t.get_device() != dev:
        _wrong_device(t, name, dev)
    s0, s1 = t.stride()
    if r * c > 0 and ((s1 != 1 and c > 1) or (s0 < c and r > 1)):
        raise ValueError(f"{name}: expected rows apart, with unit column stride")
    return s0 if r > 1 and r * c > 0 else c      # one row or none: its pitch says nothing


def _device(t, name):
    dev = t.get_device()
    if dev < 0:
        _on_gpu(t, name)
    return dev


def quant_act_block(x, gate: bool = False, count=None, qx=None, sx=None, stream=None):
    """FP8 quantization of bf16 X [T, C] with one scale per token and 128 channels ->
    (codes uint8 [T, C], sx fp32 [blocks of C, T]).

    gate: X is [T, 2C] and what is quantized is silu(X[:, :C]) * X[:, C:].  count: int32 [1] on
    the GPU; rows from count on are skipped (routing.offsets[-1:] where not every pair is laid
    out)."""
    dev = _device(x, "x")
    ldx = _pitch(x, _BF16, "x", dev)
    T, C = x.shape
    if gate:
        if C % 2:
            raise ValueError(f"x: expected an even number of columns, got {C}")
        C //= 2
    kb = (C + 127) // 128
    if qx is None:
        qx, ldq = _empty(x, (T, C), stream, _U8), C
    else:
        ldq = _pitch(qx, torch.uint8, "qx", dev, T, C)
    if sx is None:
        sx, lds = _empty(x, (kb, T), stream, _F32), T
    else:
        lds = max(_pitch(sx, _F32, "sx", dev, kb, T), T)
    if count is not None:
        _index(count, (1,), _I32, "count", dev)
    _call(lib().ptpc_quant_act_block, dev, x.data_ptr(), T, C, ldx, gate,
          None if count is None else count.data_ptr(), qx.data_ptr(), ldq, sx.data_ptr(), lds,
          _stream(dev, stream))
    return qx, sx


def _block_weight(like, shape, stream):
    Ci, Co = shape[-2:]
    E = shape[0] if len(shape) == 3 else None
    scales = (_blocks(Co), _blocks(Ci)) if E is None else (E, _blocks(Co), _blocks(Ci))
    n = packed_bytes(Ci, Co) * (1 if E is None else E)
    return BlockWeight(_empty(like, (n,), stream, torch.uint8), _empty(like, scales, stream, _F32),
                       Ci, Co, E)


def quant_weight_block(w, stream=None) -> BlockWeight:
    """bf16 W [Ci, Co], or [experts, Ci, Co], quantized with one scale per 128 x 128 and packed."""
    dev = _device(w, "w")
    if w.dtype is not _BF16:
        raise TypeError(f"w: expected {_BF16}, got {w.dtype}")
    if w.dim() not in (2, 3):
        raise ValueError("w: expected [Ci, Co] or [experts, Ci, Co]")
    Ci, Co = w.shape[-2:]
    ldw, step = w.stride()[-2:]
    if Ci < 2:
        ldw = Co
    if w.numel() > 0 and ((step != 1 and Co > 1) or ldw < Co):
        raise ValueError("w: expected rows apart, with unit column stride")
    bw = _block_weight(w, w.shape, stream)
    _call(lib().ptpc_quant_weight_block, dev, w.data_ptr(), bw.experts if w.dim() == 3 else 1, Ci,
          Co, max(ldw, Co), w.stride(0) if w.dim() == 3 else 0,
          bw.data.data_ptr(), bw.sw.data_ptr(), _stream(dev, stream))
    return bw


def pack_weight_block(codes, scales, stream=None) -> BlockWeight:
    """E4M3 codes (uint8 or float8_e4m3fn) [Ci, Co] or [experts, Ci, Co] and their scales fp32
    [.., blocks of Ci, blocks of Co], as a checkpoint holds them, packed.  Codes may be the
    transposed view of a [Co, Ci] tensor (either of the last two strides is 1)."""
    dev = _device(codes, "codes")
    if codes.dtype is torch.float8_e4m3fn:
        codes = codes.view(torch.uint8)
    if codes.dtype is not torch.uint8:
        raise TypeError(f"codes: expected torch.uint8 or torch.float8_e4m3fn, got {codes.dtype}")
    if codes.dim() not in (2, 3):
        raise ValueError("codes: expected [Ci, Co] or [experts, Ci, Co]")
    Ci, Co = codes.shape[-2:]
    if scales.dtype is not _F32:
        raise TypeError(f"scales: expected {_F32}, got {scales.dtype}")
    want = tuple(codes.shape[:-2]) + (_blocks(Ci), _blocks(Co))
    if tuple(scales.shape) != want:
        raise ValueError(f"scales: expected shape {want}, got {tuple(scales.shape)}")
    if scales.get_device() != dev:
        _wrong_device(scales, "scales", dev)
    ck, co = codes.stride()[-2:]
    if codes.numel() > 0 and ck != 1 and co != 1:
        raise ValueError("codes: expected unit stride along Ci or Co")
    many = codes.dim() == 3
    bw = _block_weight(codes, codes.shape, stream)
    _call(lib().ptpc_pack_weight_block, dev, codes.data_ptr(), codes.stride(0) if many else 0, ck,
          co, scales.data_ptr(), scales.stride(0) if many else 0, *scales.stride()[-2:],
          bw.experts if many else 1, Ci, Co, bw.data.data_ptr(), bw.sw.data_ptr(),
          _stream(dev, stream))
    return bw


def gemm_block_kernel(R: int, Ci: int, Co: int, experts: int = None):
    """Name of the kernel gemm_block (R tokens) or gemm_experts (R pairs) launches (None if none)."""
    r = lib().ptpc_gemm_block_kernel(R, experts or 0, Ci, Co)
    return r.decode() if r is not None else None


def _product_args(qx, sx, bw):
    dev = bw._device
    if (bw.data.data_ptr(), bw.sw.data_ptr()) != bw._args:
        bw._moved()
    ldq = _pitch(qx, torch.uint8, "qx", dev, None, bw.Ci)
    T = qx.shape[0]
    lds = _pitch(sx, _F32, "sx", dev, bw._kb, T)
    return dev, T, ldq, lds if lds > T else T


def gemm_block(qx, sx, bw: BlockWeight, out=None, stream=None):
    """bf16 [T, Co] = X W with X = qx scaled by sx [blocks of Ci, T] (quant_act_block) and W the
    block-scaled weight; each block's sum is scaled and added in fp32."""
    if bw.experts is not None:
        raise ValueError("bw: expected the weight of one layer")
    dev, T, ldq, lds = _product_args(qx, sx, bw)
    Co = bw.Co
    if out is None:
        out, ldo = _empty(qx, (T, Co), stream, _BF16), Co
    else:
        ldo = _pitch(out, _BF16, "out", dev, T, Co)
    _call(lib().ptpc_gemm_block, dev, qx.data_ptr(), ldq, sx.data_ptr(), lds, *bw._args, T, bw.Ci,
          Co, out.data_ptr(), ldo, _stream(dev, stream))
    return out


def linear_block(x, bw: BlockWeight, stream=None):
    """Block-scaled quantization of X followed by the product (one layer's forward)."""
    qx, sx = quant_act_block(x, stream=stream)
    return gemm_block(qx, sx, bw, stream=stream)


def route_experts(logits, top_k: int, scoring: str = "softmax", bias=None, groups: int = 1,
                  top_groups: int = 1, group_top: int = 2, renorm: bool = True, scale: float = 1.0,
                  first: int = 0, local: int = None, workspace=None, stream=None) -> Routing:
    """The top_k of the experts for each token, their weights, and the pairs sorted by expert.

    logits [T, E] fp32 or bf16.  scoring "softmax" or "sigmoid"; the experts are chosen by score
    + bias (fp32 [E]), within the top_groups of `groups` groups whose group_top best are best;
    weights are the scores without bias, divided by their sum if renorm, times scale.  Of equal
    scores the lowest index goes first; the choice is made in 64 bits.  Only the pairs of experts
    first .. first + local - 1 are laid out (default: all).  workspace: uint8,
    route_experts_workspace_bytes."""
    dev = _device(logits, "logits")
    bf16 = logits.dtype is _BF16
    ldl = _pitch(logits, _BF16 if bf16 else _F32, "logits", dev)
    T, E = logits.shape
    if scoring not in ("softmax", "sigmoid"):
        raise ValueError(f"scoring: expected 'softmax' or 'sigmoid', got {scoring!r}")
    if bias is not None:
        _index(bias, (E,), _F32, "bias", dev)
    if local is None:
        local = E - first
    if top_k < 1 or local < 1:
        raise ValueError(f"top_k, local: expected at least 1, got {top_k}, {local}")
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        new, pairs = logits.new_empty, (T, top_k)
        ids, slots = new(pairs, dtype=_I32), new(pairs, dtype=_I32)
        weights = new(pairs, dtype=_F32)
        offsets, rows = new(local + 1, dtype=_I32), new(T * top_k, dtype=_I32)
    need = route_experts_workspace_bytes(T, local)
    nbytes = 0
    if need > 0 or workspace is not None:
        if workspace is None:
            workspace = _empty(logits, (need,), stream, torch.uint8)
        else:
            _scratch(workspace, need, "workspace")
            if workspace.get_device() != dev:
                _wrong_device(workspace, "workspace", dev)
        nbytes = workspace.numel() * workspace.element_size()
    ptrs = offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), weights.data_ptr()
    _call(lib().ptpc_route_experts, dev, logits.data_ptr(), bf16, ldl,
          None if bias is None else bias.data_ptr(), T, E, top_k, scoring == "sigmoid", groups,
          top_groups, group_top, renorm, scale, first, local, ids.data_ptr(), ptrs[3], *ptrs[:3],
          workspace.data_ptr() if nbytes else None, nbytes, _stream(dev, stream))
    return Routing.__new__(Routing)._fill(ids, weights, offsets, rows, slots, dev, pairs, local, ptrs)


@functools.lru_cache(maxsize=4096)
def route_experts_workspace_bytes(T: int, local: int) -> int:
    return int(lib().ptpc_route_experts_workspace_bytes(T, local))


def gemm_experts(qx, sx, bw: BlockWeight, routing: Routing, gather: bool = False, out=None,
                 stream=None):
    """The experts' products, rows sorted by expert: bf16 [T * top_k, Co].

    gather: qx [T, Ci] holds the tokens, and row i is token rows[i] // top_k; otherwise qx
    [T * top_k, Ci] is in the rows' order already (the output of an earlier product, gated and
    quantized).  Rows that no expert has are not written."""
    experts, Co = bw.experts, bw.Co
    if experts is None:
        raise ValueError("bw: expected the weight of experts")
    offsets, rows, _, _ = routing._ptrs
    if offsets is None or rows is None:
        raise ValueError("routing: expected offsets and rows")
    if routing.offsets.data_ptr() != offsets or routing.rows.data_ptr() != rows:
        routing._moved()
    if routing._experts != experts:
        raise ValueError(f"routing: expected the rows of {experts} experts, got "
                         f"{routing._experts}")
    dev, T, ldq, lds = _product_args(qx, sx, bw)
    if routing._device != dev:
        _wrong_device(routing.rows, "routing", dev)
    tokens, top_k = routing._shape
    R = tokens * top_k
    if T != (tokens if gather else R):
        raise ValueError(f"qx: expected {tokens if gather else R} rows, got {T}")
    if out is None:
        out, ldo = _empty(qx, (R, Co), stream, _BF16), Co
    else:
        ldo = _pitch(out, _BF16, "out", dev, R, Co)
    _call(lib().ptpc_gemm_experts, dev, qx.data_ptr(), ldq, sx.data_ptr(), lds, *bw._args, offsets,
          rows if gather else None, top_k, experts, T, R, bw.Ci, Co, out.data_ptr(), ldo,
          _stream(dev, stream))
    return out


def combine_experts(y, routing: Routing, out=None, stream=None):
    """Each token's weighted sum of its experts' rows: bf16 [T, C] from y [T * top_k, C]."""
    dev = routing._device
    _, _, slots, weights = routing._ptrs
    if slots is None or weights is None:
        raise ValueError("routing: expected slots and weights")
    if routing.slots.data_ptr() != slots or routing.weights.data_ptr() != weights:
        routing._moved()
    T, top_k = routing._shape
    R = T * top_k
    ldy = _pitch(y, _BF16, "y", dev, R)
    C = y.shape[1]
    if out is None:
        out, ldo = _empty(y, (T, C), stream), C
    else:
        ldo = _pitch(out, _BF16, "out", dev, T, C)
    _call(lib().ptpc_combine_experts, dev, y.data_ptr(), ldy, R, slots, weights, T, top_k, C,
          out.data_ptr(), ldo, _stream(dev, stream))
    return out
