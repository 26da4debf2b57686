"""GB300 (sm_103a) dynamic-redundant-expert hot path: thin Python binding.

The computation lives in ``libmep.so`` (hand-written CUDA behind the C ABI of
``include/mep.h``). This module only marshals torch CUDA tensors into that
ABI: it checks dtypes, shapes and devices, allocates outputs when the caller
does not pass them, and passes raw device pointers plus torch's current
stream. It never computes a step itself and has no CPU fallback: if the
library is missing, every call raises.

Entry points (same names as the C ABI):

* :func:`mep_plan` -- routing histogram, home-first planner, cu_seqlens and
  destination rows for one layer ("月之暗面开源MoonEP：面向MoE训练的专家并行
  通信库", sections 核心技术 and 内存契约与权重布局);
* :func:`mep_dispatch` -- fused permute into the static [R, S*K, H] buffer;
* :func:`mep_combine` -- fused weighted unpermute back to [R*S, H];
* :func:`mep_reduce_grad` -- slot gradients into home gradients, consumed
  slots zeroed;
* :func:`mep_prefetch` -- redundant experts' weights copied into their slots;
* :func:`mep_dispatch_backward` / :func:`mep_combine_backward` -- gradients of
  the two permutes;
* :func:`mep_grouped_gemm` -- the experts' product over the buffer, and
  :func:`mep_grouped_wgrad` -- its weight gradients, for mep_reduce_grad;
* :func:`mep_layer_norm` / :func:`mep_layer_norm_backward` -- the norm in front
  of the router;
* :func:`mep_swiglu` / :func:`mep_swiglu_backward` -- the experts' gated
  activation;
* :func:`mep_ckpt_save` / :func:`mep_ckpt_load` -- activations kept in 8 bits
  for the backward pass; the norm and the activation write them as they go, and
  all three backward operators read them directly.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import NamedTuple, Optional

__all__ = [
    "MepError", "Plan", "library_path", "load_library", "status_string", "version",
    "plan_workspace_bytes", "plan_kernel_count", "mep_plan", "mep_plan_remote_fallback", "mep_dispatch", "mep_combine", "mep_reduce_grad",
    "mep_prefetch", "mep_dispatch_backward", "mep_combine_backward", "STATUS",
    "grouped_gemm_workspace_bytes", "mep_grouped_gemm", "grouped_wgrad_workspace_bytes", "mep_grouped_wgrad",
    "ckpt_row_bytes", "mep_ckpt_save", "mep_ckpt_load", "layer_norm_backward_workspace_bytes", "mep_layer_norm",
    "mep_layer_norm_backward", "mep_swiglu", "mep_swiglu_backward",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libmep.so"
_lock = threading.Lock()
_lib = None

# Codes from include/mep.h.
STATUS = {
    0: "MEP_OK",
    1: "MEP_ERR_INVALID_ARG",
    2: "MEP_ERR_CUDA",
    3: "MEP_ERR_BAD_ROUTING",
    4: "MEP_ERR_CAPACITY",
    5: "MEP_ERR_BAD_POSITION",
    6: "MEP_ERR_BAD_SLOT_MAP",
    7: "MEP_ERR_TIMEOUT",
    8: "MEP_ERR_BAD_SEQLENS",
}
STATUS_CODE = {v: k for k, v in STATUS.items()}

# (name, restype, argtypes) of every function include/mep.h declares.
_VP = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
# element types of the training operators (MEP_BF16, MEP_F32, MEP_CKPT8)
_BF16, _F32, _CKPT8 = 0, 1, 2
SIGNATURES = [
    ("mep_version", _I, []),
    ("mep_status_string", ctypes.c_char_p, [_I]),
    ("mep_plan_workspace_bytes", _I, [_I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t)]),
    ("mep_plan_kernel_count", _I, [_I, _I, _I, _I, _I, ctypes.POINTER(_I)]),
    ("mep_plan", _I, [_VP, _I, _I, _I, _I, _I, _VP, ctypes.c_size_t, _VP, _VP, _VP, _VP, _VP, _VP]),
    ("mep_plan_remote_fallback", _I, [_VP, _I, _I, _I, _I, _I, _VP, ctypes.c_size_t, _VP, _VP, _VP, _VP, _VP, _VP]),
    ("mep_plan_static_scratch", _I, [_VP, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP]),
    ("mep_dispatch", _I, [_VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP]),
    ("mep_combine", _I, [_VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP]),
    ("mep_reduce_grad", _I, [_VP, _I, _I, _I, ctypes.c_int64, _VP, _VP, _VP, _VP]),
    ("mep_prefetch", _I, [_VP, _I, _I, _I, ctypes.c_int64, _VP, _VP, _VP, _VP]),
    ("mep_dispatch_backward", _I, [_VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP]),
    ("mep_combine_backward", _I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _VP]),
    ("mep_grouped_gemm_workspace_bytes", _I, [_I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t)]),
    ("mep_grouped_gemm", _I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _VP, ctypes.c_size_t,
                              _VP, _VP]),
    ("mep_ckpt_row_bytes", _I, [_L, ctypes.POINTER(ctypes.c_size_t)]),
    ("mep_ckpt_save", _I, [_VP, _I, _L, _L, _VP, _VP]),
    ("mep_ckpt_load", _I, [_VP, _L, _L, _I, _VP, _VP]),
    ("mep_layer_norm", _I, [_VP, _I, _VP, _VP, _I, ctypes.c_float, _L, _L, _VP, _VP, _VP, _VP, _VP, _VP]),
    ("mep_layer_norm_backward_workspace_bytes", _I, [_L, _L, ctypes.POINTER(ctypes.c_size_t)]),
    ("mep_layer_norm_backward", _I, [_VP, _I, _VP, _I, _VP, _I, _VP, _VP, _L, _L, _VP, ctypes.c_size_t, _VP,
                                     _VP, _VP, _I, _VP]),
    ("mep_swiglu", _I, [_VP, _L, _L, _VP, _VP, _VP]),
    ("mep_swiglu_backward", _I, [_VP, _VP, _I, _L, _L, _VP, _VP, _VP]),
    ("mep_grouped_wgrad_workspace_bytes", _I, [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t)]),
    ("mep_grouped_wgrad", _I, [_VP, _I, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _I, _VP, ctypes.c_size_t,
                               _VP, _VP, _VP]),
    ("mep_wait_selftest", _I, [_VP, ctypes.c_int64, _VP, _VP]),
]


class MepError(RuntimeError):
    """A host-side error code returned by the library."""

    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} returned {STATUS.get(code, code)}: {status_string(code)}")


def library_path() -> str:
    return os.path.join(_PKG, _LIB_NAME)


def load_library():
    """Load libmep.so (built in-tree by ``_build.build()``); raises if absent."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with load_balancing_topk_gb300._build.build() "
                    "(there is no fallback implementation)")
            lib = ctypes.CDLL(path)
            for name, res, args in SIGNATURES:
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def version() -> tuple[int, int]:
    v = load_library().mep_version()
    return v >> 16, v & 0xFFFF


def status_string(code: int) -> str:
    return load_library().mep_status_string(int(code)).decode()


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise MepError(fn, rc)


def plan_workspace_bytes(R: int, S: int, K: int, E: int, B: int) -> int:
    out = ctypes.c_size_t(0)
    _check("mep_plan_workspace_bytes",
           load_library().mep_plan_workspace_bytes(R, S, K, E, B, ctypes.byref(out)))
    return int(out.value)


def plan_kernel_count(R: int, S: int, K: int, E: int, B: int) -> int:
    """Kernels one mep_plan call enqueues for these sizes (launch accounting)."""
    n = _I(0)
    _check("mep_plan_kernel_count", load_library().mep_plan_kernel_count(R, S, K, E, B, ctypes.byref(n)))
    return int(n.value)


def grouped_gemm_workspace_bytes(R: int, S: int, K: int, E: int, B: int) -> int:
    out = ctypes.c_size_t(0)
    _check("mep_grouped_gemm_workspace_bytes",
           load_library().mep_grouped_gemm_workspace_bytes(R, S, K, E, B, ctypes.byref(out)))
    return int(out.value)


# ---------------------------------------------------------------------------
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _need(t, name, dtype, shape=None, device=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    torch = _torch()
    return torch.cuda.current_stream(device).cuda_stream


class Plan(NamedTuple):
    """Outputs of :func:`mep_plan` (all on the device)."""

    expert_counts: "torch.Tensor"   # int32 [E]
    cu_seqlens: "torch.Tensor"      # int32 [R, E+B]
    slot_expert: "torch.Tensor"     # int32 [R, B]
    dst_pos: "torch.Tensor"         # int32 [R*S, K]
    status: "torch.Tensor"          # int32 [1]
    workspace: "torch.Tensor"       # uint8 scratch, reusable for the same sizes


def mep_plan(topk_idx, R: int, S: int, K: int, E: int, B: int, out: Optional[Plan] = None) -> Plan:
    """Plan one layer's routing. ``topk_idx`` is int32 [R*S, K] on the device.

    Nothing is synchronised: read ``status`` (0 = ok) when convenient.
    """
    return _plan("mep_plan", topk_idx, R, S, K, E, B, out)


def mep_plan_remote_fallback(topk_idx, R: int, S: int, K: int, E: int, B: int,
                             out: Optional[Plan] = None) -> Plan:
    """mep_plan under the inference reading: pieces beyond a rank's B slots
    take the expert's own row (served by its home weights) instead of failing."""
    return _plan("mep_plan_remote_fallback", topk_idx, R, S, K, E, B, out)


def _plan(fn: str, topk_idx, R, S, K, E, B, out):
    torch = _torch()
    _need(topk_idx, "topk_idx", torch.int32, (R * S, K))
    dev = topk_idx.device
    ws_bytes = plan_workspace_bytes(R, S, K, E, B)
    if out is None:
        out = Plan(
            expert_counts=torch.empty(E, dtype=torch.int32, device=dev),
            cu_seqlens=torch.empty((R, E + B), dtype=torch.int32, device=dev),
            slot_expert=torch.empty((R, B), dtype=torch.int32, device=dev),
            dst_pos=torch.empty((R * S, K), dtype=torch.int32, device=dev),
            status=torch.empty(1, dtype=torch.int32, device=dev),
            workspace=torch.empty(ws_bytes, dtype=torch.uint8, device=dev),
        )
    else:
        _need(out.expert_counts, "expert_counts", torch.int32, (E,), dev)
        _need(out.cu_seqlens, "cu_seqlens", torch.int32, (R, E + B), dev)
        _need(out.slot_expert, "slot_expert", torch.int32, (R, B), dev)
        _need(out.dst_pos, "dst_pos", torch.int32, (R * S, K), dev)
        _need(out.status, "status", torch.int32, (1,), dev)
        _need(out.workspace, "workspace", torch.uint8, None, dev)
        if out.workspace.numel() < ws_bytes:
            raise ValueError(f"workspace has {out.workspace.numel()} bytes, needs {ws_bytes}")
    with torch.cuda.device(dev):
        rc = getattr(load_library(), fn)(
            _ptr(topk_idx), R, S, K, E, B, _ptr(out.workspace), out.workspace.numel(),
            _ptr(out.expert_counts), _ptr(out.cu_seqlens), _ptr(out.slot_expert),
            _ptr(out.dst_pos), _ptr(out.status), _stream(dev))
    _check(fn, rc)
    return out


def mep_dispatch(hidden, dst_pos, status, R: int, S: int, K: int, buf=None):
    """buf[dst_pos[t, k]] = hidden[t]; returns buf (bf16 [R*S*K, H])."""
    torch = _torch()
    _need(hidden, "hidden", torch.bfloat16)
    N, H = hidden.shape
    if N != R * S:
        raise ValueError("hidden must be [R*S, H]")
    dev = hidden.device
    _need(dst_pos, "dst_pos", torch.int32, (N, K), dev)
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    if buf is None:
        buf = torch.empty((N * K, H), dtype=torch.bfloat16, device=dev)
    else:
        _need(buf, "buf", torch.bfloat16, None, dev)
        if buf.numel() != N * K * H:
            raise ValueError("buf must hold R*S*K rows of H")
    with torch.cuda.device(dev):
        rc = load_library().mep_dispatch(_ptr(hidden), _ptr(dst_pos), _ptr(status), R, S, K, H,
                                         _ptr(buf), _stream(dev))
    _check("mep_dispatch", rc)
    return buf


def mep_combine(y, topk_w, dst_pos, status, R: int, S: int, K: int, out=None):
    """out[t] = bf16(sum_k topk_w[t, k] * y[dst_pos[t, k]]) (fp32 fma in k order)."""
    torch = _torch()
    _need(y, "y", torch.bfloat16)
    H = y.shape[-1]
    N = R * S
    if y.numel() != N * K * H:
        raise ValueError("y must hold R*S*K rows of H")
    dev = y.device
    _need(topk_w, "topk_w", torch.float32, (N, K), dev)
    _need(dst_pos, "dst_pos", torch.int32, (N, K), dev)
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    if out is None:
        out = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, "out", torch.bfloat16, (N, H), dev)
    with torch.cuda.device(dev):
        rc = load_library().mep_combine(_ptr(y), _ptr(topk_w), _ptr(dst_pos), _ptr(status),
                                        R, S, K, H, _ptr(out), _stream(dev))
    _check("mep_combine", rc)
    return out


def mep_reduce_grad(slot_expert, home_grad, slot_grad, status, E: int):
    """home_grad[e] += slots of e in (r, b) order; consumed slots zeroed. In place.

    home_grad: fp32 [E, ...]; slot_grad: fp32 [R, B, ...] with the same
    trailing element count (H*H'); slot_expert: int32 [R, B].
    """
    torch = _torch()
    _need(slot_expert, "slot_expert", torch.int32)
    R, B = slot_expert.shape
    dev = slot_expert.device
    _need(home_grad, "home_grad", torch.float32, None, dev)
    _need(slot_grad, "slot_grad", torch.float32, None, dev)
    if home_grad.numel() % E:
        raise ValueError("home_grad must be [E, H*H']")
    HHp = home_grad.numel() // E
    if slot_grad.numel() != R * B * HHp:
        raise ValueError("slot_grad must be [R, B, H*H']")
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    with torch.cuda.device(dev):
        rc = load_library().mep_reduce_grad(_ptr(slot_expert), E, R, B, HHp, _ptr(home_grad),
                                            _ptr(slot_grad), _ptr(status), _stream(dev))
    _check("mep_reduce_grad", rc)
    return home_grad, slot_grad


def mep_prefetch(slot_expert, home_w, slot_w, status, E: int):
    """slot_w[r, b] = home_w[slot_expert[r, b]] for every used slot (in place).

    home_w: [E, ...]; slot_w: [R, B, ...] with the same dtype and trailing
    size; slot_expert: int32 [R, B]. Any dtype (the copy is bytewise).
    """
    torch = _torch()
    _need(slot_expert, "slot_expert", torch.int32)
    R, B = slot_expert.shape
    dev = slot_expert.device
    _need(home_w, "home_w", home_w.dtype, None, dev)
    _need(slot_w, "slot_w", home_w.dtype, None, dev)
    nbytes = home_w.numel() * home_w.element_size()
    if nbytes % E:
        raise ValueError("home_w must be [E, ...]")
    per = nbytes // E
    if slot_w.numel() * slot_w.element_size() != R * B * per:
        raise ValueError("slot_w must be [R, B, ...] with home_w's trailing size")
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    with torch.cuda.device(dev):
        rc = load_library().mep_prefetch(_ptr(slot_expert), E, R, B, per, _ptr(home_w),
                                         _ptr(slot_w), _ptr(status), _stream(dev))
    _check("mep_prefetch", rc)
    return slot_w


def mep_dispatch_backward(dbuf, dst_pos, status, R: int, S: int, K: int, dhidden=None):
    """dhidden[t] = bf16(sum_k dbuf[dst_pos[t, k]]) (fp32 adds in k order)."""
    torch = _torch()
    _need(dbuf, "dbuf", torch.bfloat16)
    H = dbuf.shape[-1]
    N = R * S
    if dbuf.numel() != N * K * H:
        raise ValueError("dbuf must hold R*S*K rows of H")
    dev = dbuf.device
    _need(dst_pos, "dst_pos", torch.int32, (N, K), dev)
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    if dhidden is None:
        dhidden = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
    else:
        _need(dhidden, "dhidden", torch.bfloat16, (N, H), dev)
    with torch.cuda.device(dev):
        rc = load_library().mep_dispatch_backward(_ptr(dbuf), _ptr(dst_pos), _ptr(status), R, S, K,
                                                  H, _ptr(dhidden), _stream(dev))
    _check("mep_dispatch_backward", rc)
    return dhidden


def mep_combine_backward(dout, y, topk_w, dst_pos, status, R: int, S: int, K: int, dy=None,
                         dw=None):
    """(dy, dw) with dy[dst_pos[t,k]] = bf16(w[t,k] * dout[t]) and
    dw[t,k] = <dout[t], y[dst_pos[t,k]]> (fp32)."""
    torch = _torch()
    _need(dout, "dout", torch.bfloat16)
    N, H = dout.shape
    if N != R * S:
        raise ValueError("dout must be [R*S, H]")
    dev = dout.device
    _need(y, "y", torch.bfloat16, None, dev)
    if y.numel() != N * K * H:
        raise ValueError("y must hold R*S*K rows of H")
    _need(topk_w, "topk_w", torch.float32, (N, K), dev)
    _need(dst_pos, "dst_pos", torch.int32, (N, K), dev)
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    if dy is None:
        dy = torch.empty((N * K, H), dtype=torch.bfloat16, device=dev)
    else:
        _need(dy, "dy", torch.bfloat16, None, dev)
        if dy.numel() != N * K * H:
            raise ValueError("dy must hold R*S*K rows of H")
    if dw is None:
        dw = torch.empty((N, K), dtype=torch.float32, device=dev)
    else:
        _need(dw, "dw", torch.float32, (N, K), dev)
    with torch.cuda.device(dev):
        rc = load_library().mep_combine_backward(_ptr(dout), _ptr(y), _ptr(topk_w), _ptr(dst_pos),
                                                 _ptr(status), R, S, K, H, _ptr(dy), _ptr(dw),
                                                 _stream(dev))
    _check("mep_combine_backward", rc)
    return dy, dw


def mep_grouped_gemm(x, cu_seqlens, w_home, w_slot, status, R: int, S: int, K: int,
                     y=None, workspace=None):
    """y[row] = bf16(x[row] @ W_j) for the group j of every buffer row.

    x: bf16 [R*S*K, H] (the dispatch buffer); cu_seqlens: int32 [R, E+B];
    w_home: bf16 [E, H, H']; w_slot: bf16 [R, B, H, H'] (None when B == 0).
    Group j of rank r uses w_home[j] below E and w_slot[r, j - E] above.
    Returns y, bf16 [R*S*K, H'].
    """
    torch = _torch()
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(w_home, "w_home", torch.bfloat16, None, dev)
    E, H, Hp = w_home.shape
    _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
    if cu_seqlens.dim() != 2 or cu_seqlens.shape[0] != R:
        raise ValueError("cu_seqlens must be [R, E+B]")
    B = cu_seqlens.shape[1] - E
    if B < 0:
        raise ValueError("cu_seqlens must have E+B columns")
    if x.numel() != R * S * K * H:
        raise ValueError("x must hold R*S*K rows of H")
    if B > 0:
        _need(w_slot, "w_slot", torch.bfloat16, (R, B, H, Hp), dev)
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    if y is None:
        y = torch.empty((R * S * K, Hp), dtype=torch.bfloat16, device=dev)
    else:
        _need(y, "y", torch.bfloat16, (R * S * K, Hp), dev)
    need = grouped_gemm_workspace_bytes(R, S, K, E, B)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        rc = load_library().mep_grouped_gemm(_ptr(x), _ptr(cu_seqlens), _ptr(w_home),
                                             _ptr(w_slot) if B > 0 else None, _ptr(status), R, S,
                                             K, E, B, H, Hp, _ptr(workspace), need, _ptr(y),
                                             _stream(dev))
    _check("mep_grouped_gemm", rc)
    return y


# The calls below are short next to what a check or a launch costs on the host,
# so their checks look at a good tensor once (_good) and name what is wrong
# (_need) only when something is; sizes that the library computes are kept.
def _good(t, name, dtype, shape, dev):
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == dev:
            return t
    except AttributeError:
        pass
    return _need(t, name, dtype, shape, dev)


def _call(fn: str, dev, *args) -> None:
    """Enqueue one library call on the current stream of dev."""
    torch = _torch()
    entry = getattr(_lib if _lib is not None else load_library(), fn)
    index = dev.index
    if torch._C._cuda_getDevice() == index:
        rc = entry(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            rc = entry(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != 0:
        raise MepError(fn, rc)


def _cuda_device(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


@functools.lru_cache(maxsize=256)
def ckpt_row_bytes(C: int) -> int:
    """Bytes of one checkpoint row of C columns (a multiple of 32)."""
    out = ctypes.c_size_t(0)
    _check("mep_ckpt_row_bytes", load_library().mep_ckpt_row_bytes(int(C), ctypes.byref(out)))
    return int(out.value)


@functools.lru_cache(maxsize=256)
def layer_norm_backward_workspace_bytes(N: int, H: int) -> int:
    """Bytes of mep_layer_norm_backward's workspace for up to N rows of H columns."""
    out = ctypes.c_size_t(0)
    _check("mep_layer_norm_backward_workspace_bytes",
           load_library().mep_layer_norm_backward_workspace_bytes(int(N), int(H), ctypes.byref(out)))
    return int(out.value)


@functools.lru_cache(maxsize=256)
def grouped_wgrad_workspace_bytes(R: int, S: int, K: int, E: int, B: int, H: int, Hp: int) -> int:
    """Bytes of mep_grouped_wgrad's workspace for up to S tokens a rank."""
    out = ctypes.c_size_t(0)
    _check("mep_grouped_wgrad_workspace_bytes",
           load_library().mep_grouped_wgrad_workspace_bytes(R, S, K, E, B, H, Hp, ctypes.byref(out)))
    return int(out.value)


def _float_type(t, name) -> int:
    """MEP_BF16 or MEP_F32 of a tensor that may be either."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is torch.bfloat16:
        return _BF16
    if t.dtype is torch.float32:
        return _F32
    raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")


def _matrix(t, name) -> int:
    """Type of a dense CUDA matrix in bf16 or fp32."""
    kind = _float_type(t, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return kind


def _need_params(weight, bias, H, dev) -> int:
    """Checks a norm's weight and bias (each may be None); their type."""
    if weight is not None:
        kind = _float_type(weight, "weight")
        _good(weight, "weight", weight.dtype, (H,), dev)
        if bias is not None:
            if _float_type(bias, "bias") != kind:
                raise TypeError("weight and bias must have the same dtype")
            _good(bias, "bias", bias.dtype, (H,), dev)
        return kind
    if bias is not None:
        kind = _float_type(bias, "bias")
        _good(bias, "bias", bias.dtype, (H,), dev)
        return kind
    return _F32


def mep_ckpt_save(x, ckpt=None):
    """x (bf16 or fp32 [N, C]) in 8 bits: checkpoint rows, uint8 [N, ckpt_row_bytes(C)].

    Signed bytes with one power-of-two scale per 128 columns, in one row, so
    that mep_dispatch can permute the rows seen as bf16.
    """
    torch = _torch()
    kind = _matrix(x, "x")
    N, C = x.shape
    dev, rb = x.device, ckpt_row_bytes(C)
    if ckpt is None:
        ckpt = torch.empty((N, rb), dtype=torch.uint8, device=dev)
    else:
        _good(ckpt, "ckpt", torch.uint8, (N, rb), dev)
    _call("mep_ckpt_save", dev, x.data_ptr(), kind, N, C, ckpt.data_ptr())
    return ckpt


def mep_ckpt_load(ckpt, C: int, x=None, dtype=None):
    """The values of checkpoint rows (uint8 [N, ckpt_row_bytes(C)]): [N, C] in x's
    dtype, or ``dtype`` (bf16 unless given; both hold the values exactly)."""
    torch = _torch()
    dev, rb = _cuda_device(ckpt, "ckpt"), ckpt_row_bytes(C)
    if ckpt.dim() != 2 or ckpt.shape[1] != rb:
        raise ValueError(f"ckpt must be [N, {rb}] for {C} columns")
    N = ckpt.shape[0]
    _good(ckpt, "ckpt", torch.uint8, (N, rb), dev)
    if x is None:
        x = torch.empty((N, C), dtype=torch.bfloat16 if dtype is None else dtype, device=dev)
        kind = _float_type(x, "x")
    else:
        kind = _float_type(x, "x")
        _good(x, "x", x.dtype if dtype is None else dtype, (N, C), dev)
    _call("mep_ckpt_load", dev, ckpt.data_ptr(), N, C, kind, x.data_ptr())
    return x


def mep_layer_norm(x, weight=None, bias=None, eps: float = 1e-5, y=None, mean=None, rstd=None,
                   x_ckpt=None, y_ckpt=None):
    """(y, mean, rstd) of the layer norm of every row of x (bf16 or fp32 [N, H]).

    weight, bias: bf16 or fp32 [H], or None. y has x's dtype; mean and rstd are
    fp32 [N]. x_ckpt, y_ckpt: uint8 [N, ckpt_row_bytes(H)] to keep x (for
    mep_layer_norm_backward) and y (for mep_grouped_wgrad) in, or None.
    """
    torch = _torch()
    kind = _matrix(x, "x")
    N, H = x.shape
    dev = x.device
    p_kind = _need_params(weight, bias, H, dev)
    y = torch.empty_like(x) if y is None else _good(y, "y", x.dtype, (N, H), dev)
    f32 = torch.float32
    mean = torch.empty(N, dtype=f32, device=dev) if mean is None else _good(mean, "mean", f32, (N,), dev)
    rstd = torch.empty(N, dtype=f32, device=dev) if rstd is None else _good(rstd, "rstd", f32, (N,), dev)
    if x_ckpt is not None:
        _good(x_ckpt, "x_ckpt", torch.uint8, (N, ckpt_row_bytes(H)), dev)
    if y_ckpt is not None:
        _good(y_ckpt, "y_ckpt", torch.uint8, (N, ckpt_row_bytes(H)), dev)
    _call("mep_layer_norm", dev, x.data_ptr(), kind, _ptr(weight), _ptr(bias), p_kind, eps, N, H,
          y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _ptr(x_ckpt), _ptr(y_ckpt))
    return y, mean, rstd


def mep_layer_norm_backward(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None,
                            accumulate: bool = False, params: bool = True, workspace=None):
    """(dx, dweight, dbias) of mep_layer_norm.

    dy: bf16 or fp32 [N, H]; x: the norm's input in dy's dtype, or its
    checkpoint rows (uint8, the norm's x_ckpt); weight: as in the forward pass.
    dx has dy's dtype, dweight and dbias are fp32 [H] (added to where
    ``accumulate``). ``params=False``: dx alone, (dx, None, None).
    """
    torch = _torch()
    kind = _matrix(dy, "dy")
    N, H = dy.shape
    dev, f32 = dy.device, torch.float32
    if isinstance(x, torch.Tensor) and x.dtype is torch.uint8:
        x_kind = _CKPT8
        _good(x, "x", torch.uint8, (N, ckpt_row_bytes(H)), dev)
    else:
        x_kind = kind
        _good(x, "x", dy.dtype, (N, H), dev)
    p_kind = _need_params(weight, None, H, dev)
    _good(mean, "mean", f32, (N,), dev)
    _good(rstd, "rstd", f32, (N,), dev)
    dx = torch.empty_like(dy) if dx is None else _good(dx, "dx", dy.dtype, (N, H), dev)
    need = 0
    if params:
        if accumulate and (dweight is None or dbias is None):
            raise ValueError("accumulate needs dweight and dbias to add to")
        dweight = torch.empty(H, dtype=f32, device=dev) if dweight is None else _good(dweight, "dweight", f32, (H,), dev)
        dbias = torch.empty(H, dtype=f32, device=dev) if dbias is None else _good(dbias, "dbias", f32, (H,), dev)
        need = layer_norm_backward_workspace_bytes(N, H)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            _need(workspace, "workspace", torch.uint8, None, dev)
            if workspace.numel() < need:
                raise ValueError(f"workspace has {workspace.numel()} bytes, needs {need}")
    elif dweight is not None or dbias is not None:
        raise ValueError("params=False computes neither dweight nor dbias")
    _call("mep_layer_norm_backward", dev, dy.data_ptr(), kind, x.data_ptr(), x_kind, _ptr(weight), p_kind,
          mean.data_ptr(), rstd.data_ptr(), N, H, _ptr(workspace) if params else None, need, dx.data_ptr(),
          _ptr(dweight), _ptr(dbias), 1 if accumulate else 0)
    return dx, dweight, dbias


def mep_swiglu(gu, a=None, ckpt=None):
    """a = bf16(g * sigmoid(g) * u), g and u the two halves of every row of gu (bf16 [rows, 2F]).

    ckpt: uint8 [rows, 2, ckpt_row_bytes(F)] to keep gu in for the backward pass, or None.
    """
    torch = _torch()
    dev, bf16 = _cuda_device(gu, "gu"), torch.bfloat16
    if gu.dim() != 2 or gu.shape[1] < 2 or gu.shape[1] % 2:
        raise ValueError("gu must be [rows, 2F]")
    rows, F = gu.shape[0], gu.shape[1] // 2
    _good(gu, "gu", bf16, (rows, 2 * F), dev)
    a = torch.empty((rows, F), dtype=bf16, device=dev) if a is None else _good(a, "a", bf16, (rows, F), dev)
    if ckpt is not None:
        _good(ckpt, "ckpt", torch.uint8, (rows, 2, ckpt_row_bytes(F)), dev)
    _call("mep_swiglu", dev, gu.data_ptr(), rows, F, a.data_ptr(), _ptr(ckpt))
    return a


def mep_swiglu_backward(da, gu, dgu=None, a=None, again: bool = True):
    """(dgu, a) of mep_swiglu from da (bf16 [rows, F]) and gu (bf16 [rows, 2F], or the
    checkpoint rows kept of it, uint8 [rows, 2, ckpt_row_bytes(F)]).

    dgu: bf16 [rows, 2F]. a: the activation once more, computed from what gu
    stands for (None where ``again`` is false).
    """
    torch = _torch()
    dev, bf16 = _cuda_device(da, "da"), torch.bfloat16
    if da.dim() != 2:
        raise ValueError("da must be [rows, F]")
    rows, F = da.shape
    _good(da, "da", bf16, (rows, F), dev)
    if isinstance(gu, torch.Tensor) and gu.dtype is torch.uint8:
        kind = _CKPT8
        _good(gu, "gu", torch.uint8, (rows, 2, ckpt_row_bytes(F)), dev)
    else:
        kind = _BF16
        _good(gu, "gu", bf16, (rows, 2 * F), dev)
    dgu = (torch.empty((rows, 2 * F), dtype=bf16, device=dev) if dgu is None
           else _good(dgu, "dgu", bf16, (rows, 2 * F), dev))
    if not again:
        if a is not None:
            raise ValueError("again=False does not compute a")
    elif a is None:
        a = torch.empty((rows, F), dtype=bf16, device=dev)
    else:
        _good(a, "a", bf16, (rows, F), dev)
    _call("mep_swiglu_backward", dev, da.data_ptr(), gu.data_ptr(), kind, rows, F, dgu.data_ptr(), _ptr(a))
    return dgu, a


def mep_grouped_wgrad(x, dy, cu_seqlens, home_grad, slot_grad, status, R: int, S: int, K: int,
                      accumulate: bool = False, workspace=None):
    """Weight gradients of mep_grouped_gemm, in place: home_grad[e] = sum of x[row]^T dy[row]
    over the rows of group e of every rank, slot_grad[r, b] over rank r's rows of slot b.

    x: bf16 [R*S*K, H], or checkpoint rows uint8 [R*S*K, ckpt_row_bytes(H)]; dy:
    bf16 [R*S*K, H']; cu_seqlens: int32 [R, E+B]; home_grad: fp32 [E, H, H'];
    slot_grad: fp32 [R, B, H, H'] (None when B == 0), as mep_reduce_grad reads
    them. Slots without rows are left alone. Returns (home_grad, slot_grad).
    """
    torch = _torch()
    dev = _cuda_device(dy, "dy")
    if not isinstance(home_grad, torch.Tensor) or home_grad.dim() != 3:
        raise ValueError("home_grad must be [E, H, H']")
    E, H, Hp = home_grad.shape
    _good(home_grad, "home_grad", torch.float32, (E, H, Hp), dev)
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 2 or cu_seqlens.shape[0] != R:
        raise ValueError("cu_seqlens must be [R, E+B]")
    B = cu_seqlens.shape[1] - E
    if B < 0:
        raise ValueError("cu_seqlens must have E+B columns")
    _good(cu_seqlens, "cu_seqlens", torch.int32, (R, E + B), dev)
    rows = R * S * K
    _good(dy, "dy", torch.bfloat16, dy.shape, dev)
    if isinstance(x, torch.Tensor) and x.dtype is torch.uint8:
        kind, width = _CKPT8, ckpt_row_bytes(H)
        _good(x, "x", torch.uint8, x.shape, dev)
    else:
        kind, width = _BF16, H
        _need(x, "x", torch.bfloat16, None, dev)
    if x.numel() != rows * width:
        raise ValueError(f"x must hold R*S*K rows of {width}")
    if dy.numel() != rows * Hp:
        raise ValueError("dy must hold R*S*K rows of H'")
    if B > 0:
        _good(slot_grad, "slot_grad", torch.float32, (R, B, H, Hp), dev)
    if status is not None:
        _good(status, "status", torch.int32, (1,), dev)
    need = grouped_wgrad_workspace_bytes(R, S, K, E, B, H, Hp)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", torch.uint8, None, dev)
        if workspace.numel() < need:
            raise ValueError(f"workspace has {workspace.numel()} bytes, needs {need}")
    _call("mep_grouped_wgrad", dev, x.data_ptr(), kind, dy.data_ptr(), cu_seqlens.data_ptr(), _ptr(status),
          R, S, K, E, B, H, Hp, 1 if accumulate else 0, workspace.data_ptr(), workspace.numel(),
          home_grad.data_ptr(), slot_grad.data_ptr() if B > 0 else None)
    return home_grad, slot_grad


def mep_wait_selftest(limit_ns: int, device=None):
    """Run the bounded-wait self-test on the device; returns (status, elapsed_ns)
    tensors (int32 [1], int64 [1]) after it is enqueued (not synchronised)."""
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    elapsed = torch.zeros(1, dtype=torch.int64, device=dev)
    with torch.cuda.device(dev):
        rc = load_library().mep_wait_selftest(_ptr(status), int(limit_ns), _ptr(elapsed),
                                              _stream(dev))
    _check("mep_wait_selftest", rc)
    return status, elapsed
