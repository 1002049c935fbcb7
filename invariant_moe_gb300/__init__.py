"""Python binding of libbimoe.so, the batch-invariant MoE hot path for GB300.

Argument marshalling only: every function checks tensor dtypes / devices /
contiguity, passes raw device pointers and the current CUDA stream to the C
ABI declared in ``include/bimoe.h``, and raises on a non-zero status.  All
arithmetic runs in the library's CUDA kernels; there is no CPU fallback.  If
the library is missing the first call raises ``RuntimeError`` -- build it with
``python -m invariant_moe_gb300._build`` (or ``__graft_entry__.build()``).

Names follow the C entry points: ``bi_router_gemm``, ``bi_topk``,
``bi_moe_forward`` and the per-stage calls.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbimoe.so")

BI_OK = 0
STATUS = {0: "BI_OK", 1: "BI_ERR_INVALID_ARG", 2: "BI_ERR_UNSUPPORTED", 3: "BI_ERR_WORKSPACE",
          4: "BI_ERR_CUDA", 5: "BI_ERR_DEVICE"}
DEVERR = {0: "none", 1: "expert id out of range", 2: "repeated expert in a row",
          3: "bounded wait timed out", 4: "offsets / perm are not a grouping of the pairs"}

# every symbol include/bimoe.h declares (checked by the CPU test-suite)
EXPORTS = [
    "bi_status_str", "bi_last_error_message", "bi_version", "bi_device_error",
    "bi_cast_bf16_to_f32", "bi_router_gemm", "bi_router_gemm_schedule",
    "bi_router_gemm_splitk_negctl", "bi_topk", "bi_moe_workspace_bytes", "bi_moe_forward",
    "bi_moe_permute_workspace_bytes", "bi_moe_permute", "bi_moe_gather",
    "bi_moe_gate_up", "bi_moe_down", "bi_moe_combine", "bi_moe_combine_consume", "bi_moe_forward_noalloc",
    "bi_fp32_fma_probe", "bi_wait_timeout_probe", "bi_moe_gemm_variant", "bi_router_topk", "bi_router_topk_schedule",
    "bi_topk_window", "bi_router_gemm_bf16", "bi_router_gemm_bf16_schedule", "bi_router_topk_bf16",
    "bi_moe_gather_routing", "bi_moe_scatter_contrib", "bi_router_topk_bf16_schedule",
    "bi_moe_gate_up_tokens", "bi_moe_gate_up_feed", "bi_moe_layer", "bi_moe_decode_fused",
    "bi_ffn_workspace_bytes", "bi_ffn_forward", "bi_ffn_forward_train", "bi_ffn_backward",
    "bi_ffn_schedule",
    "bi_mx4_scale_bytes", "bi_mx4_quantize", "bi_mx4_dequantize", "bi_mx4_gemm", "bi_mx4_gate_up",
    "bi_mx4_form",
]


class BimoeError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn}: {STATUS.get(status, status)}: {msg}")
        self.status = status


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """dlopen libbimoe.so and declare its signatures (no GPU needed)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"CUDA library {path} is missing; build it with "
                "`python -m invariant_moe_gb300._build`")
        lib = ctypes.CDLL(path)
        P, I64, I32, SZ, ST = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                               ctypes.c_size_t, ctypes.c_int)
        sig = {
            "bi_status_str": ([ctypes.c_int], ctypes.c_char_p),
            "bi_last_error_message": ([], ctypes.c_char_p),
            "bi_version": ([], ctypes.c_char_p),
            "bi_device_error": ([P], ST),
            "bi_cast_bf16_to_f32": ([P, P, I64, P], ST),
            "bi_router_gemm": ([P, P, P, P, I64, I64, I64, P], ST),
            "bi_router_gemm_schedule": ([P, P, P, P, I64, I64, I64, I32, P], ST),
            "bi_router_gemm_splitk_negctl": ([P, P, P, P, I64, I64, I64, P], ST),
            "bi_topk": ([P, P, P, P, I64, I64, I32, P], ST),
            "bi_moe_workspace_bytes": ([I64, I64, I64, I32, I64], SZ),
            "bi_moe_forward": ([P, P, P, P, P, P, I64, I64, I64, I32, I64, P, SZ, P], ST),
            "bi_moe_permute_workspace_bytes": ([I64, I64], SZ),
            "bi_moe_permute": ([P, P, P, I64, I64, I32, P, SZ, P], ST),
            "bi_moe_gather": ([P, P, P, P, I64, I64, I64, I32, P], ST),
            "bi_moe_gate_up": ([P, P, P, P, P, P, I64, I64, I64, I32, I64, P], ST),
            "bi_moe_down": ([P, P, P, P, P, I64, I64, I64, I32, I64, P], ST),
            "bi_moe_combine": ([P, P, I64, I64, I32, P], ST),
            "bi_moe_combine_consume": ([P, P, I64, I64, I32, P], ST),
            "bi_moe_gemm_variant": ([I32, P], ST),
            "bi_moe_gate_up_feed": ([I32, P], ST),
            "bi_moe_decode_fused": ([I32, P], ST),
            "bi_moe_layer": ([P, P, P, P, P, P, P, P, P, I64, I64, I64, I32, I64, P, SZ, P], ST),
            "bi_moe_gate_up_tokens": ([P, P, P, P, P, P, I64, I64, I64, I32, I64, P], ST),
            "bi_router_topk": ([P, P, P, P, P, P, P, I64, I64, I64, I32, P], ST),
            "bi_router_topk_schedule": ([P, P, P, P, P, P, P, I64, I64, I64, I32, I32, P], ST),
            "bi_topk_window": ([P, I64, P, P, I64, I64, I32, P, P], ST),
            "bi_router_gemm_bf16": ([P, P, P, P, I64, I64, I64, P], ST),
            "bi_router_gemm_bf16_schedule": ([P, P, P, P, I64, I64, I64, I32, P], ST),
            "bi_router_topk_bf16": ([P, P, P, P, P, P, P, I64, I64, I64, I32, P], ST),
            "bi_router_topk_bf16_schedule": ([P, P, P, P, P, P, P, I64, I64, I64, I32, I32, P], ST),
            "bi_moe_forward_noalloc": ([P, P, P, P, P, P, I64, I64, I64, I32, I64, P], ST),
            "bi_fp32_fma_probe": ([P, I64, I32, P], ST),
            "bi_wait_timeout_probe": ([I32, P], ST),
            "bi_moe_gather_routing": ([P, P, P, P, P, P, I64, I64, I32, I64, P], ST),
            "bi_ffn_workspace_bytes": ([I64, I64, I64], SZ),
            "bi_ffn_forward": ([P, I64, P, P, P, I64, P, I64, I64, I64, I64, P, SZ, P], ST),
            "bi_ffn_forward_train": ([P, I64, P, P, P, I64, P, I64, P, P, I64, I64, I64, P], ST),
            "bi_ffn_backward": ([P, I64, P, I64, P, P, P, P, P, I64, P, P, I32, I64, I64, I64, P, SZ, P], ST),
            "bi_ffn_schedule": ([I32, P], ST),
            "bi_mx4_scale_bytes": ([I64, I64], SZ),
            "bi_mx4_quantize": ([P, I32, I64, P, P, I64, I64, P], ST),
            "bi_mx4_dequantize": ([P, P, P, I32, I64, I64, I64, P], ST),
            "bi_mx4_gemm": ([P, P, P, P, P, I64, P, I64, I64, I64, I64, P], ST),
            "bi_mx4_form": ([I32, P], ST),
            "bi_mx4_gate_up": ([P, P, P, P, P, I64, I64, I64, I64, P], ST),
            "bi_moe_scatter_contrib": ([P, P, P, P, I64, I64, I64, I32, P], ST),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
        return lib


def _call(name, *args):
    lib = load_library()
    st = getattr(lib, name)(*args)
    if st != BI_OK:
        raise BimoeError(name, st, lib.bi_last_error_message().decode())


def _ptr(t, dtype, name, device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on_stream(stream, f, *args):
    """f(*args) with ``stream`` current, for calls that allocate: what they allocate then comes from that
    stream's memory pool, which hands nothing to other work before the kernels launched here have run, and
    holds nothing that work pending on another stream still uses.  What f allocated and returns is also kept,
    once dropped, until the work that the caller has put on the current stream by then is done."""
    here = torch.cuda.current_stream(stream.device)
    if isinstance(args[0], torch.Tensor) and args[0].is_cuda and args[0].device != stream.device:
        raise ValueError(f"stream is on {stream.device}, expected {args[0].device}")
    with torch.cuda.stream(stream):
        out = f(*args)
    if here.cuda_stream != stream.cuda_stream:
        for t in out if isinstance(out, tuple) else (out,):
            if t is not None and not any(t is a for a in args):
                t.record_stream(here)
    return out


def device_error() -> int:
    """Read and clear the device error word (synchronises the device)."""
    lib = load_library()
    v = ctypes.c_int32(0)
    st = lib.bi_device_error(ctypes.byref(v))
    if st != BI_OK:
        raise BimoeError("bi_device_error", st, lib.bi_last_error_message().decode())
    return v.value


# ----------------------------------------------------------------- router --
def bi_cast_bf16_to_f32(x, out=None, stream=None):
    if stream is not None and out is None:
        return _on_stream(stream, bi_cast_bf16_to_f32, x)
    out = out if out is not None else torch.empty(x.shape, dtype=torch.float32, device=x.device)
    _call("bi_cast_bf16_to_f32", _ptr(x, torch.bfloat16, "x"), _ptr(out, torch.float32, "out", x.device),
          x.numel(), _stream(stream))
    return out


def bi_router_gemm(x, w, bias=None, out=None, schedule=0, stream=None):
    """y[M,N] = x[M,K] @ w[N,K]^T (+ bias), fp32, batch-invariant recipe.  x is
    fp32 or bf16 (bf16 values are read as their exact fp32 values)."""
    if stream is not None and out is None:
        return _on_stream(stream, bi_router_gemm, x, w, bias, None, schedule)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("w must be [N, K]")
    out = out if out is not None else torch.empty(M, N, dtype=torch.float32, device=x.device)
    if out.shape != (M, N):
        raise ValueError("out must be [M, N]")
    bf16 = x.dtype == torch.bfloat16
    args = (_ptr(x, torch.bfloat16 if bf16 else torch.float32, "x"), _ptr(w, torch.float32, "w", x.device),
            _ptr(bias, torch.float32, "bias", x.device), _ptr(out, torch.float32, "out", x.device),
            M, K, N)
    name = "bi_router_gemm_bf16" if bf16 else "bi_router_gemm"
    if schedule:
        _call(name + "_schedule", *args, schedule, _stream(stream))
    else:
        _call(name, *args, _stream(stream))
    return out


def bi_router_gemm_splitk_negctl(x, w, bias=None, out=None, stream=None):
    """Negative control (tests only): K split depends on M."""
    if stream is not None and out is None:
        return _on_stream(stream, bi_router_gemm_splitk_negctl, x, w, bias)
    M, K = x.shape
    N = w.shape[0]
    out = out if out is not None else torch.empty(M, N, dtype=torch.float32, device=x.device)
    _call("bi_router_gemm_splitk_negctl", _ptr(x, torch.float32, "x"),
          _ptr(w, torch.float32, "w", x.device), _ptr(bias, torch.float32, "bias", x.device),
          _ptr(out, torch.float32, "out", x.device), M, K, N, _stream(stream))
    return out


# ------------------------------------------------------------------ top-k --
def bi_topk(scores, top_k, ids=None, wts=None, probs=None, want_probs=False, stream=None):
    """(ids int32 [M,k], wts fp32 [M,k], probs fp32 [M,E] or None)."""
    if stream is not None and (ids is None or wts is None or (want_probs and probs is None)):
        return _on_stream(stream, bi_topk, scores, top_k, ids, wts, probs, want_probs)
    M, E = scores.shape
    dev = scores.device
    ids = ids if ids is not None else torch.empty(M, top_k, dtype=torch.int32, device=dev)
    wts = wts if wts is not None else torch.empty(M, top_k, dtype=torch.float32, device=dev)
    if want_probs and probs is None:
        probs = torch.empty(M, E, dtype=torch.float32, device=dev)
    _call("bi_topk", _ptr(scores, torch.float32, "scores"), _ptr(probs, torch.float32, "probs", dev),
          _ptr(ids, torch.int32, "ids", dev), _ptr(wts, torch.float32, "wts", dev),
          M, E, top_k, _stream(stream))
    return ids, wts, probs


# -------------------------------------------------------------------- MoE --
def bi_moe_workspace_bytes(M, H, E, top_k, I) -> int:
    return int(load_library().bi_moe_workspace_bytes(M, H, E, top_k, I))


def moe_workspace(M, H, E, top_k, I, device):
    n = bi_moe_workspace_bytes(M, H, E, top_k, I)
    if n == 0 and M > 0:
        raise ValueError("unsupported MoE sizes")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def bi_moe_forward(x, ids, wts, w13, w2, out=None, workspace=None, stream=None):
    """out[M,H] bf16 = batch-invariant SwiGLU MoE of x [M,H] bf16."""
    if stream is not None and (out is None or workspace is None):
        return _on_stream(stream, bi_moe_forward, x, ids, wts, w13, w2, out, workspace)
    M, H, E, I, top_k = _check_moe_shapes(x, ids, wts, w13, w2, out)
    dev = x.device
    out = out if out is not None else torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = moe_workspace(M, H, E, top_k, I, dev)
    _call("bi_moe_forward", _ptr(x, torch.bfloat16, "x"), _ptr(ids, torch.int32, "ids", dev),
          _ptr(wts, torch.float32, "wts", dev), _ptr(w13, torch.bfloat16, "w13", dev),
          _ptr(w2, torch.bfloat16, "w2", dev), _ptr(out, torch.bfloat16, "out", dev),
          M, H, E, top_k, I, _ptr(workspace, torch.uint8, "workspace", dev),
          workspace.numel(), _stream(stream))
    return out


def _check_moe_shapes(x, ids, wts, w13, w2, out):
    M, H = x.shape
    E, twoI, H2 = w13.shape
    I = twoI // 2
    if H2 != H or twoI % 2 or tuple(w2.shape) != (E, H, I):
        raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
    if ids.dim() != 2 or ids.shape[0] != M or tuple(wts.shape) != tuple(ids.shape):
        raise ValueError("ids and wts must be [M, top_k]")
    if out is not None and tuple(out.shape) != (M, H):
        raise ValueError("out must be [M, H]")
    return M, H, E, I, ids.shape[1]


def bi_moe_forward_noalloc(x, ids, wts, w13, w2, out=None, stream=None):
    """bi_moe_forward with the library's built-in scratch array instead of a
    caller workspace (for callers that cannot allocate device memory; the
    output tensor, if not given, is still allocated here by torch).  The call
    runs with x's device current, whose scratch array the library uses."""
    if stream is not None and out is None:
        return _on_stream(stream, bi_moe_forward_noalloc, x, ids, wts, w13, w2)
    M, H, E, I, top_k = _check_moe_shapes(x, ids, wts, w13, w2, out)
    dev = x.device
    if not x.is_cuda:
        raise ValueError("x must live on a CUDA device")
    with torch.cuda.device(dev):
        out = out if out is not None else torch.empty(M, H, dtype=torch.bfloat16, device=dev)
        if stream is not None and stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, expected {dev}")
        _call("bi_moe_forward_noalloc", _ptr(x, torch.bfloat16, "x"), _ptr(ids, torch.int32, "ids", dev),
              _ptr(wts, torch.float32, "wts", dev), _ptr(w13, torch.bfloat16, "w13", dev),
              _ptr(w2, torch.bfloat16, "w2", dev), _ptr(out, torch.bfloat16, "out", dev),
              M, H, E, top_k, I, _stream(stream))
    return out


def bi_moe_permute(ids, E, offsets=None, perm=None, workspace=None, stream=None):
    if stream is not None and (offsets is None or perm is None or workspace is None):
        return _on_stream(stream, bi_moe_permute, ids, E, offsets, perm, workspace)
    M, top_k = ids.shape
    dev = ids.device
    lib = load_library()
    offsets = offsets if offsets is not None else torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = perm if perm is not None else torch.empty(max(M * top_k, 1), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(int(lib.bi_moe_permute_workspace_bytes(M, E)), 256),
                                dtype=torch.uint8, device=dev)
    _call("bi_moe_permute", _ptr(ids, torch.int32, "ids"), _ptr(offsets, torch.int32, "offsets", dev),
          _ptr(perm, torch.int32, "perm", dev), M, E, top_k,
          _ptr(workspace, torch.uint8, "workspace", dev), workspace.numel(), _stream(stream))
    return offsets, perm


def bi_moe_gather(x, offsets, perm, top_k, x_perm=None, stream=None):
    """x_perm [M*top_k, H] bf16: token rows in expert order."""
    if stream is not None and x_perm is None:
        return _on_stream(stream, bi_moe_gather, x, offsets, perm, top_k)
    M, H = x.shape
    E = offsets.numel() - 1
    dev = x.device
    x_perm = x_perm if x_perm is not None else torch.empty(M * top_k, H, dtype=torch.bfloat16, device=dev)
    _call("bi_moe_gather", _ptr(x, torch.bfloat16, "x"), _ptr(offsets, torch.int32, "offsets", dev),
          _ptr(perm, torch.int32, "perm", dev), _ptr(x_perm, torch.bfloat16, "x_perm", dev),
          M, H, E, top_k, _stream(stream))
    return x_perm


def bi_moe_gate_up(x_perm, offsets, perm, wts, w13, top_k, act=None, stream=None):
    """act [M*top_k, I] bf16 from gathered rows x_perm [M*top_k, H]."""
    if stream is not None and act is None:
        return _on_stream(stream, bi_moe_gate_up, x_perm, offsets, perm, wts, w13, top_k)
    P, H = x_perm.shape
    M = P // top_k
    E, twoI, _ = w13.shape
    I = twoI // 2
    dev = x_perm.device
    act = act if act is not None else torch.empty(P, I, dtype=torch.bfloat16, device=dev)
    _call("bi_moe_gate_up", _ptr(x_perm, torch.bfloat16, "x_perm"),
          _ptr(offsets, torch.int32, "offsets", dev), _ptr(perm, torch.int32, "perm", dev),
          _ptr(wts, torch.float32, "wts", dev), _ptr(w13, torch.bfloat16, "w13", dev),
          _ptr(act, torch.bfloat16, "act", dev), M, H, E, top_k, I, _stream(stream))
    return act


def bi_moe_gate_up_tokens(x, offsets, perm, wts, w13, top_k, act=None, stream=None):
    """act [M*top_k, I] bf16, the gate/up GEMM gathering the token rows of
    x [M, H] itself (no gathered copy)."""
    if stream is not None and act is None:
        return _on_stream(stream, bi_moe_gate_up_tokens, x, offsets, perm, wts, w13, top_k)
    M, H = x.shape
    E, twoI, _ = w13.shape
    I = twoI // 2
    dev = x.device
    act = act if act is not None else torch.empty(M * top_k, I, dtype=torch.bfloat16, device=dev)
    _call("bi_moe_gate_up_tokens", _ptr(x, torch.bfloat16, "x"),
          _ptr(offsets, torch.int32, "offsets", dev), _ptr(perm, torch.int32, "perm", dev),
          _ptr(wts, torch.float32, "wts", dev), _ptr(w13, torch.bfloat16, "w13", dev),
          _ptr(act, torch.bfloat16, "act", dev), M, H, E, top_k, I, _stream(stream))
    return act


def bi_moe_gate_up_feed(mode):
    """How bi_moe_forward feeds the gate/up GEMM (0 automatic = the gathered
    copy, 1 gathered copy, 2 gathered by the GEMM); returns the previous
    setting."""
    prev = ctypes.c_int32(0)
    _call("bi_moe_gate_up_feed", int(mode), ctypes.byref(prev))
    return prev.value


def bi_moe_decode_fused(mode):
    """How bi_moe_layer runs a decode-sized batch's expert GEMMs (0 automatic
    = one launch where it applies, 1 = a gate/up and a down launch); returns
    the previous setting."""
    prev = ctypes.c_int32(0)
    _call("bi_moe_decode_fused", int(mode), ctypes.byref(prev))
    return prev.value


def bi_moe_down(act, offsets, perm, w2, M, top_k, contrib=None, stream=None):
    if stream is not None and contrib is None:
        return _on_stream(stream, bi_moe_down, act, offsets, perm, w2, M, top_k)
    E, H, I = w2.shape
    dev = act.device
    contrib = contrib if contrib is not None else torch.empty(M * top_k, H, dtype=torch.float32, device=dev)
    _call("bi_moe_down", _ptr(act, torch.bfloat16, "act"), _ptr(offsets, torch.int32, "offsets", dev),
          _ptr(perm, torch.int32, "perm", dev), _ptr(w2, torch.bfloat16, "w2", dev),
          _ptr(contrib, torch.float32, "contrib", dev), M, H, E, top_k, I, _stream(stream))
    return contrib


def bi_moe_gather_routing(ids, wts, offsets, perm, experts_per_rank, lid=None, pw=None, stream=None):
    """(lid int32 [M*top_k], pw fp32 [M*top_k]): for each permuted position,
    the expert's index on the rank that owns it and the routing probability."""
    if stream is not None and (lid is None or pw is None):
        return _on_stream(stream, bi_moe_gather_routing, ids, wts, offsets, perm, experts_per_rank, lid, pw)
    M, top_k = ids.shape
    E = offsets.numel() - 1
    dev = ids.device
    P = M * top_k
    lid = lid if lid is not None else torch.empty(max(P, 1), dtype=torch.int32, device=dev)
    pw = pw if pw is not None else torch.empty(max(P, 1), dtype=torch.float32, device=dev)
    _call("bi_moe_gather_routing", _ptr(ids, torch.int32, "ids"), _ptr(wts, torch.float32, "wts", dev),
          _ptr(offsets, torch.int32, "offsets", dev), _ptr(perm, torch.int32, "perm", dev),
          _ptr(lid, torch.int32, "lid", dev), _ptr(pw, torch.float32, "pw", dev), M, E, top_k,
          experts_per_rank, _stream(stream))
    return lid, pw


def bi_moe_scatter_contrib(rows, offsets, perm, M, top_k, contrib=None, stream=None):
    """contrib [M*top_k, H] fp32 with contrib[perm[p]] = rows[p] for p < offsets[E]."""
    if stream is not None and contrib is None:
        return _on_stream(stream, bi_moe_scatter_contrib, rows, offsets, perm, M, top_k)
    H = rows.shape[-1]
    E = offsets.numel() - 1
    dev = rows.device
    contrib = contrib if contrib is not None else torch.empty(M * top_k, H, dtype=torch.float32, device=dev)
    _call("bi_moe_scatter_contrib", _ptr(rows, torch.float32, "rows"), _ptr(offsets, torch.int32, "offsets", dev),
          _ptr(perm, torch.int32, "perm", dev), _ptr(contrib, torch.float32, "contrib", dev), M, H, E, top_k,
          _stream(stream))
    return contrib


def bi_moe_combine(contrib, M, top_k, out=None, stream=None):
    if stream is not None and out is None:
        return _on_stream(stream, bi_moe_combine, contrib, M, top_k)
    H = contrib.shape[-1]
    dev = contrib.device
    out = out if out is not None else torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    _call("bi_moe_combine", _ptr(contrib, torch.float32, "contrib"), _ptr(out, torch.bfloat16, "out", dev),
          M, H, top_k, _stream(stream))
    return out


def bi_moe_combine_consume(contrib, M, top_k, out=None, stream=None):
    """bi_moe_combine for a caller that never reads ``contrib`` again: its
    lines are dropped from L2 once summed, and its contents are indeterminate
    afterwards."""
    if stream is not None and out is None:
        return _on_stream(stream, bi_moe_combine_consume, contrib, M, top_k)
    H = contrib.shape[-1]
    dev = contrib.device
    out = out if out is not None else torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    _call("bi_moe_combine_consume", _ptr(contrib, torch.float32, "contrib"),
          _ptr(out, torch.bfloat16, "out", dev), M, H, top_k, _stream(stream))
    return out


def bi_router_topk(x, w, top_k, bias=None, out=None, want_probs=False, schedule=0, stream=None,
                   ids=None, wts=None):
    """Router scores and top-k selection in one call (the selection grid as a
    programmatic dependent of the router grid; schedule 10 forces the
    one-kernel cluster path for up to 4 rows, 1..9 a router schedule).  Returns
    (scores [M,N] fp32, ids [M,top_k] int32, wts [M,top_k] fp32, probs or None)."""
    if stream is not None and (out is None or ids is None or wts is None or want_probs):
        return _on_stream(stream, bi_router_topk, x, w, top_k, bias, out, want_probs, schedule, None, ids, wts)
    M, K = x.shape
    N = w.shape[0]
    dev = x.device
    y = out if out is not None else torch.empty(M, N, dtype=torch.float32, device=dev)
    ids = ids if ids is not None else torch.empty(M, top_k, dtype=torch.int32, device=dev)
    wts = wts if wts is not None else torch.empty(M, top_k, dtype=torch.float32, device=dev)
    if ids.shape != (M, top_k) or wts.shape != (M, top_k):
        raise ValueError("ids and wts must be [M, top_k]")
    probs = torch.empty(M, N, dtype=torch.float32, device=dev) if want_probs else None
    ptrs = (_ptr(w, torch.float32, "w", dev), _ptr(bias, torch.float32, "bias", dev),
            _ptr(y, torch.float32, "out", dev), _ptr(probs, torch.float32, "probs", dev),
            _ptr(ids, torch.int32, "ids", dev), _ptr(wts, torch.float32, "wts", dev))
    if x.dtype == torch.bfloat16:
        _call("bi_router_topk_bf16_schedule", _ptr(x, torch.bfloat16, "x"), *ptrs, M, K, N, top_k, schedule,
              _stream(stream))
    else:
        _call("bi_router_topk_schedule", _ptr(x, torch.float32, "x"), *ptrs, M, K, N, top_k, schedule,
              _stream(stream))
    return y, ids, wts, probs


def bi_topk_window(scores, k, row_start=None, row_end=None, num_cols=None, out=None, stream=None):
    """Windowed per-row top-k: int32 [n_rows, k] window-relative columns of
    the k best in-window scores, ascending, -1 tail.  scores is fp32
    [n_rows, ld] with unit column stride (row stride ld >= num_cols)."""
    if stream is not None and out is None:
        return _on_stream(stream, bi_topk_window, scores, k, row_start, row_end, num_cols)
    if scores.dim() != 2 or scores.stride(1) != 1:
        raise ValueError("scores must be 2-D with unit column stride")
    n_rows = scores.shape[0]
    ld = scores.stride(0) if n_rows > 1 else scores.shape[1]
    num_cols = scores.shape[1] if num_cols is None else num_cols
    dev = scores.device
    if scores.dtype != torch.float32 or not scores.is_cuda:
        raise TypeError("scores must be a CUDA float32 tensor")
    out = out if out is not None else torch.empty(n_rows, k, dtype=torch.int32, device=dev)
    _call("bi_topk_window", ctypes.c_void_p(scores.data_ptr()), ld,
          _ptr(row_start, torch.int64, "row_start", dev), _ptr(row_end, torch.int64, "row_end", dev),
          n_rows, num_cols, k, _ptr(out, torch.int32, "out", dev), _stream(stream))
    return out


def bi_moe_gemm_variant(variant):
    """Select the expert-GEMM schedule for the process (0 automatic, 1 one CTA
    per tile, 2 CTA pairs, 3 CTA pairs with interleaved gate/up rows for the
    gate/up GEMM, 4 one CTA per tile with interleaved gate/up rows); returns
    the previous setting."""
    prev = ctypes.c_int32(0)
    _call("bi_moe_gemm_variant", int(variant), ctypes.byref(prev))
    return prev.value


def bi_fp32_fma_probe(blocks, iters, stream=None, out=None):
    """Run the FP32 FMA throughput probe; returns its output tensor."""
    if stream is not None and out is None:
        return _on_stream(stream, bi_fp32_fma_probe, blocks, iters)
    if out is None:
        out = torch.empty(blocks * 256, dtype=torch.float32, device="cuda")
    elif out.numel() < blocks * 256:
        raise ValueError("out holds fewer than blocks * 256 floats")
    _call("bi_fp32_fma_probe", _ptr(out, torch.float32, "out"), blocks, iters, _stream(stream))
    return out


def bi_wait_timeout_probe(which=0, stream=None):
    """Test use only: a kernel whose bounded wait runs out (about one second):
    which = 0 the mbarrier wait, 1 the arrival-count wait; read the recorded
    BI_DEVERR_WAIT_TIMEOUT with device_error()."""
    _call("bi_wait_timeout_probe", int(which), _stream(stream))


def bi_moe_layer(x, w_router, w13, w2, top_k, bias=None, out=None, scores=None, ids=None, wts=None,
                 workspace=None, stream=None):
    """Whole hot path of one MoE layer in one library call: router (on the
    bf16 tokens, read as their exact fp32 values) -> top-k -> experts.
    Returns (out, scores, ids, wts)."""
    if stream is not None and any(t is None for t in (out, scores, ids, wts, workspace)):
        return _on_stream(stream, bi_moe_layer, x, w_router, w13, w2, top_k, bias, out, scores, ids, wts,
                          workspace)
    M, H = x.shape
    E, H2 = w_router.shape
    if H2 != H:
        raise ValueError("w_router must be [E, H]")
    dev = x.device
    ids = ids if ids is not None else torch.empty(M, top_k, dtype=torch.int32, device=dev)
    wts = wts if wts is not None else torch.empty(M, top_k, dtype=torch.float32, device=dev)
    _, _, _, I, _ = _check_moe_shapes(x, ids, wts, w13, w2, out)
    if w13.shape[0] != E:
        raise ValueError("w_router, w13 and w2 must have the same number of experts")
    out = out if out is not None else torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    scores = scores if scores is not None else torch.empty(M, E, dtype=torch.float32, device=dev)
    if tuple(scores.shape) != (M, E):
        raise ValueError("scores must be [M, E]")
    if workspace is None:
        workspace = moe_workspace(M, H, E, top_k, I, dev)
    _call("bi_moe_layer", _ptr(x, torch.bfloat16, "x"), _ptr(w_router, torch.float32, "w_router", dev),
          _ptr(bias, torch.float32, "bias", dev), _ptr(w13, torch.bfloat16, "w13", dev),
          _ptr(w2, torch.bfloat16, "w2", dev), _ptr(out, torch.bfloat16, "out", dev),
          _ptr(scores, torch.float32, "scores", dev), _ptr(ids, torch.int32, "ids", dev),
          _ptr(wts, torch.float32, "wts", dev), M, H, E, top_k, I,
          _ptr(workspace, torch.uint8, "workspace", dev), workspace.numel(), _stream(stream))
    return out, scores, ids, wts


def moe_layer(x_bf16, w_router, w13, w2, top_k, bias=None, stream=None):
    """Whole hot path of one MoE layer (bi_moe_layer).  Returns (out, scores,
    ids, wts)."""
    return bi_moe_layer(x_bf16, w_router, w13, w2, top_k, bias=bias, stream=stream)


# ------------------------------------ dense gated feed-forward block --
_BF, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream
_fns = {}


_current_device = torch._C._cuda_getDevice


def _bind(name):
    f = _fns[name] = getattr(load_library(), name)
    return f


def _fail(name, status):
    raise BimoeError(name, status, load_library().bi_last_error_message().decode())


def _device_of(t, name):
    """Device number of a CUDA tensor (checked once per call, the other tensors against it)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    return t.get_device()


def _flat(t, dtype, name, device):
    """Address of a contiguous tensor on device number ``device``."""
    if t.dtype is dtype and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    return _ptr(t, dtype, name, torch.device("cuda", device)).value  # says what is wrong


def _rows(t, dtype, name, rows, cols, device):
    """(address, row stride) of a [rows, cols] tensor with unit column stride on device number ``device``."""
    if t.dtype is dtype and t.get_device() == device and t.shape == (rows, cols) and t.is_contiguous():
        return t.data_ptr(), cols
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {[rows, cols]}, got {list(t.shape)}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), (t.stride(0) if rows > 1 else cols)


def _check_ffn_shapes(x, w13, w2):
    if x.dim() != 2 or w13.dim() != 2 or w2.dim() != 2:
        raise ValueError("x, w13 and w2 must be 2-D")
    M, H = x.shape
    H2, I = w2.shape
    if w13.shape != (2 * I, H) or H2 != H:
        raise ValueError("w13 must be [2I, H] and w2 [H, I]")
    return M, H, I


def ffn_workspace(M, H, I, device):
    """Workspace of bi_ffn_forward and bi_ffn_backward at these sizes."""
    n = int(load_library().bi_ffn_workspace_bytes(M, H, I))
    if n == 0:
        raise ValueError("unsupported feed-forward sizes: " + load_library().bi_last_error_message().decode())
    return torch.empty(n, dtype=_U8, device=device)


def ffn_saved(M, I, device):
    """(gu fp32 [M, 2I], act bf16 [M, I]): what bi_ffn_forward_train keeps for bi_ffn_backward."""
    return torch.empty(M, 2 * I, dtype=_F32, device=device), torch.empty(M, I, dtype=_BF, device=device)


def bi_ffn_forward(x, w13, w2, addend=None, out=None, workspace=None, stream=None):
    """out [M,H] bf16 = (silu(x Wg^T) * (x Wu^T)) W2^T (+ addend), w13 [2I,H] = [Wg; Wu],
    w2 [H,I]; x, addend and out may be rows of wider tensors (row stride a multiple of 8)."""
    if stream is not None and (out is None or workspace is None):
        return _on_stream(stream, bi_ffn_forward, x, w13, w2, addend, out, workspace)
    M, H, I = _check_ffn_shapes(x, w13, w2)
    dev = _device_of(x, "x")
    px, ldx = _rows(x, _BF, "x", M, H, dev)
    pa, lda = _rows(addend, _BF, "addend", M, H, dev) if addend is not None else (None, 0)
    if out is None:
        out = torch.empty(M, H, dtype=_BF, device=x.device)
    po, ldo = _rows(out, _BF, "out", M, H, dev)
    if workspace is None:
        workspace = ffn_workspace(M, H, I, x.device)
    if dev != _current_device():  # the call runs with the tensors' device current
        with torch.cuda.device(dev):
            return bi_ffn_forward(x, w13, w2, addend, out, workspace, stream)
    f = _fns.get("bi_ffn_forward") or _bind("bi_ffn_forward")
    st = f(px, ldx, _flat(w13, _BF, "w13", dev), _flat(w2, _BF, "w2", dev), pa, lda, po, ldo, M, H, I,
           _flat(workspace, _U8, "workspace", dev), workspace.numel(),
           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _fail("bi_ffn_forward", st)
    return out


def bi_ffn_forward_train(x, w13, w2, addend=None, out=None, gu=None, act=None, stream=None):
    """bi_ffn_forward that keeps what bi_ffn_backward reads.  Returns (out, gu fp32 [M,2I], act bf16 [M,I])."""
    if stream is not None and (out is None or gu is None or act is None):
        return _on_stream(stream, bi_ffn_forward_train, x, w13, w2, addend, out, gu, act)
    M, H, I = _check_ffn_shapes(x, w13, w2)
    dev = _device_of(x, "x")
    px, ldx = _rows(x, _BF, "x", M, H, dev)
    pa, lda = _rows(addend, _BF, "addend", M, H, dev) if addend is not None else (None, 0)
    if out is None:
        out = torch.empty(M, H, dtype=_BF, device=x.device)
    po, ldo = _rows(out, _BF, "out", M, H, dev)
    if gu is None:
        gu = torch.empty(M, 2 * I, dtype=_F32, device=x.device)
    if act is None:
        act = torch.empty(M, I, dtype=_BF, device=x.device)
    if gu.shape != (M, 2 * I) or act.shape != (M, I):
        raise ValueError("gu must be [M, 2I] and act [M, I]")
    if dev != _current_device():  # the call runs with the tensors' device current
        with torch.cuda.device(dev):
            return bi_ffn_forward_train(x, w13, w2, addend, out, gu, act, stream)
    f = _fns.get("bi_ffn_forward_train") or _bind("bi_ffn_forward_train")
    st = f(px, ldx, _flat(w13, _BF, "w13", dev), _flat(w2, _BF, "w2", dev), pa, lda, po, ldo,
           _flat(gu, _F32, "gu", dev), _flat(act, _BF, "act", dev), M, H, I,
           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _fail("bi_ffn_forward_train", st)
    return out, gu, act


def bi_ffn_backward(dout, x, w13, w2, gu, act, dx=None, dw13=None, dw2=None, need=(True, True, True),
                    accumulate=False, workspace=None, stream=None):
    """(dx, dw13, dw2) from dout [M,H]; None for each that ``need`` does not ask for.  dw13 and dw2
    are bf16 (the default) or both fp32; with ``accumulate`` the gradients are added to the fp32
    tensors given."""
    if stream is not None and (workspace is None or any(n and t is None for n, t in zip(need, (dx, dw13, dw2)))):
        return _on_stream(stream, bi_ffn_backward, dout, x, w13, w2, gu, act, dx, dw13, dw2, need, accumulate,
                          workspace)
    M, H, I = _check_ffn_shapes(x, w13, w2)
    dev = _device_of(x, "x")
    px, ldx = _rows(x, _BF, "x", M, H, dev)
    pdo, lddo = _rows(dout, _BF, "dout", M, H, dev)
    if gu.shape != (M, 2 * I) or act.shape != (M, I):
        raise ValueError("gu must be [M, 2I] and act [M, I]")
    wd = next((t.dtype for t, n in ((dw13, need[1]), (dw2, need[2])) if n and t is not None), _BF)
    if wd not in (_BF, _F32):
        raise TypeError(f"dw13 and dw2 must be bfloat16 or float32, got {wd}")
    if accumulate and (wd != _F32 or (need[1] and dw13 is None) or (need[2] and dw2 is None)):
        raise ValueError("accumulate needs the fp32 tensors that the gradients are added to")
    pdx = p13 = p2 = None
    lddx = 0
    if need[0]:
        if dx is None:
            dx = torch.empty(M, H, dtype=_BF, device=x.device)
        pdx, lddx = _rows(dx, _BF, "dx", M, H, dev)
    if need[1]:
        if dw13 is None:
            dw13 = torch.empty(2 * I, H, dtype=wd, device=x.device)
        if dw13.shape != (2 * I, H):
            raise ValueError("dw13 must be [2I, H]")
        p13 = _flat(dw13, wd, "dw13", dev)
    if need[2]:
        if dw2 is None:
            dw2 = torch.empty(H, I, dtype=wd, device=x.device)
        if dw2.shape != (H, I):
            raise ValueError("dw2 must be [H, I]")
        p2 = _flat(dw2, wd, "dw2", dev)
    if workspace is None:
        workspace = ffn_workspace(M, H, I, x.device)
    mode = 0 if wd is _BF else (2 if accumulate else 1)
    if dev != _current_device():  # the call runs with the tensors' device current
        with torch.cuda.device(dev):
            return bi_ffn_backward(dout, x, w13, w2, gu, act, dx, dw13, dw2, need, accumulate, workspace, stream)
    f = _fns.get("bi_ffn_backward") or _bind("bi_ffn_backward")
    st = f(pdo, lddo, px, ldx, _flat(w13, _BF, "w13", dev), _flat(w2, _BF, "w2", dev),
           _flat(gu, _F32, "gu", dev), _flat(act, _BF, "act", dev), pdx, lddx, p13, p2, mode, M, H, I,
           _flat(workspace, _U8, "workspace", dev), workspace.numel(),
           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _fail("bi_ffn_backward", st)
    return dx if need[0] else None, dw13 if need[1] else None, dw2 if need[2] else None


def bi_ffn_schedule(mode):
    """Which kernel runs the feed-forward products over tokens (0 automatic, 1 CTA pairs, 2 slices over a
    cluster); returns the previous setting."""
    prev = ctypes.c_int32(0)
    _call("bi_ffn_schedule", int(mode), ctypes.byref(prev))
    return prev.value


# ------------------------------------ microscaled 4-bit floating point --
def mx4_scale_shape(R, K):
    """Shape of the scale tiles of an [R, K] matrix."""
    return ((R + 127) // 128, (K + 127) // 128, 512)


def mx4_empty(R, K, device):
    """(codes uint8 [R, K/2], scale tiles uint8): uninitialised buffers for bi_mx4_quantize."""
    return (torch.empty(R, K // 2, dtype=_U8, device=device),
            torch.empty(mx4_scale_shape(R, K), dtype=_U8, device=device))


def mx4_tile_scales(s):
    """Row-major E8M0 scales uint8 [R, K/32] (as checkpoints hold them) in the tiled layout."""
    R, n = s.shape
    rt, kt = (R + 127) // 128, (n + 3) // 4
    p = torch.zeros(rt * 128, kt * 4, dtype=_U8, device=s.device)
    p[:R, :n] = s
    return p.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(rt, kt, 512).contiguous()


def mx4_untile_scales(t, R, K):
    """The inverse of mx4_tile_scales: uint8 [R, K/32]."""
    rt, kt, _ = t.shape
    return t.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:R, :K // 32].contiguous()


def mx4_interleave_gate_up(w13):
    """Rows of w13 [2I, ...] = [Wg; Wu] in the order bi_mx4_gate_up wants: 16 gate rows, their 16 up rows, ..."""
    if w13.shape[0] % 32:
        raise ValueError("w13 must have 2I rows, I a multiple of 16")
    I = w13.shape[0] // 2
    return w13.view(2, I // 16, 16, *w13.shape[1:]).transpose(0, 1).reshape(w13.shape).contiguous()


def _mx4_operand(q, s, name, device):
    """(addresses, rows, K) of a quantised matrix on device number ``device``."""
    R, half = q.shape
    # the common case in one condition; otherwise find out what is wrong
    if not (q.dtype is _U8 and s.dtype is _U8 and q.get_device() == device and s.get_device() == device
            and q.is_contiguous() and s.is_contiguous() and s.shape == ((R + 127) >> 7, (half + 63) >> 6, 512)):
        _flat(q, _U8, name + " codes", device)
        _flat(s, _U8, name + " scales", device)
        raise ValueError(f"{name} scales must be {list(mx4_scale_shape(R, 2 * half))}, got {list(s.shape)}")
    return q.data_ptr(), s.data_ptr(), R, 2 * half


def bi_mx4_quantize(x, q=None, scales=None, stream=None):
    """(codes, scale tiles) of x [R,K], bf16 or fp32, K a multiple of 32; x may be rows of a wider tensor."""
    if stream is not None and (q is None or scales is None):
        return _on_stream(stream, bi_mx4_quantize, x, q, scales)
    if x.dim() != 2:
        raise ValueError("x must be [R, K]")
    R, K = x.shape
    if K % 32:
        raise ValueError("K must be a multiple of 32")
    dev = _device_of(x, "x")
    f32 = x.dtype is _F32
    px, ldx = _rows(x, _F32 if f32 else _BF, "x", R, K, dev)
    if q is None or scales is None:
        nq, ns = mx4_empty(R, K, x.device)
        q, scales = nq if q is None else q, ns if scales is None else scales
    pq, ps, R2, K2 = _mx4_operand(q, scales, "q", dev)
    if R2 != R or K2 != K:
        raise ValueError("q must be [R, K/2]")
    if dev != _current_device():  # the call runs with the tensors' device current
        with torch.cuda.device(dev):
            return bi_mx4_quantize(x, q, scales, stream)
    f = _fns.get("bi_mx4_quantize") or _bind("bi_mx4_quantize")
    st = f(px, f32, ldx, pq, ps, R, K,
           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _fail("bi_mx4_quantize", st)
    return q, scales


def bi_mx4_dequantize(q, scales, out=None, dtype=torch.bfloat16, stream=None):
    """The values [R,K] (bf16 or fp32, both exact) that codes and scale tiles stand for."""
    if stream is not None and out is None:
        return _on_stream(stream, bi_mx4_dequantize, q, scales, out, dtype)
    dev = _device_of(q, "q codes")
    pq, ps, R, K = _mx4_operand(q, scales, "q", dev)
    if out is None:
        out = torch.empty(R, K, dtype=dtype, device=q.device)
    f32 = out.dtype is _F32
    po, ldo = _rows(out, _F32 if f32 else _BF, "out", R, K, dev)
    if dev != _current_device():  # the call runs with the tensors' device current
        with torch.cuda.device(dev):
            return bi_mx4_dequantize(q, scales, out, dtype, stream)
    f = _fns.get("bi_mx4_dequantize") or _bind("bi_mx4_dequantize")
    st = f(pq, ps, po, f32, ldo, R, K,
           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _fail("bi_mx4_dequantize", st)
    return out


def bi_mx4_gemm(xq, xs, wq, ws, addend=None, out=None, stream=None):
    """out [M,N] bf16 = X W^T (+ addend) of two quantised matrices X [M,K], W [N,K]."""
    if stream is not None and out is None:
        return _on_stream(stream, bi_mx4_gemm, xq, xs, wq, ws, addend, out)
    dev = _device_of(xq, "x codes")
    px, pxs, M, K = _mx4_operand(xq, xs, "x", dev)
    pw, pws, N, K2 = _mx4_operand(wq, ws, "w", dev)
    if K2 != K:
        raise ValueError("x and w must have the same K")
    pa, lda = _rows(addend, _BF, "addend", M, N, dev) if addend is not None else (None, 0)
    if out is None:
        out = torch.empty(M, N, dtype=_BF, device=xq.device)
    po, ldo = _rows(out, _BF, "out", M, N, dev)
    if dev != _current_device():  # the call runs with the tensors' device current
        with torch.cuda.device(dev):
            return bi_mx4_gemm(xq, xs, wq, ws, addend, out, stream)
    f = _fns.get("bi_mx4_gemm") or _bind("bi_mx4_gemm")
    st = f(px, pxs, pw, pws, pa, lda, po, ldo, M, N, K,
           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _fail("bi_mx4_gemm", st)
    return out


def bi_mx4_gate_up(xq, xs, w13q, w13s, out=None, stream=None):
    """act [M,I] bf16 = silu(X Wg^T) * (X Wu^T), the weight's rows interleaved by mx4_interleave_gate_up
    before they were quantised."""
    if stream is not None and out is None:
        return _on_stream(stream, bi_mx4_gate_up, xq, xs, w13q, w13s, out)
    dev = _device_of(xq, "x codes")
    px, pxs, M, K = _mx4_operand(xq, xs, "x", dev)
    pw, pws, N, K2 = _mx4_operand(w13q, w13s, "w13", dev)
    if K2 != K or N % 32:
        raise ValueError("x and w13 must have the same K, and w13 2I rows, I a multiple of 16")
    if out is None:
        out = torch.empty(M, N // 2, dtype=_BF, device=xq.device)
    po, ldo = _rows(out, _BF, "out", M, N // 2, dev)
    if dev != _current_device():  # the call runs with the tensors' device current
        with torch.cuda.device(dev):
            return bi_mx4_gate_up(xq, xs, w13q, w13s, out, stream)
    f = _fns.get("bi_mx4_gate_up") or _bind("bi_mx4_gate_up")
    st = f(px, pxs, pw, pws, po, ldo, M, N // 2, K,
           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _fail("bi_mx4_gate_up", st)
    return out


def bi_mx4_form(mode):
    """Which form of the kernel runs the 4-bit products (0 automatic, 1 single CTAs, 2 CTA pairs with 192 tokens
    a tile, 3 CTA pairs with 256); returns the previous setting."""
    prev = ctypes.c_int32(0)
    _call("bi_mx4_form", int(mode), ctypes.byref(prev))
    return prev.value
