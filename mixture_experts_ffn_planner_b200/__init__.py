"""Python binding of the B200 fused MoE expert-FFN forward (``libmoe_ffn.so``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/moe_ffn.h``.  PyTorch supplies
device memory and streams.  There is no CPU or PyTorch fallback: if the
library cannot be built or loaded, every call raises.

Entry points (same names as the C ABI):

* ``moe_align`` -- routing planner: expert histogram, prefix sums over counts
  padded to ``block_m``, and the row-to-token map ("[RFC] Fused W8A8 MoE
  megakernel on H20", Design; "Prime Flash MoE: Fused MoE Kernels for
  Blackwell", API / Shapes).
* ``moe_route_align`` -- the router ahead of the planner: softmax over the
  experts, top-k, renormalised weights, then the planner on the kept ids
  ("Prime Flash MoE", Usage; "[RFC] Fused W8A8 MoE megakernel on H20",
  Results so far).
* ``fused_moe_bf16`` / ``fused_moe_mxfp8`` -- gather, gate/up GEMM, SwiGLU
  (mxfp8: on-chip requant of the intermediate), down GEMM and the top-k
  weighted reduction into ``out`` ("Prime Flash MoE", intro / API / Shapes).
* ``fused_moe_mxfp4`` -- the mxfp8 forward with MXFP4 (e2m1) weights, two
  values per byte (DeepGEMM #411 "SM90 FP8 x MXFP4 MegaMoE" operand pairing).
* ``pack_scales_blocked`` -- weight scales into 512-byte tiles of
  128 MN x 128 K ("Prime Flash MoE", Scale layout (mxfp8)).
* ``moe_ep_dispatch_plan`` / ``moe_ep_dispatch_pack`` / ``moe_ep_combine`` --
  the device work around an expert-parallel exchange (DeepGEMM #411 "SM90 FP8
  x MXFP4 MegaMoE", Summary: dispatch, routed experts, combine).
* ``moe_permute`` / ``moe_unpermute`` and their ``_backward`` -- a training
  step's token rows in the planner's order and back (weighted sum over a
  token's routes), with the gradients; ``moe_route_slots`` inverts the
  planner's order for them.
* ``moe_expert_up`` / ``moe_expert_down`` and their ``_backward`` -- the
  experts' products on those rows and the gradients by rows and by weights.
* ``moe_orthogonalize`` -- the experts' weight update made nearly orthogonal
  by Newton-Schulz steps.

The training calls (from ``moe_route_slots`` on) are plain functions on tensors:
autograd records none of them, and their results require no gradient, whatever
their inputs do.  A gradient is what the ``_backward`` call returns; a layer in
an autograd graph wraps each pair in a ``torch.autograd.Function``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

from . import _build

__all__ = [
    "MoeError", "load", "moe_align", "moe_align_capacity", "moe_route_align", "fused_moe_bf16", "fused_moe_mxfp8",
    "fused_moe_mxfp4", "DTYPE_MXFP4",
    "pack_scales_blocked", "pack_scales_blocked_bytes", "moe_workspace_bytes", "moe_device_status",
    "Tuning", "DTYPE_BF16", "DTYPE_MXFP8", "LIB_PATH", "fused_moe_bf16_noalloc",
    "fused_moe_bf16_noalloc_max_workspace", "moe_ep_dispatch_plan", "moe_ep_dispatch_pack", "moe_ep_combine",
    "moe_route_slots", "moe_permute", "moe_permute_backward", "moe_unpermute", "moe_unpermute_backward",
    "moe_expert_up", "moe_expert_down", "moe_expert_down_backward", "moe_expert_up_backward",
    "moe_orthogonalize", "moe_orthogonalize_workspace_bytes",
]

DTYPE_BF16 = 0
DTYPE_MXFP8 = 1
DTYPE_MXFP4 = 2
LIB_PATH = _build.LIB

_ERRORS = {-1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED", -3: "MOE_ERR_ALIGNMENT",
           -4: "MOE_ERR_WORKSPACE", -5: "MOE_ERR_CUDA", -6: "MOE_ERR_TIMEOUT"}


class MoeError(RuntimeError):
    """A C-ABI call returned a negative status."""

    def __init__(self, code: int, message: str):
        self.code = int(code)
        self.name = _ERRORS.get(self.code, f"status {code}")
        super().__init__(f"{self.name}: {message}")


class Tuning(ctypes.Structure):
    """``moe_tuning``: 0 in a field keeps the library's default."""
    _fields_ = [("stages", ctypes.c_int), ("num_ctas", ctypes.c_int),
                ("phase_events", ctypes.POINTER(ctypes.c_void_p)), ("wait_timeout_ns", ctypes.c_longlong),
                ("small_batch", ctypes.c_int)]

    @staticmethod
    def with_events(events, stages: int = 0, num_ctas: int = 0) -> "Tuning":
        """Tuning whose timing hook records the four given torch.cuda.Event objects."""
        for e in events:
            e.record()  # forces creation of the underlying cudaEvent_t
        arr = (ctypes.c_void_p * 4)(*[e.cuda_event for e in events])
        t = Tuning(stages, num_ctas, ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)))
        t._keep = arr
        return t


_lock = threading.Lock()
_lib = None
_dtypes = {}  # torch's types by short name, once the library is loaded

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float

_SIGS = {
    "moe_last_error": ([], ctypes.c_char_p),
    "moe_device_status": ([_P], _I),
    "moe_align_capacity": ([_I, _I, _I, _I], _I64),
    "moe_align": ([_P, _I, _I, _I, _I, _P, _P, _P, _I64, _P], _I),
    "moe_route_align": ([_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _I64, _P], _I),
    "pack_scales_blocked_bytes": ([_I, _I, _I], _I64),
    "pack_scales_blocked": ([_P, _P, _I, _I, _I, _P], _I),
    "moe_workspace_bytes": ([_I, _I, _I, _I, _I, _I, _I], _I64),
    "fused_moe_bf16": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I64, _P, _I64, _P, _P], _I),
    "fused_moe_mxfp8": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I64, _P, _I64,
                         _P, _P], _I),
    "fused_moe_mxfp4": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I64, _P, _I64,
                         _P, _P], _I),
    "fused_moe_bf16_noalloc_max_workspace": ([], _I64),
    "moe_ep_dispatch_plan": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "moe_ep_dispatch_pack": ([_P, _I64, _P, _I64, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "moe_ep_combine": ([_P, _P, _I, _I, _I, _I, _P, _P, _P], _I),
    "fused_moe_bf16_noalloc": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I64, _P, _P], _I),
    "moe_route_slots": ([_P, _P, _I64, _I, _I, _P, _P], _I),
    "moe_permute": ([_P, _I, _P, _P, _P, _I64, _I, _I, _I, _P, _P], _I),
    "moe_permute_backward": ([_P, _I, _P, _I64, _I, _I, _I, _P, _P], _I),
    "moe_unpermute": ([_P, _I, _P, _P, _I64, _I, _I, _I, _P, _P], _I),
    "moe_orthogonalize_workspace_bytes": ([_I, _I, _I], _I64),
    "moe_orthogonalize": ([_P, _I, _I, _I, _I, _I, _F, _F, _F, _F, _P, _P, _I64, _P], _I),
    "moe_expert_up": ([_P, _P, _P, _P, _P, _I64, _I, _I, _I, _I, _P, _P, _P], _I),
    "moe_expert_down": ([_P, _P, _P, _P, _P, _I64, _I, _I, _I, _I, _P, _P], _I),
    "moe_expert_down_backward": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I, _I, _I, _I, _P, _P, _I, _I, _P], _I),
    "moe_expert_up_backward": ([_P, _P, _P, _P, _P, _P, _I64, _I, _I, _I, _I, _P, _P, _I, _I, _P], _I),
    "moe_unpermute_backward": ([_P, _P, _I, _P, _P, _P, _P, _I64, _I, _I, _I, _P, _P, _P], _I),
}


def load(build_if_stale: bool = True) -> ctypes.CDLL:
    """Loads libmoe_ffn.so (compiling it first if a source is newer)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if build_if_stale and _build.stale():
            try:
                _build.build()
            except Exception as exc:  # no toolchain: use the library that is there, if any
                if not os.path.exists(_build.LIB):
                    raise ImportError(f"libmoe_ffn.so is missing and could not be built: {exc}") from exc
        if not os.path.exists(_build.LIB):
            raise ImportError(f"libmoe_ffn.so not found at {_build.LIB}; run __graft_entry__.build()")
        lib = ctypes.CDLL(_build.LIB)
        for name, (args, res) in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        import torch

        _dtypes.update(i32=torch.int32, f32=torch.float32, bf16=torch.bfloat16)
        _lib = lib
        return lib


def _check(rc: int):
    if rc != 0:
        msg = load().moe_last_error()
        raise MoeError(rc, msg.decode() if msg else "")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


@contextlib.contextmanager
def _on_device(dev, stream):
    """Makes ``dev`` (the device of the call's tensors) the current CUDA device
    for the C call and yields the stream handle to launch on.

    The library launches on the current device and builds its TMA descriptors
    from the tensors' addresses, so a call whose tensors live on another
    device than the current one would read that device's memory from the
    wrong GPU.  ``stream``: None (the current stream of ``dev``), a
    ``torch.cuda.Stream`` (must belong to ``dev``) or a raw ``cudaStream_t``
    handle as an int (the caller vouches for its device)."""
    import torch

    if getattr(dev, "type", None) != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {dev}")
    with torch.cuda.device(dev):
        if stream is None:
            handle = torch.cuda.current_stream(dev).cuda_stream
        elif hasattr(stream, "cuda_stream"):
            sdev = getattr(stream, "device", dev)
            if torch.device(sdev) != torch.device(dev):
                raise ValueError(f"stream belongs to {sdev} but the tensors are on {dev}")
            handle = stream.cuda_stream
        else:
            handle = int(stream)
        yield handle


def _need(t, name, dtypes, device=True):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _ffn_shapes(fmt: str, x, w1, w2, topk_weights, out, sorted_token_ids, expert_ids, num_tokens_post_padded,
                block_m: int, x_scales=None, w1_scales=None, w2_scales=None):
    """The C ABI takes its sizes from x and w1 and trusts every other buffer, so the shapes (and the
    device) of all of them are checked here before a launch: a short buffer would be read or written
    out of bounds by the kernels.  fmt: "bf16", "mxfp8" or "mxfp4" (packed weights, two per byte)."""
    if x.dim() != 2 or w1.dim() != 3:
        raise ValueError("x must be (T, K) and w1 (E, N, K)")
    T, K = x.shape
    E, N = w1.shape[0], w1.shape[1]
    pack = 2 if fmt == "mxfp4" else 1
    if N % 2:
        raise ValueError(f"N = {N} must be even (gate and up halves)")
    want = {"w1": (E, N, K // pack), "w2": (E, K, N // 2 // pack), "out": (T, K)}
    for name, t in (("w1", w1), ("w2", w2), ("out", out)):
        if tuple(t.shape) != want[name]:
            raise ValueError(f"{name} must have shape {want[name]}, got {tuple(t.shape)}")
    if topk_weights.dim() != 2 or topk_weights.shape[0] != T:
        raise ValueError(f"topk_weights must be (T={T}, top_k), got {tuple(topk_weights.shape)}")
    if expert_ids.numel() < (sorted_token_ids.numel() + block_m - 1) // block_m or num_tokens_post_padded.numel() < 1:
        raise ValueError("expert_ids must hold ceil(sorted_token_ids.numel() / block_m) entries and "
                         "num_tokens_post_padded one")
    tensors = [w1, w2, out, topk_weights, sorted_token_ids, expert_ids, num_tokens_post_padded]
    if fmt != "bf16":
        if tuple(x_scales.shape) != (T, K // 32):
            raise ValueError(f"x_scales must have shape {(T, K // 32)}, got {tuple(x_scales.shape)}")
        for name, t, mn, ks in (("w1_scales_blocked", w1_scales, N, K // 32),
                                ("w2_scales_blocked", w2_scales, K, N // 2 // 32)):
            need = pack_scales_blocked_bytes(E, mn, ks)
            if t.numel() < need:
                raise ValueError(f"{name} must hold {need} bytes (pack_scales_blocked of ({E}, {mn}, {ks}))")
        tensors += [x_scales, w1_scales, w2_scales]
    for t in tensors:
        if t.device != x.device:
            raise ValueError(f"all tensors must be on {x.device}, got one on {t.device}")


def _same_device(first, *rest):
    for t in rest:
        if t.device != first.device:
            raise ValueError(f"all tensors must be on {first.device}, got one on {t.device}")


# ---------------------------------------------------------------- sizes
def moe_align_capacity(T: int, top_k: int, E: int, block_m: int) -> int:
    return int(load().moe_align_capacity(T, top_k, E, block_m))


def pack_scales_blocked_bytes(E: int, MN: int, KS: int) -> int:
    return int(load().pack_scales_blocked_bytes(E, MN, KS))


def moe_workspace_bytes(dtype: int, T: int, K: int, N: int, E: int, top_k: int, block_m: int) -> int:
    n = int(load().moe_workspace_bytes(dtype, T, K, N, E, top_k, block_m))
    if n < 0:
        raise MoeError(-1, "moe_workspace_bytes: invalid arguments")
    return n


# ---------------------------------------------------------------- calls
def moe_align(topk_ids, E: int, block_m: int, sorted_token_ids=None, expert_ids=None,
              num_tokens_post_padded=None, stream=None):
    """Routing planner.  Returns (sorted_token_ids, expert_ids, num_tokens_post_padded)."""
    import torch

    _need(topk_ids, "topk_ids", (torch.int32,))
    T, top_k = topk_ids.shape
    cap = moe_align_capacity(T, top_k, E, block_m)
    if cap < 0:
        raise MoeError(-1, "moe_align: invalid sizes")
    dev = topk_ids.device
    if sorted_token_ids is None:
        sorted_token_ids = torch.empty(cap, dtype=torch.int32, device=dev)
    if expert_ids is None:
        expert_ids = torch.empty((sorted_token_ids.numel() + block_m - 1) // block_m, dtype=torch.int32,
                                 device=dev)
    if num_tokens_post_padded is None:
        num_tokens_post_padded = torch.empty(1, dtype=torch.int32, device=dev)
    for t, n in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                 (num_tokens_post_padded, "num_tokens_post_padded")):
        _need(t, n, (torch.int32,))
    if expert_ids.numel() < (sorted_token_ids.numel() + block_m - 1) // block_m:
        raise ValueError("expert_ids must hold ceil(capacity / block_m) entries")
    _same_device(topk_ids, sorted_token_ids, expert_ids, num_tokens_post_padded)
    with _on_device(topk_ids.device, stream) as s:
        _check(load().moe_align(_ptr(topk_ids), T, top_k, E, block_m, _ptr(sorted_token_ids), _ptr(expert_ids),
                                _ptr(num_tokens_post_padded), sorted_token_ids.numel(), s))
    return sorted_token_ids, expert_ids, num_tokens_post_padded


def moe_route_align(logits, top_k: int, block_m: int, bias=None, topk_ids=None, topk_weights=None,
                    sorted_token_ids=None, expert_ids=None, num_tokens_post_padded=None, stream=None,
                    n_shared: int = 0):
    """Router + planner.  logits (T, E) fp32, bias (E,) fp32 or None; n_shared shared experts
    (indices E.., weight 1) follow the routed ones.  Returns (topk_ids, topk_weights,
    sorted_token_ids, expert_ids, num_tokens_post_padded), the first two (T, top_k + n_shared)."""
    import torch

    _need(logits, "logits", (torch.float32,))
    T, E = logits.shape
    if bias is not None:
        _need(bias, "bias", (torch.float32,))
        if bias.numel() != E:
            raise ValueError("bias must hold E values")
    kk = top_k + n_shared
    cap = moe_align_capacity(T, kk, E + n_shared, block_m)
    if cap < 0:
        raise MoeError(-1, "moe_route_align: invalid sizes")
    dev = logits.device
    if topk_ids is None:
        topk_ids = torch.empty((T, kk), dtype=torch.int32, device=dev)
    if topk_weights is None:
        topk_weights = torch.empty((T, kk), dtype=torch.float32, device=dev)
    if sorted_token_ids is None:
        sorted_token_ids = torch.empty(cap, dtype=torch.int32, device=dev)
    if expert_ids is None:
        expert_ids = torch.empty((sorted_token_ids.numel() + block_m - 1) // block_m, dtype=torch.int32,
                                 device=dev)
    if num_tokens_post_padded is None:
        num_tokens_post_padded = torch.empty(1, dtype=torch.int32, device=dev)
    _need(topk_ids, "topk_ids", (torch.int32,))
    _need(topk_weights, "topk_weights", (torch.float32,))
    if topk_ids.numel() < T * kk or topk_weights.numel() < T * kk:
        raise ValueError("topk_ids / topk_weights must hold T * (top_k + n_shared) entries")
    for t, n in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                 (num_tokens_post_padded, "num_tokens_post_padded")):
        _need(t, n, (torch.int32,))
    if expert_ids.numel() < (sorted_token_ids.numel() + block_m - 1) // block_m:
        raise ValueError("expert_ids must hold ceil(capacity / block_m) entries")
    _same_device(logits, *([] if bias is None else [bias]), topk_ids, topk_weights, sorted_token_ids, expert_ids,
                 num_tokens_post_padded)
    with _on_device(logits.device, stream) as s:
        _check(load().moe_route_align(_ptr(logits), _ptr(bias), T, E, top_k, n_shared, block_m, _ptr(topk_ids),
                                      _ptr(topk_weights), _ptr(sorted_token_ids), _ptr(expert_ids),
                                      _ptr(num_tokens_post_padded), sorted_token_ids.numel(), s))
    return topk_ids, topk_weights, sorted_token_ids, expert_ids, num_tokens_post_padded


def pack_scales_blocked(scales, out=None, stream=None):
    """(E, MN, KS) uint8 e8m0 scales, row major -> blocked 512-byte tiles (uint8, flat)."""
    import torch

    _need(scales, "scales", (torch.uint8,))
    E, MN, KS = scales.shape
    n = pack_scales_blocked_bytes(E, MN, KS)
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=scales.device)
    _need(out, "out", (torch.uint8,))
    if out.numel() < n:
        raise ValueError(f"out must hold {n} bytes")
    _same_device(scales, out)
    with _on_device(scales.device, stream) as s:
        _check(load().pack_scales_blocked(_ptr(scales), _ptr(out), E, MN, KS, s))
    return out


def _workspace(dtype, T, K, N, E, top_k, block_m, workspace, device):
    import torch

    need = moe_workspace_bytes(dtype, T, K, N, E, top_k, block_m)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    _need(workspace, "workspace", (torch.uint8,))
    return workspace


def fused_moe_bf16(x, w1, w2, sorted_token_ids, expert_ids, num_tokens_post_padded, topk_weights, out,
                   block_m: int, workspace=None, tune: Tuning | None = None, stream=None):
    """bf16 path.  x (T,K), w1 (E,N,K), w2 (E,K,N/2) bf16; topk_weights (T,top_k) fp32; out (T,K) bf16."""
    import torch

    for t, n in ((x, "x"), (w1, "w1"), (w2, "w2"), (out, "out")):
        _need(t, n, (torch.bfloat16,))
    _need(topk_weights, "topk_weights", (torch.float32,))
    for t, n in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                 (num_tokens_post_padded, "num_tokens_post_padded")):
        _need(t, n, (torch.int32,))
    _ffn_shapes("bf16", x, w1, w2, topk_weights, out, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m)
    T, K = x.shape
    E, N, _ = w1.shape
    top_k = topk_weights.shape[1]
    ws = _workspace(DTYPE_BF16, T, K, N, E, top_k, block_m, workspace, x.device)
    _same_device(x, ws)
    with _on_device(x.device, stream) as s:
        _check(load().fused_moe_bf16(
            _ptr(x), _ptr(w1), _ptr(w2), _ptr(sorted_token_ids), _ptr(expert_ids), _ptr(num_tokens_post_padded),
            _ptr(topk_weights), _ptr(out), T, K, N, E, top_k, block_m, sorted_token_ids.numel(), _ptr(ws),
            ws.numel(), None if tune is None else ctypes.byref(tune), s))
    return out


def fused_moe_mxfp8(x, x_scales, w1, w1_scales_blocked, w2, w2_scales_blocked, sorted_token_ids, expert_ids,
                    num_tokens_post_padded, topk_weights, out, block_m: int, workspace=None,
                    tune: Tuning | None = None, stream=None):
    """mxfp8 path.  e4m3 codes as uint8 (or float8_e4m3fn), e8m0 scales as uint8; out (T,K) bf16."""
    import torch

    u8 = (torch.uint8, torch.float8_e4m3fn)
    for t, n in ((x, "x"), (w1, "w1"), (w2, "w2")):
        _need(t, n, u8)
    for t, n in ((x_scales, "x_scales"), (w1_scales_blocked, "w1_scales_blocked"),
                 (w2_scales_blocked, "w2_scales_blocked")):
        _need(t, n, (torch.uint8,))
    _need(out, "out", (torch.bfloat16,))
    _need(topk_weights, "topk_weights", (torch.float32,))
    for t, n in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                 (num_tokens_post_padded, "num_tokens_post_padded")):
        _need(t, n, (torch.int32,))
    _ffn_shapes("mxfp8", x, w1, w2, topk_weights, out, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m,
                x_scales, w1_scales_blocked, w2_scales_blocked)
    T, K = x.shape
    E, N, _ = w1.shape
    top_k = topk_weights.shape[1]
    ws = _workspace(DTYPE_MXFP8, T, K, N, E, top_k, block_m, workspace, x.device)
    _same_device(x, ws)
    with _on_device(x.device, stream) as s:
        _check(load().fused_moe_mxfp8(
            _ptr(x), _ptr(x_scales), _ptr(w1), _ptr(w1_scales_blocked), _ptr(w2), _ptr(w2_scales_blocked),
            _ptr(sorted_token_ids), _ptr(expert_ids), _ptr(num_tokens_post_padded), _ptr(topk_weights), _ptr(out),
            T, K, N, E, top_k, block_m, sorted_token_ids.numel(), _ptr(ws), ws.numel(),
            None if tune is None else ctypes.byref(tune), s))
    return out


def fused_moe_mxfp4(x, x_scales, w1, w1_scales_blocked, w2, w2_scales_blocked, sorted_token_ids, expert_ids,
                    num_tokens_post_padded, topk_weights, out, block_m: int, workspace=None,
                    tune: Tuning | None = None, stream=None):
    """mxfp8 activations, MXFP4 weights: w1 (E, N, K/2) and w2 (E, K, N/4) uint8 of packed e2m1 codes
    (even index in the low nibble); scales and the rest as fused_moe_mxfp8."""
    import torch

    _need(x, "x", (torch.uint8, torch.float8_e4m3fn))
    for t, n in ((w1, "w1"), (w2, "w2"), (x_scales, "x_scales"), (w1_scales_blocked, "w1_scales_blocked"),
                 (w2_scales_blocked, "w2_scales_blocked")):
        _need(t, n, (torch.uint8,))
    _need(out, "out", (torch.bfloat16,))
    _need(topk_weights, "topk_weights", (torch.float32,))
    for t, n in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                 (num_tokens_post_padded, "num_tokens_post_padded")):
        _need(t, n, (torch.int32,))
    _ffn_shapes("mxfp4", x, w1, w2, topk_weights, out, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m,
                x_scales, w1_scales_blocked, w2_scales_blocked)
    T, K = x.shape
    E, N, _ = w1.shape
    top_k = topk_weights.shape[1]
    ws = _workspace(DTYPE_MXFP4, T, K, N, E, top_k, block_m, workspace, x.device)
    _same_device(x, ws)
    with _on_device(x.device, stream) as s:
        _check(load().fused_moe_mxfp4(
            _ptr(x), _ptr(x_scales), _ptr(w1), _ptr(w1_scales_blocked), _ptr(w2), _ptr(w2_scales_blocked),
            _ptr(sorted_token_ids), _ptr(expert_ids), _ptr(num_tokens_post_padded), _ptr(topk_weights), _ptr(out),
            T, K, N, E, top_k, block_m, sorted_token_ids.numel(), _ptr(ws), ws.numel(),
            None if tune is None else ctypes.byref(tune), s))
    return out


def fused_moe_bf16_noalloc_max_workspace() -> int:
    """Size of the library-owned workspace used by fused_moe_bf16_noalloc."""
    return int(load().fused_moe_bf16_noalloc_max_workspace())


def fused_moe_bf16_noalloc(x, w1, w2, sorted_token_ids, expert_ids, num_tokens_post_padded, topk_weights, out,
                           block_m: int, tune: Tuning | None = None, stream=None):
    """fused_moe_bf16 without a caller workspace: uses the library's fixed-size
    device scratch, so nothing is allocated.  For callers that cannot allocate
    device memory; problems needing more than
    fused_moe_bf16_noalloc_max_workspace() bytes are rejected."""
    import torch

    for t, n in ((x, "x"), (w1, "w1"), (w2, "w2"), (out, "out")):
        _need(t, n, (torch.bfloat16,))
    _need(topk_weights, "topk_weights", (torch.float32,))
    for t, n in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                 (num_tokens_post_padded, "num_tokens_post_padded")):
        _need(t, n, (torch.int32,))
    _ffn_shapes("bf16", x, w1, w2, topk_weights, out, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m)
    T, K = x.shape
    E, N, _ = w1.shape
    top_k = topk_weights.shape[1]
    with _on_device(x.device, stream) as s:
        _check(load().fused_moe_bf16_noalloc(
            _ptr(x), _ptr(w1), _ptr(w2), _ptr(sorted_token_ids), _ptr(expert_ids), _ptr(num_tokens_post_padded),
            _ptr(topk_weights), _ptr(out), T, K, N, E, top_k, block_m, sorted_token_ids.numel(),
            None if tune is None else ctypes.byref(tune), s))
    return out


def moe_ep_dispatch_plan(topk_ids, E: int, world: int, order=None, send_counts=None, stream=None):
    """Routes grouped by owner rank (experts split into `world` equal ranges).  Returns (order
    (T*top_k,) int32: route ids t*top_k+j reaching an expert, grouped by rank, then -1;
    send_counts (world,) int32)."""
    import torch

    _need(topk_ids, "topk_ids", (torch.int32,))
    T, top_k = topk_ids.shape
    dev = topk_ids.device
    order = torch.empty(T * top_k, dtype=torch.int32, device=dev) if order is None else order
    send_counts = torch.empty(world, dtype=torch.int32, device=dev) if send_counts is None else send_counts
    _need(order, "order", (torch.int32,))
    _need(send_counts, "send_counts", (torch.int32,))
    if order.numel() < T * top_k or send_counts.numel() < world:
        raise ValueError("order must hold T*top_k entries and send_counts world entries")
    _same_device(topk_ids, order, send_counts)
    with _on_device(dev, stream) as s:
        _check(load().moe_ep_dispatch_plan(_ptr(topk_ids), T, top_k, E, world, _ptr(order), _ptr(send_counts), s))
    return order, send_counts


def moe_ep_dispatch_pack(x, topk_ids, topk_weights, order, n: int, E: int, world: int, x_scales=None, stream=None):
    """The send buffers of the first n entries of `order`: (rows (n, K) in x's dtype, scales (n, K/32) uint8 or
    None, owner-local expert ids (n,) int32, routing weights (n,) fp32)."""
    import torch

    _need(topk_ids, "topk_ids", (torch.int32,))
    _need(topk_weights, "topk_weights", (torch.float32,))
    _need(order, "order", (torch.int32,))
    if not x.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be a contiguous (T, K) tensor")
    T, top_k = topk_ids.shape
    if x.shape[0] != T or tuple(topk_weights.shape) != (T, top_k) or order.numel() < n:
        raise ValueError("x, topk_ids, topk_weights and order disagree in shape")
    dev = x.device
    rows = torch.empty((n, x.shape[1]), dtype=x.dtype, device=dev)
    scales = None
    if x_scales is not None:
        _need(x_scales, "x_scales", (torch.uint8,))
        if x_scales.shape[0] != T:
            raise ValueError("x_scales must have one row per token")
        scales = torch.empty((n, x_scales.shape[1]), dtype=torch.uint8, device=dev)
    local_e = torch.empty(n, dtype=torch.int32, device=dev)
    w = torch.empty(n, dtype=torch.float32, device=dev)
    _same_device(x, topk_ids, topk_weights, order, *([] if x_scales is None else [x_scales]))
    with _on_device(dev, stream) as s:
        _check(load().moe_ep_dispatch_pack(
            _ptr(x), x.shape[1] * x.element_size(), _ptr(x_scales), 0 if x_scales is None else x_scales.shape[1],
            _ptr(topk_ids), _ptr(topk_weights), _ptr(order), n, T, top_k, E, world, _ptr(rows), _ptr(scales),
            _ptr(local_e), _ptr(w), s))
    return rows, scales, local_e, w


def moe_ep_combine(y, order, n: int, T: int, top_k: int, out=None, slot=None, stream=None):
    """out (T, K) bf16: per token, the sum in route order (fp32) of its routes' rows of y (n, K) bf16, row i
    belonging to route order[i]."""
    import torch

    _need(y, "y", (torch.bfloat16,))
    _need(order, "order", (torch.int32,))
    K = y.shape[1]
    dev = y.device
    out = torch.empty((T, K), dtype=torch.bfloat16, device=dev) if out is None else out
    slot = torch.empty(max(T * top_k, 1), dtype=torch.int32, device=dev) if slot is None else slot
    _need(out, "out", (torch.bfloat16,))
    _need(slot, "slot", (torch.int32,))
    if tuple(out.shape) != (T, K) or slot.numel() < T * top_k or y.shape[0] < n or order.numel() < n:
        raise ValueError("out must be (T, K), slot hold T*top_k entries, y and order n rows")
    _same_device(y, order, out, slot)
    with _on_device(dev, stream) as s:
        _check(load().moe_ep_combine(_ptr(y), _ptr(order), n, T, top_k, K, _ptr(slot), _ptr(out), s))
    return out


# ---------------------------------------------------------------- training
def _call(fn, dev, stream, *args):
    """fn(*args, stream handle) with ``dev`` current.  A small call is bound by what happens here, so where no
    device has to be switched the stream's handle is taken as it is, without a Stream object (12.5 us a permute
    of 8 tokens with one, and with every check of _tensor made on its own)."""
    import torch

    if stream is None and dev.index == torch._C._cuda_getDevice() and dev.type == "cuda":
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with _on_device(dev, stream) as s:
            rc = fn(*args, s)
    if rc != 0:
        _check(rc)


def _new(shape, dtype, dev, stream):
    """A tensor the call is about to write, allocated on the stream that will write it: memory freed by work
    still pending on the current stream is then not handed to another one."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    elif torch.device(getattr(stream, "device", dev)) != torch.device(dev):
        raise ValueError(f"stream belongs to {stream.device} but the tensors are on {dev}")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _tensor(t, name, dtype, dev, shape):
    """One argument of a training call: type, layout, device and shape (the kernels trust all four)."""
    if t is not None and t.dtype is dtype and t.get_device() == dev.index and t.shape == shape and t.is_contiguous():
        return  # (the index of a CPU tensor is -1, that of its device None)
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != dev:
        raise ValueError(f"all tensors must be on {dev}, got {name} on {t.device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows_dtype(t, name):
    """MOE_ROWS_* of a (rows, K) tensor."""
    import torch

    if t is None:
        raise ValueError(f"{name} is required")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float32:
        return 1
    raise TypeError(f"{name}: dtype {t.dtype} not in (torch.bfloat16, torch.float32)")


def _rows_code(t):
    return 1 if t.dtype is _dtypes["f32"] else 0


def _slots_shape(slots):
    import torch

    if slots is None:
        raise ValueError("slots is required")
    if slots.dim() != 2:
        raise ValueError("slots must be (T, top_k)")
    T, top_k = slots.shape
    _tensor(slots, "slots", torch.int32, slots.device, (T, top_k))
    return T, top_k, slots.device


def _order(sorted_token_ids, num_tokens_post_padded, dev):
    """Capacity of the planner's order."""
    import torch

    if sorted_token_ids is None:
        raise ValueError("sorted_token_ids is required")
    capacity = sorted_token_ids.numel()
    _tensor(sorted_token_ids, "sorted_token_ids", torch.int32, dev, (capacity,))
    _tensor(num_tokens_post_padded, "num_tokens_post_padded", torch.int32, dev, (1,))
    return capacity


def moe_route_slots(sorted_token_ids, num_tokens_post_padded, T: int, top_k: int, slots=None, stream=None):
    """Inverse of the planner's order: slots (T, top_k) int32, the place of every route in sorted_token_ids
    or -1.  What moe_permute, moe_unpermute and their gradients address rows with."""
    import torch

    dev = getattr(sorted_token_ids, "device", None)
    capacity = _order(sorted_token_ids, num_tokens_post_padded, dev)
    if slots is None:
        slots = _new((T, top_k), torch.int32, dev, stream)
    _tensor(slots, "slots", torch.int32, dev, (T, top_k))
    _call(load().moe_route_slots, dev, stream, _ptr(sorted_token_ids), _ptr(num_tokens_post_padded), capacity, T, top_k,
          _ptr(slots))
    return slots


def _rows_quick(slots, token, rows, order, weights):
    """Whether the tensors of a call on rows fit one another, as far as one look tells: True, or False where
    the checks one by one have to say what is missing or wrong.  token (T, K) and rows (capacity, K) of one
    type, order None or (sorted_token_ids, num_tokens_post_padded), weights None or (T, top_k).  A call of few
    tokens is bound by the host, and the checks one by one are a third of it."""
    try:
        T, K = token.shape
        i, capacity, dtype, i32 = slots.get_device(), rows.shape[0], token.dtype, _dtypes["i32"]
        return (i >= 0 and slots.dtype is i32 and slots.shape[0] == T and slots.dim() == 2 and slots.is_contiguous()
                and (dtype is _dtypes["bf16"] or dtype is _dtypes["f32"]) and token.get_device() == i
                and token.is_contiguous() and rows.dtype is dtype and rows.shape == (capacity, K)
                and rows.get_device() == i and rows.is_contiguous()
                and (weights is None or (weights.dtype is _dtypes["f32"] and weights.shape == slots.shape
                                         and weights.get_device() == i and weights.is_contiguous()))
                and (order is None or (order[0].dtype is i32 and order[0].shape == (capacity,)
                                       and order[0].get_device() == i and order[0].is_contiguous()
                                       and order[1].dtype is i32 and order[1].shape == (1,)
                                       and order[1].get_device() == i)))
    except (AttributeError, KeyError, IndexError, ValueError):  # None, before the library is loaded, other dimensions
        return False


def moe_permute(x, sorted_token_ids, num_tokens_post_padded, slots, out=None, stream=None):
    """Token rows x (T, K), bf16 or fp32, in the planner's order: returns rows (capacity, K) with
    rows[slots[t, j]] = x[t], zeros in padding rows; rows at or past num_tokens_post_padded are not written."""
    if out is None or not _rows_quick(slots, x, out, (sorted_token_ids, num_tokens_post_padded), None):
        _rows_dtype(x, "x")
        T, _, dev = _slots_shape(slots)
        K = x.shape[1]
        _tensor(x, "x", x.dtype, dev, (T, K))
        capacity = _order(sorted_token_ids, num_tokens_post_padded, dev)
        if out is None:
            out = _new((capacity, K), x.dtype, dev, stream)
        _tensor(out, "out", x.dtype, dev, (capacity, K))
    T, top_k = slots.shape
    capacity, K = out.shape
    _call(load().moe_permute, slots.device, stream, x.data_ptr(), _rows_code(x), sorted_token_ids.data_ptr(),
          num_tokens_post_padded.data_ptr(), slots.data_ptr(), capacity, T, top_k, K, out.data_ptr())
    return out


def moe_permute_backward(grad_rows, slots, out=None, stream=None):
    """Gradient of moe_permute by x: (T, K), the sum in route order of the rows grad_rows (capacity, K) of a
    token's routes."""
    if out is None or not _rows_quick(slots, out, grad_rows, None, None):
        _rows_dtype(grad_rows, "grad_rows")
        T, _, dev = _slots_shape(slots)
        capacity, K = grad_rows.shape
        _tensor(grad_rows, "grad_rows", grad_rows.dtype, dev, (capacity, K))
        if out is None:
            out = _new((T, K), grad_rows.dtype, dev, stream)
        _tensor(out, "out", grad_rows.dtype, dev, (T, K))
    T, top_k = slots.shape
    capacity, K = grad_rows.shape
    _call(load().moe_permute_backward, slots.device, stream, grad_rows.data_ptr(), _rows_code(grad_rows),
          slots.data_ptr(), capacity, T, top_k, K, out.data_ptr())
    return out


def moe_unpermute(y, slots, topk_weights, out=None, stream=None):
    """out (T, K): per token the sum in route order of topk_weights[t, j] * y[slots[t, j]], y (capacity, K) bf16
    or fp32; fp32 sums, one rounding."""
    if out is None or topk_weights is None or not _rows_quick(slots, out, y, None, topk_weights):
        import torch

        _rows_dtype(y, "y")
        T, top_k, dev = _slots_shape(slots)
        capacity, K = y.shape
        _tensor(y, "y", y.dtype, dev, (capacity, K))
        _tensor(topk_weights, "topk_weights", torch.float32, dev, (T, top_k))
        if out is None:
            out = _new((T, K), y.dtype, dev, stream)
        _tensor(out, "out", y.dtype, dev, (T, K))
    T, top_k = slots.shape
    capacity, K = y.shape
    _call(load().moe_unpermute, slots.device, stream, y.data_ptr(), _rows_code(y), slots.data_ptr(),
          topk_weights.data_ptr(), capacity, T, top_k, K, out.data_ptr())
    return out


def moe_unpermute_backward(grad_out, y, sorted_token_ids, num_tokens_post_padded, slots, topk_weights, grad_y=None,
                           grad_weights=None, stream=None):
    """Gradients of moe_unpermute: (grad_y (capacity, K) with grad_y[slots[t, j]] = topk_weights[t, j] *
    grad_out[t] and zeros in padding rows, grad_weights (T, top_k) fp32 = <grad_out[t], y[slots[t, j]]>)."""
    import torch

    _rows_dtype(grad_out, "grad_out")
    T, top_k, dev = _slots_shape(slots)
    K = grad_out.shape[1]
    _tensor(grad_out, "grad_out", grad_out.dtype, dev, (T, K))
    capacity = _order(sorted_token_ids, num_tokens_post_padded, dev)
    _tensor(y, "y", grad_out.dtype, dev, (capacity, K))
    _tensor(topk_weights, "topk_weights", torch.float32, dev, (T, top_k))
    if grad_y is None:
        grad_y = _new((capacity, K), grad_out.dtype, dev, stream)
    if grad_weights is None:
        grad_weights = _new((T, top_k), torch.float32, dev, stream)
    _tensor(grad_y, "grad_y", grad_out.dtype, dev, (capacity, K))
    _tensor(grad_weights, "grad_weights", torch.float32, dev, (T, top_k))
    _call(load().moe_unpermute_backward, dev, stream, _ptr(grad_out), _ptr(y), _rows_code(grad_out),
          _ptr(sorted_token_ids), _ptr(num_tokens_post_padded), _ptr(slots), _ptr(topk_weights), capacity, T, top_k, K,
          _ptr(grad_y), _ptr(grad_weights))
    return grad_y, grad_weights


def _expert_plan(w, name, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m):
    """Device and capacity of an expert product, w (E, rows, cols) its weights."""
    import torch

    if w is None:
        raise ValueError(f"{name} is required")
    if w.dim() != 3:
        raise ValueError(f"{name} must have three dimensions, got {w.dim()}")
    dev = w.device
    _tensor(w, name, torch.bfloat16, dev, tuple(w.shape))
    capacity = _order(sorted_token_ids, num_tokens_post_padded, dev)
    if block_m < 1:
        raise ValueError("block_m must be positive")
    if expert_ids is None:
        raise ValueError("expert_ids is required")
    blocks = (capacity + block_m - 1) // block_m
    if expert_ids.numel() < blocks:
        raise ValueError(f"expert_ids must hold ceil(capacity / block_m) = {blocks} entries")
    _tensor(expert_ids, "expert_ids", torch.int32, dev, (expert_ids.numel(),))
    return dev, capacity


def _expert_quick(w, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m, *rows):
    """The same as _rows_quick for an expert product: w (E, rows, cols) and every (tensor, width) of `rows` bf16."""
    try:
        i, bf16, i32, capacity = w.get_device(), _dtypes["bf16"], _dtypes["i32"], sorted_token_ids.shape[0]
        if not (i >= 0 and w.dtype is bf16 and w.dim() == 3 and w.is_contiguous()
                and sorted_token_ids.dtype is i32 and sorted_token_ids.dim() == 1
                and sorted_token_ids.get_device() == i and sorted_token_ids.is_contiguous()
                and block_m > 0 and expert_ids.dtype is i32 and expert_ids.dim() == 1
                and expert_ids.shape[0] * block_m >= capacity and expert_ids.get_device() == i
                and expert_ids.is_contiguous()
                and num_tokens_post_padded.dtype is i32 and num_tokens_post_padded.shape == (1,)
                and num_tokens_post_padded.get_device() == i):
            return False
        for t, width in rows:
            if not (t.dtype is bf16 and t.shape == (capacity, width) and t.get_device() == i and t.is_contiguous()):
                return False
        return True
    except (AttributeError, KeyError, IndexError):
        return False


def _weight_grad(grad, name, w, accumulate, dev, stream):
    """(gradient buffer, MOE_ROWS_* of it); a new one is bf16."""
    import torch

    if grad is None:
        if accumulate:
            raise ValueError(f"accumulate needs {name}")
        return _new(tuple(w.shape), torch.bfloat16, dev, stream), 0
    if grad.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"{name}: dtype {grad.dtype} not in (torch.bfloat16, torch.float32)")
    if accumulate and grad.dtype != torch.float32:
        raise TypeError(f"{name}: accumulating needs an fp32 buffer, got {grad.dtype}")
    _tensor(grad, name, grad.dtype, dev, tuple(w.shape))
    return grad, int(grad.dtype == torch.float32)


def moe_expert_up(rows, w1, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m: int, h=None, act=None,
                  stream=None):
    """Gate/up product with SwiGLU on rows (capacity, K) in the planner's order, w1 (E, N, K), all bf16: returns
    (h (capacity, N), act (capacity, N/2)) with h = rows . w1[e]^T and act = silu(gate) * up from the unrounded h."""
    plan = (sorted_token_ids, expert_ids, num_tokens_post_padded)
    E, N, K = getattr(w1, "shape", ()) if getattr(w1, "ndim", 0) == 3 else (0, 1, 0)
    if N % 2 or not _expert_quick(w1, *plan, block_m, (rows, K), (h, N), (act, N // 2)):
        import torch

        bf16 = torch.bfloat16
        dev, capacity = _expert_plan(w1, "w1", *plan, block_m)
        E, N, K = w1.shape
        if N % 2:
            raise ValueError(f"N = {N} must be even (gate and up halves)")
        _tensor(rows, "rows", bf16, dev, (capacity, K))
        if h is None:
            h = _new((capacity, N), bf16, dev, stream)
        if act is None:
            act = _new((capacity, N // 2), bf16, dev, stream)
        _tensor(h, "h", bf16, dev, (capacity, N))
        _tensor(act, "act", bf16, dev, (capacity, N // 2))
    _call(load().moe_expert_up, w1.device, stream, rows.data_ptr(), w1.data_ptr(), *map(_ptr, plan), rows.shape[0], K, N,
          E, block_m, h.data_ptr(), act.data_ptr())
    return h, act


def moe_expert_down(act, w2, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m: int, out=None, stream=None):
    """Down product on act (capacity, N/2), w2 (E, K, N/2), bf16: returns y (capacity, K) = act . w2[e]^T."""
    plan = (sorted_token_ids, expert_ids, num_tokens_post_padded)
    E, K, half = getattr(w2, "shape", ()) if getattr(w2, "ndim", 0) == 3 else (0, 0, 0)
    if not _expert_quick(w2, *plan, block_m, (act, half), (out, K)):
        import torch

        bf16 = torch.bfloat16
        dev, capacity = _expert_plan(w2, "w2", *plan, block_m)
        E, K, half = w2.shape
        _tensor(act, "act", bf16, dev, (capacity, half))
        if out is None:
            out = _new((capacity, K), bf16, dev, stream)
        _tensor(out, "out", bf16, dev, (capacity, K))
    _call(load().moe_expert_down, w2.device, stream, act.data_ptr(), w2.data_ptr(), *map(_ptr, plan), act.shape[0], K,
          2 * half, E, block_m, out.data_ptr())
    return out


def moe_expert_down_backward(grad_y, h, act, w2, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m: int,
                             grad_h=None, grad_w2=None, accumulate: bool = False, stream=None):
    """Gradients of moe_expert_down and of the SwiGLU before it: grad_y (capacity, K), h (capacity, N), act
    (capacity, N/2), w2 (E, K, N/2), bf16.  Returns (grad_h (capacity, N) bf16, grad_w2 (E, K, N/2) bf16, or fp32
    when such a buffer is given, which accumulate=True adds to)."""
    plan = (sorted_token_ids, expert_ids, num_tokens_post_padded)
    E, K, half = getattr(w2, "shape", ()) if getattr(w2, "ndim", 0) == 3 else (0, 0, 0)
    quick = _expert_quick(w2, *plan, block_m, (grad_y, K), (h, 2 * half), (act, half), (grad_h, 2 * half))
    if not quick:
        import torch

        bf16 = torch.bfloat16
        dev, capacity = _expert_plan(w2, "w2", *plan, block_m)
        E, K, half = w2.shape
        _tensor(grad_y, "grad_y", bf16, dev, (capacity, K))
        _tensor(h, "h", bf16, dev, (capacity, 2 * half))
        _tensor(act, "act", bf16, dev, (capacity, half))
    grad_w2, gdt = _weight_grad(grad_w2, "grad_w2", w2, accumulate, w2.device, stream)
    if not quick:
        if grad_h is None:
            grad_h = _new((capacity, 2 * half), bf16, dev, stream)
        _tensor(grad_h, "grad_h", bf16, dev, (capacity, 2 * half))
    _call(load().moe_expert_down_backward, w2.device, stream, grad_y.data_ptr(), h.data_ptr(), act.data_ptr(),
          w2.data_ptr(), *map(_ptr, plan), act.shape[0], K, 2 * half, E, block_m, grad_h.data_ptr(), grad_w2.data_ptr(),
          gdt, int(accumulate))
    return grad_h, grad_w2


def moe_expert_up_backward(grad_h, rows, w1, sorted_token_ids, expert_ids, num_tokens_post_padded, block_m: int,
                           grad_rows=None, grad_w1=None, accumulate: bool = False, stream=None):
    """Gradients of the gate/up product: grad_h (capacity, N), rows (capacity, K), w1 (E, N, K), bf16.  Returns
    (grad_rows (capacity, K) bf16, grad_w1 (E, N, K) bf16, or fp32 when such a buffer is given, which
    accumulate=True adds to)."""
    plan = (sorted_token_ids, expert_ids, num_tokens_post_padded)
    E, N, K = getattr(w1, "shape", ()) if getattr(w1, "ndim", 0) == 3 else (0, 0, 0)
    quick = _expert_quick(w1, *plan, block_m, (grad_h, N), (rows, K), (grad_rows, K))
    if not quick:
        import torch

        bf16 = torch.bfloat16
        dev, capacity = _expert_plan(w1, "w1", *plan, block_m)
        E, N, K = w1.shape
        _tensor(grad_h, "grad_h", bf16, dev, (capacity, N))
        _tensor(rows, "rows", bf16, dev, (capacity, K))
    grad_w1, gdt = _weight_grad(grad_w1, "grad_w1", w1, accumulate, w1.device, stream)
    if not quick:
        if grad_rows is None:
            grad_rows = _new((capacity, K), bf16, dev, stream)
        _tensor(grad_rows, "grad_rows", bf16, dev, (capacity, K))
    _call(load().moe_expert_up_backward, w1.device, stream, grad_h.data_ptr(), rows.data_ptr(), w1.data_ptr(),
          *map(_ptr, plan), rows.shape[0], K, N, E, block_m, grad_rows.data_ptr(), grad_w1.data_ptr(), gdt,
          int(accumulate))
    return grad_rows, grad_w1


def moe_orthogonalize_workspace_bytes(E: int, M: int, N: int) -> int:
    n = int(load().moe_orthogonalize_workspace_bytes(E, M, N))
    if n < 0:
        raise MoeError(-1, "moe_orthogonalize_workspace_bytes: invalid arguments")
    return n


def moe_orthogonalize(g, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, out=None,
                      workspace=None, stream=None):
    """Every matrix of g (E, M, N), bf16 or fp32, made nearly orthogonal: X = g / (|g|_F + eps), then `steps` times
    X <- a X + (b A + c A A) X with A = X X^T and (a, b, c) the coefficients.  Returns out (E, M, N) bf16 (which may
    be a bf16 g itself)."""
    import torch

    if g is None:
        raise ValueError("g is required")
    if g.dim() != 3:
        raise ValueError(f"g must be (E, M, N), got {g.dim()} dimensions")
    if g.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"g: dtype {g.dtype} not in (torch.bfloat16, torch.float32)")
    dev, shape = g.device, tuple(g.shape)
    _tensor(g, "g", g.dtype, dev, shape)
    a, b, c = coefficients
    if out is None:
        out = _new(shape, torch.bfloat16, dev, stream)
    _tensor(out, "out", torch.bfloat16, dev, shape)
    if g.numel() == 0:
        return out
    if workspace is None:
        workspace = _new((moe_orthogonalize_workspace_bytes(*shape),), torch.uint8, dev, stream)
    _tensor(workspace, "workspace", torch.uint8, dev, (workspace.numel(),))
    _call(load().moe_orthogonalize, dev, stream, _ptr(g), int(g.dtype == torch.float32), *shape, steps, a, b, c, eps,
          _ptr(out), _ptr(workspace), workspace.numel())
    return out


def moe_device_status(stream=None, device=None):
    """Waits for the stream; raises MoeError(MOE_ERR_TIMEOUT) if a device-side wait of this library
    on that device gave up.  ``device``: default the stream's device, else the current one."""
    import torch

    if device is None:
        device = getattr(stream, "device", None) or torch.device("cuda", torch.cuda.current_device())
    with _on_device(torch.device(device), stream) as s:
        _check(load().moe_device_status(s))
