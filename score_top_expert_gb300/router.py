"""Python binding of the router's C ABI (include/moe_router.h).

Argument marshalling only: every function checks tensor devices, dtypes and
shapes, allocates missing outputs with torch, passes raw device pointers and
the current torch stream to the library, and raises on a nonzero status.
All router arithmetic runs in the library's CUDA kernels; there is no other
implementation behind these names.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

MR_SOFTMAX, MR_SIGMOID, MR_SOFTMAX_POST = 0, 1, 2
MR_F32, MR_BF16 = 0, 1
MR_PATH_AUTO, MR_PATH_SEGMENT, MR_PATH_STAGED, MR_PATH_REGISTER = 0, 1, 2, 3
STATUS = {0: "MR_OK", -1: "MR_ERR_INVALID", -2: "MR_ERR_UNSUPPORTED", -3: "MR_ERR_CUDA"}

_SCORE = {"softmax": MR_SOFTMAX, "sigmoid": MR_SIGMOID, "softmax_post": MR_SOFTMAX_POST}
_DTYPE = {torch.float32: MR_F32, torch.bfloat16: MR_BF16}

_lib = None
_fast = None  # the CPython call shim, when built (same C entry points as ctypes)


class RouterError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        msg = lib().moe_router_strerror(code).decode()
        super().__init__(f"{fn}: {STATUS.get(code, code)} ({msg})")


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded C library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(
                f"router CUDA library not built ({path} missing); run "
                "`python -m score_top_expert_gb300.build`")
        L = ctypes.CDLL(path)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.router_topk_fwd.argtypes = [vp, i, i, i, i, i, i, i, f, vp, vp, vp, vp, vp]
        L.router_topk_fwd_compact.argtypes = [vp, i, i, i, i, i, i, i, f, vp, vp, i, vp, i, vp,
                                              vp, vp, vp, vp]
        L.router_expert_maps_workspace_bytes.argtypes = [i, i]
        L.router_expert_maps_workspace_bytes.restype = ctypes.c_size_t
        L.router_expert_maps.argtypes = [vp, i, i, i, i, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                         vp]
        L.router_topk_fwd_maps.argtypes = [vp, i, i, i, i, i, i, i, f, vp, vp, i, vp, i, vp, vp,
                                           vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.router_topk_bwd.argtypes = [vp, vp, vp, i, i, i, i, i, f, vp, vp]
        L.router_aux_scores_fwd.argtypes = [vp, i, i, i, i, i, vp, vp, vp, vp]
        L.router_aux_scores_bwd.argtypes = [vp, vp, i, i, i, i, i, vp, vp]
        for fn in ("router_topk_fwd", "router_topk_fwd_compact", "router_topk_fwd_maps",
                   "router_expert_maps", "router_topk_bwd",
                   "router_aux_scores_fwd",
                   "router_aux_scores_bwd", "moe_router_force_path",
                   "moe_router_force_fwd_lanes", "moe_router_version",
                   "moe_router_device_status"):
            getattr(L, fn).restype = ctypes.c_int
        L.moe_router_force_path.argtypes = [i]
        L.moe_router_force_fwd_lanes.argtypes = [i]
        L.moe_router_version.argtypes = []
        L.moe_router_device_status.argtypes = [ctypes.POINTER(ctypes.c_int)]
        L.moe_router_selftest_bounded_wait.argtypes = [ctypes.c_uint, vp]
        L.router_aux_loss_workspace_bytes.argtypes = [i, i]
        L.router_aux_loss_workspace_bytes.restype = ctypes.c_size_t
        L.router_aux_loss_fwd.argtypes = [vp, vp, i, i, i, f, vp, vp, vp, ctypes.c_size_t, vp]
        L.router_aux_loss_fwd.restype = ctypes.c_int
        L.router_aux_loss_fwd_noalloc.argtypes = [vp, vp, i, i, i, f, vp, vp, vp]
        L.router_aux_loss_fwd_noalloc.restype = ctypes.c_int
        L.router_aux_loss_bwd.argtypes = [vp, vp, i, i, i, f, vp, vp]
        L.router_aux_loss_bwd.restype = ctypes.c_int
        L.router_expert_matmul.argtypes = [vp, i, vp, vp, vp, i, i, i, i, i, vp, i, vp]
        L.router_expert_matmul_bwd_input.argtypes = [vp, i, vp, vp, i, i, i, i, vp, i, vp]
        L.router_expert_matmul_bwd_weight.argtypes = [vp, i, vp, vp, vp, i, i, i, i, i, vp, i, vp]
        L.router_expert_matmul_w4.argtypes = [vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, vp, i, vp]
        L.router_combine_fwd.argtypes = [vp, i, vp, vp, i, i, i, i, vp, vp]
        L.router_combine_bwd.argtypes = [vp, i, vp, vp, vp, i, i, i, i, vp, vp, vp]
        sz = ctypes.c_size_t
        L.router_expert_matmul_w8.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp]
        L.router_quantize_rows.argtypes = [vp, i, i, i, vp, vp, vp]
        L.router_combine_norm_fwd.argtypes = [vp, i, vp, vp, i, vp, vp, vp, i, f, vp, f, i, i, i,
                                              vp, vp, vp, vp, vp]
        L.router_combine_norm_bwd_workspace_bytes.argtypes = [i, i]
        L.router_combine_norm_bwd_workspace_bytes.restype = sz
        L.router_combine_norm_bwd.argtypes = [vp, vp, i, vp, vp, vp, vp, vp, i, f, vp, i, i, vp,
                                              vp, vp, vp, vp, vp, sz, vp]
        L.router_balance_loss_workspace_bytes.argtypes = [i, i, i]
        L.router_balance_loss_workspace_bytes.restype = sz
        L.router_balance_loss_fwd.argtypes = [vp, i, vp, i, vp, i, i, i, i, i, f, f, vp, vp, vp,
                                              vp, sz, vp]
        L.router_balance_loss_bwd.argtypes = [vp, vp, i, vp, vp, vp, i, i, i, i, i, f, f, vp, vp]
        for fn in ("router_expert_matmul", "router_expert_matmul_bwd_input",
                   "router_expert_matmul_bwd_weight", "router_expert_matmul_w4",
                   "router_expert_matmul_w8", "router_quantize_rows",
                   "router_combine_fwd", "router_combine_bwd", "router_combine_norm_fwd",
                   "router_combine_norm_bwd", "router_balance_loss_fwd",
                   "router_balance_loss_bwd"):
            getattr(L, fn).restype = ctypes.c_int
        L.moe_router_selftest_bounded_wait.restype = ctypes.c_int
        L.moe_router_strerror.argtypes = [i]
        L.moe_router_strerror.restype = ctypes.c_char_p
        _lib = L
        _load_fast()
    return _lib


class _CtypesCalls:
    """The hot calls through ctypes (pointers as integers, 0 for NULL), for
    an interpreter without headers to build the CPython shim."""

    def __init__(self, L):
        self.router_topk_fwd = L.router_topk_fwd
        self.router_topk_bwd = L.router_topk_bwd
        self.router_aux_scores_fwd = L.router_aux_scores_fwd
        self.router_aux_scores_bwd = L.router_aux_scores_bwd
        self.router_expert_matmul = L.router_expert_matmul
        self.router_expert_matmul_w4 = L.router_expert_matmul_w4
        self.router_combine_fwd = L.router_combine_fwd
        self.router_combine_bwd = L.router_combine_bwd
        self.router_expert_matmul_bwd_input = L.router_expert_matmul_bwd_input
        self.router_expert_matmul_bwd_weight = L.router_expert_matmul_bwd_weight
        self.router_expert_matmul_w8 = L.router_expert_matmul_w8
        self.router_quantize_rows = L.router_quantize_rows
        self.router_combine_norm_fwd = L.router_combine_norm_fwd
        self.router_combine_norm_bwd = L.router_combine_norm_bwd
        self.router_balance_loss_fwd = L.router_balance_loss_fwd
        self.router_balance_loss_bwd = L.router_balance_loss_bwd
        self.router_balance_loss_workspace_bytes = L.router_balance_loss_workspace_bytes
        self.router_combine_norm_bwd_workspace_bytes = L.router_combine_norm_bwd_workspace_bytes


def _load_fast():
    """Bind the hot calls: the CPython shim built next to the library, else
    ctypes.  Both call the same exported C entry points."""
    global _fast
    path = _build.PYCALLS
    if os.path.exists(path):
        import importlib.util
        spec = importlib.util.spec_from_file_location("_pycalls", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        _fast = mod
    else:
        _fast = _CtypesCalls(_lib)


def _calls():
    if _fast is None:
        lib()
    return _fast


# The per-call path is kept lean for decode-sized calls, where the host cost
# of a call is most of its latency: pointers go to ctypes as plain integers
# (the argtypes convert them), the stream as the raw handle of torch's current
# stream, and devices as indices.
try:
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _cur_dev = torch._C._cuda_getDevice
except AttributeError:  # pragma: no cover - older torch
    def _raw_stream(i):
        return torch.cuda.current_stream(i).cuda_stream

    _cur_dev = torch.cuda.current_device


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _ptr0(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(device) -> int:
    """Raw handle of torch's current stream on ``device`` (a torch.device or
    an index)."""
    return _raw_stream(device if isinstance(device, int) else device.index)


class _NoSwitch:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NO_SWITCH = _NoSwitch()


def _on(device):
    """Make ``device`` (a torch.device or an index) current for the library
    call; no switch (and none of its cost) when it already is."""
    idx = device if isinstance(device, int) else device.index
    if idx is None or idx == _cur_dev():
        return _NO_SWITCH
    return torch.cuda.device(idx)


def _check(fn: str, code: int):
    if code != 0:
        raise RouterError(fn, code)


def _as_input(t: torch.Tensor, name: str, dtypes) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} dtype {t.dtype} not in {dtypes}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be [T, E]")
    return t if t.is_contiguous() else t.contiguous()


def _score(score_func: str) -> int:
    try:
        return _SCORE[score_func]
    except KeyError:
        raise ValueError(f"score_func must be one of {list(_SCORE)}") from None


def _out(t, shape, dtype, device, name):
    """A caller's output tensor, checked (shape, dtype, contiguity, device),
    or a new one.  ``device``: a torch.device with an index."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() \
            or t.get_device() != device.index:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on "
                         f"{device}")
    return t


def router_topk_fwd(logits: torch.Tensor, K: int, score_func: str = "softmax",
                    num_groups: int = 0, group_topk: int = 0, scaling_factor: float = 1.0,
                    expert_bias: torch.Tensor | None = None, *, probs=None,
                    routing_map=None, scores=None):
    """Top-K router forward.  Returns (probs [T,E] logits dtype,
    routing_map [T,E] bool, scores [T,E] float32)."""
    logits = _as_input(logits, "logits", _DTYPE)
    shape = logits.shape
    T, E = shape
    dev = logits.device
    dt = logits.dtype
    if expert_bias is not None:
        if expert_bias.dtype != torch.float32 or expert_bias.numel() != E \
                or expert_bias.get_device() != dev.index:
            raise ValueError("expert_bias must be a float32 [E] tensor on the logits' device")
        expert_bias = expert_bias.contiguous()
    probs = _out(probs, shape, dt, dev, "probs")
    routing_map = _out(routing_map, shape, torch.bool, dev, "routing_map")
    scores = _out(scores, shape, torch.float32, dev, "scores")
    with _on(dev):
        rc = _calls().router_topk_fwd(logits.data_ptr(), _DTYPE[dt], T, E, int(K),
                                      _score(score_func), int(num_groups), int(group_topk),
                                      float(scaling_factor), _ptr0(expert_bias),
                                      probs.data_ptr(), routing_map.data_ptr(),
                                      scores.data_ptr(), _stream(dev))
    _check("router_topk_fwd", rc)
    return probs, routing_map, scores


def _rows_out(t, T, K, dtype, device, name):
    """A [T, >= K] output addressed by row stride (unit column stride): a
    column view of a wider buffer is written in place."""
    if t is None:
        return torch.empty((T, K), dtype=dtype, device=device)
    if t.dim() != 2 or t.shape[0] != T or t.shape[1] < K or t.dtype != dtype \
            or t.get_device() != device.index or (T > 1 and t.stride(1) != 1) \
            or t.stride(0) < K:
        raise ValueError(f"{name} must be a {dtype} [T, >= K] tensor with unit column "
                         f"stride and row stride >= K")
    return t


def router_topk_fwd_compact(logits: torch.Tensor, K: int, score_func: str = "softmax",
                            num_groups: int = 0, group_topk: int = 0,
                            scaling_factor: float = 1.0,
                            expert_bias: torch.Tensor | None = None, *, topk_weights=None,
                            topk_indices=None, token_expert_indices=True, dense=False,
                            probs=None, routing_map=None, scores=None):
    """Top-K router forward with compact outputs.  Returns (topk_weights
    [T,K] float32, topk_indices [T,K] int32, token_expert_indices [T,K] int32
    or None, probs, routing_map, scores); row t, column k holds the expert of
    rank k (selection key descending, index ascending).  topk_weights and
    topk_indices may be column views of wider buffers (written in place).
    token_expert_indices: True to allocate, False/None to skip, or a
    contiguous [T,K] int32 tensor.  The dense outputs are None unless
    dense=True or given."""
    logits = _as_input(logits, "logits", _DTYPE)
    T, E = logits.shape
    dev = logits.device
    K = int(K)
    if expert_bias is not None:
        if expert_bias.dtype != torch.float32 or expert_bias.numel() != E \
                or expert_bias.get_device() != dev.index:
            raise ValueError("expert_bias must be a float32 [E] tensor on the logits' device")
        expert_bias = expert_bias.contiguous()
    topk_weights = _rows_out(topk_weights, T, K, torch.float32, dev, "topk_weights")
    topk_indices = _rows_out(topk_indices, T, K, torch.int32, dev, "topk_indices")
    if token_expert_indices is True:
        token_expert_indices = torch.empty((T, K), dtype=torch.int32, device=dev)
    elif token_expert_indices is False:
        token_expert_indices = None
    elif token_expert_indices is not None:
        token_expert_indices = _out(token_expert_indices, (T, K), torch.int32, dev,
                                    "token_expert_indices")
    if dense or probs is not None:
        probs = _out(probs, (T, E), logits.dtype, dev, "probs")
    if dense or routing_map is not None:
        routing_map = _out(routing_map, (T, E), torch.bool, dev, "routing_map")
    if dense or scores is not None:
        scores = _out(scores, (T, E), torch.float32, dev, "scores")
    ld_w = topk_weights.stride(0) if T > 0 else K
    ld_i = topk_indices.stride(0) if T > 0 else K
    with _on(dev):
        rc = lib().router_topk_fwd_compact(
            _ptr(logits), _DTYPE[logits.dtype], T, E, K, _score(score_func), int(num_groups),
            int(group_topk), float(scaling_factor), _ptr(expert_bias), _ptr(topk_weights),
            ld_w, _ptr(topk_indices), ld_i, _ptr(token_expert_indices), _ptr(probs),
            _ptr(routing_map), _ptr(scores), _stream(dev))
    _check("router_topk_fwd_compact", rc)
    return topk_weights, topk_indices, token_expert_indices, probs, routing_map, scores


def _maps_outputs(T, E, K, dev, out):
    n = T * K
    names = ("expert_first_token_offset", "permuted_to_unpermuted", "unpermuted_to_permuted",
             "permuted_experts")
    shapes = ((E + 1,), (n,), (n,), (n,))
    out = out or {}
    return tuple(_out(out.get(nm), sh, torch.int32, dev, nm) for nm, sh in zip(names, shapes))


def _workspace(nbytes, workspace, dev):
    if workspace is None:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace needs {nbytes} bytes")
    return workspace


def router_expert_maps(topk_indices: torch.Tensor, E: int, *, out=None, workspace=None):
    """(expert, token)-sorted maps of [T, K] expert choices (int32, unit
    column stride; a column view of a wider buffer is fine).  Returns
    (expert_first_token_offset [E+1], permuted_to_unpermuted [T K],
    unpermuted_to_permuted [T K], permuted_experts [T K]), all int32; the
    choice (t, k) is the expanded row t + k T.  ``out`` may hold any of the
    four by name; the workspace is allocated here when not given."""
    if not topk_indices.is_cuda or topk_indices.dtype != torch.int32 or topk_indices.dim() != 2:
        raise ValueError("topk_indices must be a CUDA int32 [T, K] tensor")
    T, K = topk_indices.shape
    if T > 1 and topk_indices.stride(1) != 1:
        raise ValueError("topk_indices needs a unit column stride")
    dev = topk_indices.device
    ld = topk_indices.stride(0) if T > 0 else K
    offsets, p2u, u2p, pexp = _maps_outputs(T, int(E), K, dev, out)
    workspace = _workspace(lib().router_expert_maps_workspace_bytes(T, int(E)), workspace, dev)
    with _on(dev):
        rc = lib().router_expert_maps(_ptr(topk_indices), ld, T, int(E), K, _ptr(offsets),
                                      _ptr(p2u), _ptr(u2p), _ptr(pexp), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(dev))
    _check("router_expert_maps", rc)
    return offsets, p2u, u2p, pexp


def router_topk_fwd_maps(logits: torch.Tensor, K: int, score_func: str = "softmax",
                         num_groups: int = 0, group_topk: int = 0, scaling_factor: float = 1.0,
                         expert_bias: torch.Tensor | None = None, *, topk_weights=None,
                         topk_indices=None, token_expert_indices=True, out=None,
                         workspace=None):
    """Compact router forward plus the expert maps of its choices (one
    launch for up to 8 aligned tokens).  Returns (topk_weights, topk_indices,
    token_expert_indices or None, expert_first_token_offset,
    permuted_to_unpermuted, unpermuted_to_permuted, permuted_experts)."""
    logits = _as_input(logits, "logits", _DTYPE)
    T, E = logits.shape
    dev = logits.device
    K = int(K)
    if expert_bias is not None:
        if expert_bias.dtype != torch.float32 or expert_bias.numel() != E \
                or expert_bias.get_device() != dev.index:
            raise ValueError("expert_bias must be a float32 [E] tensor on the logits' device")
        expert_bias = expert_bias.contiguous()
    topk_weights = _rows_out(topk_weights, T, K, torch.float32, dev, "topk_weights")
    topk_indices = _rows_out(topk_indices, T, K, torch.int32, dev, "topk_indices")
    if token_expert_indices is True:
        token_expert_indices = torch.empty((T, K), dtype=torch.int32, device=dev)
    elif token_expert_indices is False:
        token_expert_indices = None
    elif token_expert_indices is not None:
        token_expert_indices = _out(token_expert_indices, (T, K), torch.int32, dev,
                                    "token_expert_indices")
    offsets, p2u, u2p, pexp = _maps_outputs(T, E, K, dev, out)
    workspace = _workspace(lib().router_expert_maps_workspace_bytes(T, E), workspace, dev)
    ld_w = topk_weights.stride(0) if T > 0 else K
    ld_i = topk_indices.stride(0) if T > 0 else K
    with _on(dev):
        rc = lib().router_topk_fwd_maps(
            _ptr(logits), _DTYPE[logits.dtype], T, E, K, _score(score_func), int(num_groups),
            int(group_topk), float(scaling_factor), _ptr(expert_bias), _ptr(topk_weights), ld_w,
            _ptr(topk_indices), ld_i, _ptr(token_expert_indices), _ptr(offsets), _ptr(p2u),
            _ptr(u2p), _ptr(pexp), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(dev))
    _check("router_topk_fwd_maps", rc)
    return topk_weights, topk_indices, token_expert_indices, offsets, p2u, u2p, pexp


def router_topk_bwd(grad_probs: torch.Tensor, routing_map: torch.Tensor,
                    scores: torch.Tensor, K: int, score_func: str = "softmax",
                    scaling_factor: float = 1.0, *, grad_logits=None):
    """Top-K router backward.  Returns grad_logits [T,E] in grad_probs' dtype."""
    grad_probs = _as_input(grad_probs, "grad_probs", _DTYPE)
    routing_map = _as_input(routing_map, "routing_map", (torch.bool, torch.uint8))
    scores = _as_input(scores, "scores", (torch.float32,))
    T, E = grad_probs.shape
    if routing_map.shape != grad_probs.shape or scores.shape != grad_probs.shape:
        raise ValueError("grad_probs, routing_map and scores must have the same shape")
    dev = grad_probs.device
    grad_logits = _out(grad_logits, (T, E), grad_probs.dtype, dev, "grad_logits")
    with _on(dev):
        rc = _calls().router_topk_bwd(grad_probs.data_ptr(), routing_map.data_ptr(),
                                      scores.data_ptr(), _DTYPE[grad_probs.dtype], T, E, int(K),
                                      _score(score_func), float(scaling_factor),
                                      grad_logits.data_ptr(), _stream(dev))
    _check("router_topk_bwd", rc)
    return grad_logits


def router_aux_scores_fwd(logits: torch.Tensor, K: int, score_func: str = "softmax", *,
                          scores=None, routing_map=None, intermediate=None):
    """Aux-loss scores forward.  Returns (scores q [T,E] float32,
    routing_map [T,E] bool, intermediate [T,E] float32: sigmoid(x) for sigmoid,
    q for softmax)."""
    logits = _as_input(logits, "logits", _DTYPE)
    T, E = logits.shape
    dev = logits.device
    scores = _out(scores, (T, E), torch.float32, dev, "scores")
    routing_map = _out(routing_map, (T, E), torch.bool, dev, "routing_map")
    if score_func == "sigmoid" or intermediate is not None:
        intermediate = _out(intermediate, (T, E), torch.float32, dev, "intermediate")
    with _on(dev):
        rc = _calls().router_aux_scores_fwd(logits.data_ptr(), _DTYPE[logits.dtype], T, E,
                                            int(K), _score(score_func), scores.data_ptr(),
                                            routing_map.data_ptr(), _ptr0(intermediate),
                                            _stream(dev))
    _check("router_aux_scores_fwd", rc)
    return scores, routing_map, (intermediate if intermediate is not None else scores)


def router_aux_scores_bwd(grad_scores: torch.Tensor, saved: torch.Tensor, K: int,
                          score_func: str = "softmax", dtype: torch.dtype = torch.float32,
                          *, grad_logits=None):
    """Aux-loss scores backward.  ``saved`` is the forward's scores (softmax)
    or intermediate (sigmoid).  Returns grad_logits [T,E] in ``dtype``."""
    grad_scores = _as_input(grad_scores, "grad_scores", (torch.float32,))
    saved = _as_input(saved, "saved", (torch.float32,))
    if saved.shape != grad_scores.shape:
        raise ValueError("grad_scores and saved must have the same shape")
    if dtype not in _DTYPE:
        raise ValueError(f"dtype must be one of {list(_DTYPE)}")
    T, E = grad_scores.shape
    dev = grad_scores.device
    grad_logits = _out(grad_logits, (T, E), dtype, dev, "grad_logits")
    with _on(dev):
        rc = _calls().router_aux_scores_bwd(grad_scores.data_ptr(), saved.data_ptr(),
                                            _DTYPE[dtype], T, E, int(K), _score(score_func),
                                            grad_logits.data_ptr(), _stream(dev))
    _check("router_aux_scores_bwd", rc)
    return grad_logits


def force_path(path: str) -> str:
    """Force the forward kernel path: 'auto', 'segment', 'staged' or 'register';
    returns the previous one."""
    names = {"auto": MR_PATH_AUTO, "segment": MR_PATH_SEGMENT, "staged": MR_PATH_STAGED,
             "register": MR_PATH_REGISTER}
    prev = lib().moe_router_force_path(names[path])
    if prev < 0:
        raise RouterError("moe_router_force_path", prev)
    return {v: k for k, v in names.items()}[prev]


def force_fwd_lanes(lanes: int) -> int:
    """Force the lanes per row of the segment forward (0 = automatic)."""
    prev = lib().moe_router_force_fwd_lanes(int(lanes))
    if prev < 0:
        raise RouterError("moe_router_force_fwd_lanes", prev)
    return prev


def device_status() -> int:
    """Read and clear the current device's status word (0 = no kernel gave
    up a bounded wait).  Synchronous."""
    v = ctypes.c_int(0)
    _check("moe_router_device_status", lib().moe_router_device_status(ctypes.byref(v)))
    return v.value


def selftest_bounded_wait(timeout_us: int, device=None) -> None:
    """Enqueue the diagnostic kernel whose bounded wait always runs out (see
    moe_router_selftest_bounded_wait in the header)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with _on(dev):
        _check("moe_router_selftest_bounded_wait",
               lib().moe_router_selftest_bounded_wait(int(timeout_us), _stream(dev)))


def router_aux_loss_fwd(aux_scores: torch.Tensor, routing_map: torch.Tensor, K: int,
                        coeff: float, *, loss=None, tokens_per_expert=None, workspace=None):
    """Load-balancing aux loss.  Returns (loss [1] float32, tokens_per_expert
    [E] int32).  The workspace (a uint8 CUDA tensor) is allocated here when
    not given."""
    aux_scores = _as_input(aux_scores, "aux_scores", (torch.float32,))
    routing_map = _as_input(routing_map, "routing_map", (torch.bool, torch.uint8))
    if routing_map.shape != aux_scores.shape:
        raise ValueError("aux_scores and routing_map must have the same shape")
    T, E = aux_scores.shape
    dev = aux_scores.device
    loss = _out(loss, (1,), torch.float32, dev, "loss")
    tokens_per_expert = _out(tokens_per_expert, (E,), torch.int32, dev, "tokens_per_expert")
    nbytes = lib().router_aux_loss_workspace_bytes(T, E)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    with _on(dev):
        rc = lib().router_aux_loss_fwd(_ptr(aux_scores), _ptr(routing_map), T, E, int(K),
                                       float(coeff), _ptr(loss), _ptr(tokens_per_expert),
                                       _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream(dev))
    _check("router_aux_loss_fwd", rc)
    return loss, tokens_per_expert


def router_aux_loss_fwd_noalloc(aux_scores: torch.Tensor, routing_map: torch.Tensor, K: int,
                                coeff: float, *, loss: torch.Tensor,
                                tokens_per_expert: torch.Tensor):
    """router_aux_loss_fwd for callers that cannot allocate device memory at
    the call: the library keeps its scratch in a fixed device array, and the
    caller passes the outputs (loss [1] float32, tokens_per_expert [E] int32)
    already allocated.  Calls that overlap on the GPU race on that array; the
    first call on a device looks up its address and belongs before any stream
    capture."""
    aux_scores = _as_input(aux_scores, "aux_scores", (torch.float32,))
    routing_map = _as_input(routing_map, "routing_map", (torch.bool, torch.uint8))
    if routing_map.shape != aux_scores.shape:
        raise ValueError("aux_scores and routing_map must have the same shape")
    T, E = aux_scores.shape
    dev = aux_scores.device
    if loss.get_device() != dev.index or loss.dtype != torch.float32 or loss.numel() < 1:
        raise ValueError("loss must be a float32 tensor on the inputs' device")
    if (tokens_per_expert.get_device() != dev.index or tokens_per_expert.dtype != torch.int32
            or tokens_per_expert.numel() != E or not tokens_per_expert.is_contiguous()):
        raise ValueError("tokens_per_expert must be a contiguous int32 [E] tensor on the "
                         "inputs' device")
    with _on(dev):
        rc = lib().router_aux_loss_fwd_noalloc(_ptr(aux_scores), _ptr(routing_map), T, E, int(K),
                                               float(coeff), _ptr(loss),
                                               _ptr(tokens_per_expert), _stream(dev))
    _check("router_aux_loss_fwd_noalloc", rc)
    return loss, tokens_per_expert


def router_aux_loss_bwd(grad_loss: torch.Tensor, tokens_per_expert: torch.Tensor, T: int, K: int,
                        coeff: float, *, grad_aux_scores=None):
    """Gradient of the aux loss with respect to the aux scores, [T, E] float32."""
    if not grad_loss.is_cuda or grad_loss.dtype != torch.float32 or grad_loss.numel() != 1:
        raise ValueError("grad_loss must be a CUDA float32 tensor with one element")
    if not tokens_per_expert.is_cuda or tokens_per_expert.dtype != torch.int32:
        raise ValueError("tokens_per_expert must be a CUDA int32 tensor")
    E = tokens_per_expert.numel()
    dev = tokens_per_expert.device
    grad_loss = grad_loss.contiguous()
    tokens_per_expert = tokens_per_expert.contiguous()
    grad_aux_scores = _out(grad_aux_scores, (T, E), torch.float32, dev, "grad_aux_scores")
    with _on(dev):
        rc = lib().router_aux_loss_bwd(_ptr(grad_loss), _ptr(tokens_per_expert), int(T), E, int(K),
                                       float(coeff), _ptr(grad_aux_scores), _stream(dev))
    _check("router_aux_loss_bwd", rc)
    return grad_aux_scores


# ---- the experts' products and the combination ------------------------------
# One token's calls take a few microseconds on the GPU, so the host's part is
# written flat: every check reads tensor attributes directly, and the helpers
# below run only to copy a strided input or to say what is wrong.  The two
# gradients of the products, which no single token calls, keep _on and _check.
_I32, _F32, _BF16, _U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
_I8 = torch.int8
_empty = torch.empty


def _bad(name: str, what: str):
    raise ValueError(f"{name} must be {what}")


def _rows_2d(t: torch.Tensor, name: str, index: int | None, dtypes) -> torch.Tensor:
    """Row input that did not pass the caller's quick test: copied if strided,
    refused if wrong."""
    t = _as_input(t, name, dtypes)
    if index is not None and t.get_device() != index:
        _bad(name, f"on cuda:{index}")
    return t


def _map_1d(t: torch.Tensor, name: str, index: int, numel: int | None) -> torch.Tensor:
    """Expert map that did not pass the caller's quick test."""
    if t.get_device() != index or t.dtype is not _I32 or t.dim() != 1 \
            or (numel is not None and t.numel() != numel):
        _bad(name, f"a 1-dimensional int32 tensor"
                   f"{'' if numel is None else f' of {numel} elements'} on cuda:{index}")
    return t.contiguous()


def _weight_3d(t: torch.Tensor, name: str, index: int, dtype):
    """Refuse a weight that did not pass the caller's quick test (a copy at
    each call would cost more than the product)."""
    if t.get_device() != index or t.dtype is not dtype or t.dim() != 3:
        _bad(name, f"a 3-dimensional {dtype} tensor on cuda:{index}")
    _bad(name, "contiguous")


def router_expert_matmul(x: torch.Tensor, weight: torch.Tensor,
                         expert_first_token_offset: torch.Tensor,
                         permuted_to_unpermuted: torch.Tensor | None = None, *, out=None,
                         out_dtype: torch.dtype | None = None):
    """Product of each expert's weight [E, N, D] with its rows.  Returns out
    [P, N] in ``out_dtype`` (default: x's): out[p] = weight[e] x[row(p)] for the
    permuted rows p of expert e.  With ``permuted_to_unpermuted`` (from
    router_expert_maps) x is the tokens [T, D], read through the map; without
    it x is the permuted rows [P, D].  Rows that no expert owns are left as
    they were in ``out``."""
    dt, idx = x.dtype, x.get_device()
    if idx < 0 or dt not in _DTYPE or x.dim() != 2 or not x.is_contiguous():
        x = _rows_2d(x, "x", None, _DTYPE)
    if weight.get_device() != idx or weight.dtype is not dt or weight.dim() != 3 \
            or not weight.is_contiguous():
        _weight_3d(weight, "weight", idx, dt)
    E, N, D = weight.shape
    T, cols = x.shape
    if cols != D:
        _bad("x", f"[rows, {D}]")
    off = expert_first_token_offset
    if off.get_device() != idx or off.dtype is not _I32 or off.numel() != E + 1 \
            or off.dim() != 1 or not off.is_contiguous():
        off = _map_1d(off, "expert_first_token_offset", idx, E + 1)
    p2u = permuted_to_unpermuted
    if p2u is None:
        P, p2u_ptr = T, 0
    else:
        if p2u.get_device() != idx or p2u.dtype is not _I32 or p2u.dim() != 1 \
                or not p2u.is_contiguous():
            p2u = _map_1d(p2u, "permuted_to_unpermuted", idx, None)
        P, p2u_ptr = p2u.numel(), p2u.data_ptr()
    odt = dt if out_dtype is None else out_dtype
    if odt not in _DTYPE:
        _bad("out_dtype", f"one of {list(_DTYPE)}")
    if out is None:
        out = _empty((P, N), dtype=odt, device=x.device)
    else:
        out = _out(out, (P, N), odt, x.device, "out")
    call = (_fast or _calls()).router_expert_matmul
    if idx == _cur_dev():
        rc = call(x.data_ptr(), _DTYPE[dt], weight.data_ptr(), off.data_ptr(), p2u_ptr, T, P, E, N,
                  D, out.data_ptr(), _DTYPE[odt], _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = call(x.data_ptr(), _DTYPE[dt], weight.data_ptr(), off.data_ptr(), p2u_ptr, T, P, E,
                      N, D, out.data_ptr(), _DTYPE[odt], _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_expert_matmul", rc)
    return out


def router_expert_matmul_bwd_input(grad_out: torch.Tensor, weight: torch.Tensor,
                                   expert_first_token_offset: torch.Tensor, *, grad_x=None,
                                   out_dtype: torch.dtype | None = None):
    """Gradient of router_expert_matmul by its rows: grad_x [P, D] on permuted
    rows (``out_dtype``, default grad_out's).  For tokens read through the map,
    router_combine_fwd without weights sums a token's rows."""
    g = grad_out
    idx, dt = g.get_device(), g.dtype
    if idx < 0 or dt not in _DTYPE or g.dim() != 2 or not g.is_contiguous():
        g = _rows_2d(g, "grad_out", None, _DTYPE)
    if weight.get_device() != idx or weight.dtype is not dt or weight.dim() != 3 \
            or not weight.is_contiguous():
        _weight_3d(weight, "weight", idx, dt)
    E, N, D = weight.shape
    off = expert_first_token_offset
    if off.get_device() != idx or off.dtype is not _I32 or off.numel() != E + 1 \
            or off.dim() != 1 or not off.is_contiguous():
        off = _map_1d(off, "expert_first_token_offset", idx, E + 1)
    P, cols = g.shape
    if cols != N:
        _bad("grad_out", f"[P, {N}]")
    odt = dt if out_dtype is None else out_dtype
    if odt not in _DTYPE:
        _bad("out_dtype", f"one of {list(_DTYPE)}")
    if grad_x is None:
        grad_x = _empty((P, D), dtype=odt, device=g.device)
    else:
        grad_x = _out(grad_x, (P, D), odt, g.device, "grad_x")
    with _on(idx):
        rc = (_fast or _calls()).router_expert_matmul_bwd_input(
            g.data_ptr(), _DTYPE[dt], weight.data_ptr(), off.data_ptr(), P, E, N, D,
            grad_x.data_ptr(), _DTYPE[odt], _raw_stream(idx))
    _check("router_expert_matmul_bwd_input", rc)
    return grad_x


def router_expert_matmul_bwd_weight(grad_out: torch.Tensor, x: torch.Tensor,
                                    expert_first_token_offset: torch.Tensor,
                                    permuted_to_unpermuted: torch.Tensor | None = None, *,
                                    grad_weight=None, out_dtype: torch.dtype | None = None):
    """Gradient of router_expert_matmul by its weights: grad_weight [E, N, D] in
    ``out_dtype`` (default: x's); experts without rows get zeros.  x and the
    map as in the forward."""
    g = grad_out
    idx, dt = g.get_device(), g.dtype
    if idx < 0 or dt not in _DTYPE or g.dim() != 2 or not g.is_contiguous():
        g = _rows_2d(g, "grad_out", None, _DTYPE)
    if x.get_device() != idx or x.dtype is not dt or x.dim() != 2 or not x.is_contiguous():
        x = _rows_2d(x, "x", idx, (dt,))
    off = expert_first_token_offset
    if off.get_device() != idx or off.dtype is not _I32 or off.dim() != 1 \
            or not off.is_contiguous():
        off = _map_1d(off, "expert_first_token_offset", idx, None)
    E = off.numel() - 1
    if E < 1:
        _bad("expert_first_token_offset", "of at least two elements")
    T, D = x.shape
    P, N = g.shape
    p2u, p2u_ptr = permuted_to_unpermuted, 0
    if p2u is not None:
        if p2u.get_device() != idx or p2u.dtype is not _I32 or p2u.numel() != P \
                or p2u.dim() != 1 or not p2u.is_contiguous():
            p2u = _map_1d(p2u, "permuted_to_unpermuted", idx, P)
        p2u_ptr = p2u.data_ptr()
    elif T != P:
        _bad("x", f"[{P}, D] without a map")
    odt = dt if out_dtype is None else out_dtype
    if odt not in _DTYPE:
        _bad("out_dtype", f"one of {list(_DTYPE)}")
    if grad_weight is None:
        grad_weight = _empty((E, N, D), dtype=odt, device=g.device)
    else:
        grad_weight = _out(grad_weight, (E, N, D), odt, g.device, "grad_weight")
    with _on(idx):
        rc = (_fast or _calls()).router_expert_matmul_bwd_weight(
            g.data_ptr(), _DTYPE[dt], x.data_ptr(), off.data_ptr(), p2u_ptr, T, P, E, N, D,
            grad_weight.data_ptr(), _DTYPE[odt], _raw_stream(idx))
    _check("router_expert_matmul_bwd_weight", rc)
    return grad_weight


def router_expert_matmul_w4(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                            expert_first_token_offset: torch.Tensor,
                            permuted_to_unpermuted: torch.Tensor | None = None, *,
                            zeros: torch.Tensor | None = None, out=None,
                            out_dtype: torch.dtype | None = None):
    """router_expert_matmul on 4-bit weights (decode batches).  x bf16; qweight
    [E, N, D / 2] uint8, two elements a byte, the even one in the low half;
    scales [E, N, D / group] bf16, zeros the same in uint8 (0..15) or None for
    8; group 32, 64 or 128.  Returns out [P, N] in ``out_dtype`` (default
    bf16)."""
    idx = x.get_device()
    if idx < 0 or x.dtype is not _BF16 or x.dim() != 2 or not x.is_contiguous():
        x = _rows_2d(x, "x", None, (_BF16,))
    if x.data_ptr() & 15:
        x = x.clone()
    if qweight.get_device() != idx or qweight.dtype is not _U8 or qweight.dim() != 3 \
            or not qweight.is_contiguous():
        _weight_3d(qweight, "qweight", idx, _U8)
    if scales.get_device() != idx or scales.dtype is not _BF16 or scales.dim() != 3 \
            or not scales.is_contiguous():
        _weight_3d(scales, "scales", idx, _BF16)
    E, N, half = qweight.shape
    Es, Ns, groups = scales.shape
    D = 2 * half
    if Es != E or Ns != N or groups < 1 or D % groups != 0:
        _bad("scales", "[E, N, D / group]")
    z_ptr = 0
    if zeros is not None:
        if zeros.get_device() != idx or zeros.dtype is not _U8 or zeros.dim() != 3 \
                or not zeros.is_contiguous():
            _weight_3d(zeros, "zeros", idx, _U8)
        if zeros.shape != scales.shape:
            _bad("zeros", "of the shape of scales")
        z_ptr = zeros.data_ptr()
    T, cols = x.shape
    if cols != D:
        _bad("x", f"[rows, {D}]")
    off = expert_first_token_offset
    if off.get_device() != idx or off.dtype is not _I32 or off.numel() != E + 1 \
            or off.dim() != 1 or not off.is_contiguous():
        off = _map_1d(off, "expert_first_token_offset", idx, E + 1)
    p2u = permuted_to_unpermuted
    if p2u is None:
        P, p2u_ptr = T, 0
    else:
        if p2u.get_device() != idx or p2u.dtype is not _I32 or p2u.dim() != 1 \
                or not p2u.is_contiguous():
            p2u = _map_1d(p2u, "permuted_to_unpermuted", idx, None)
        P, p2u_ptr = p2u.numel(), p2u.data_ptr()
    odt = _BF16 if out_dtype is None else out_dtype
    if odt not in _DTYPE:
        _bad("out_dtype", f"one of {list(_DTYPE)}")
    if out is None:
        out = _empty((P, N), dtype=odt, device=x.device)
    else:
        out = _out(out, (P, N), odt, x.device, "out")
    call = (_fast or _calls()).router_expert_matmul_w4
    if idx == _cur_dev():
        rc = call(x.data_ptr(), qweight.data_ptr(), scales.data_ptr(), z_ptr, D // groups,
                  off.data_ptr(), p2u_ptr, T, P, E, N, D, out.data_ptr(), _DTYPE[odt],
                  _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = call(x.data_ptr(), qweight.data_ptr(), scales.data_ptr(), z_ptr, D // groups,
                      off.data_ptr(), p2u_ptr, T, P, E, N, D, out.data_ptr(), _DTYPE[odt],
                      _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_expert_matmul_w4", rc)
    return out


def _vector(t: torch.Tensor, name: str, idx: int, n: int) -> torch.Tensor:
    """A contiguous float32 [n] tensor on the call's device."""
    if t.get_device() != idx or t.dtype is not _F32 or t.dim() != 1 or t.shape[0] != n:
        _bad(name, f"a float32 [{n}] tensor on cuda:{idx}")
    return t if t.is_contiguous() else t.contiguous()


def router_quantize_rows(x: torch.Tensor, *, out=None, scales=None):
    """Rows of x [R, D] in 8-bit integers with a scale for each.  Returns (q [R, D]
    int8, scales [R] float32): scales = max |x| / 127 of the row, q = x / scales to the
    nearest integer, ties to even."""
    dt, idx = x.dtype, x.get_device()
    if idx < 0 or dt not in _DTYPE or x.dim() != 2 or not x.is_contiguous():
        x = _rows_2d(x, "x", None, _DTYPE)
    R, D = x.shape
    if out is None:
        out = _empty((R, D), dtype=_I8, device=x.device)
    else:
        out = _out(out, (R, D), _I8, x.device, "out")
    if scales is None:
        scales = _empty((R,), dtype=_F32, device=x.device)
    else:
        scales = _out(scales, (R,), _F32, x.device, "scales")
    call = (_fast or _calls()).router_quantize_rows
    if idx == _cur_dev():
        rc = call(x.data_ptr(), _DTYPE[dt], R, D, out.data_ptr(), scales.data_ptr(),
                  _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = call(x.data_ptr(), _DTYPE[dt], R, D, out.data_ptr(), scales.data_ptr(),
                      _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_quantize_rows", rc)
    return out, scales


def router_expert_matmul_w8(x: torch.Tensor, x_scales: torch.Tensor, weight: torch.Tensor,
                            weight_scales: torch.Tensor, expert_first_token_offset: torch.Tensor,
                            permuted_to_unpermuted: torch.Tensor | None = None, *, out=None,
                            out_dtype: torch.dtype | None = None):
    """router_expert_matmul on 8-bit integers: x [T or P, D] int8 with a scale for
    each row (router_quantize_rows), weight [E, N, D] int8 with weight_scales [E, N].
    Returns out [P, N] in ``out_dtype`` (default bf16): the products' exact integers
    times both scales.  The maps are as in router_expert_matmul."""
    idx = x.get_device()
    if idx < 0 or x.dtype is not _I8 or x.dim() != 2 or not x.is_contiguous():
        x = _rows_2d(x, "x", None, (_I8,))
    if weight.get_device() != idx or weight.dtype is not _I8 or weight.dim() != 3 \
            or not weight.is_contiguous():
        _weight_3d(weight, "weight", idx, _I8)
    E, N, D = weight.shape
    T, cols = x.shape
    if cols != D:
        _bad("x", f"[rows, {D}]")
    if x_scales.get_device() != idx or x_scales.dtype is not _F32 or x_scales.shape != (T,) \
            or not x_scales.is_contiguous():
        x_scales = _vector(x_scales, "x_scales", idx, T)
    if weight_scales.get_device() != idx or weight_scales.dtype is not _F32 \
            or weight_scales.shape != (E, N) or not weight_scales.is_contiguous():
        _bad("weight_scales", f"a contiguous float32 [{E}, {N}] tensor on cuda:{idx}")
    off = expert_first_token_offset
    if off.get_device() != idx or off.dtype is not _I32 or off.numel() != E + 1 \
            or off.dim() != 1 or not off.is_contiguous():
        off = _map_1d(off, "expert_first_token_offset", idx, E + 1)
    p2u = permuted_to_unpermuted
    if p2u is None:
        P, p2u_ptr = T, 0
    else:
        if p2u.get_device() != idx or p2u.dtype is not _I32 or p2u.dim() != 1 \
                or not p2u.is_contiguous():
            p2u = _map_1d(p2u, "permuted_to_unpermuted", idx, None)
        P, p2u_ptr = p2u.numel(), p2u.data_ptr()
    odt = _BF16 if out_dtype is None else out_dtype
    if odt not in _DTYPE:
        _bad("out_dtype", f"one of {list(_DTYPE)}")
    if out is None:
        out = _empty((P, N), dtype=odt, device=x.device)
    else:
        out = _out(out, (P, N), odt, x.device, "out")
    call = (_fast or _calls()).router_expert_matmul_w8
    if idx == _cur_dev():
        rc = call(x.data_ptr(), x_scales.data_ptr(), weight.data_ptr(), weight_scales.data_ptr(),
                  off.data_ptr(), p2u_ptr, T, P, E, N, D, out.data_ptr(), _DTYPE[odt],
                  _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = call(x.data_ptr(), x_scales.data_ptr(), weight.data_ptr(),
                      weight_scales.data_ptr(), off.data_ptr(), p2u_ptr, T, P, E, N, D,
                      out.data_ptr(), _DTYPE[odt], _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_expert_matmul_w8", rc)
    return out


def _combine_weights(w: torch.Tensor, T: int, K: int, idx: int):
    """Checked combination weights and their row stride (a column view of a
    wider buffer is read in place)."""
    if w.dtype is not _F32 or w.shape != (T, K) or w.get_device() != idx:
        _bad("topk_weights", f"a float32 [{T}, {K}] tensor on cuda:{idx}")
    if w.is_contiguous():
        return w, K
    if w.stride(1) != 1 or w.stride(0) < K:
        return w.contiguous(), K
    return w, w.stride(0)


def router_combine_fwd(expert_out: torch.Tensor, unpermuted_to_permuted: torch.Tensor, K: int,
                       topk_weights: torch.Tensor | None = None, *, out=None):
    """Each token's sum of its K experts' outputs, weighted by ``topk_weights``
    [T, K] (None: plain sums).  expert_out [T K, D] in the maps' order; the map
    is router_expert_maps's.  Returns out [T, D] in expert_out's dtype; a choice
    with map entry -1 adds nothing."""
    z, u2p = expert_out, unpermuted_to_permuted
    idx, dt = z.get_device(), z.dtype
    if idx < 0 or dt not in _DTYPE or z.dim() != 2 or not z.is_contiguous():
        z = _rows_2d(z, "expert_out", None, _DTYPE)
    P, D = z.shape
    if u2p.get_device() != idx or u2p.dtype is not _I32 or u2p.numel() != P \
            or u2p.dim() != 1 or not u2p.is_contiguous():
        u2p = _map_1d(u2p, "unpermuted_to_permuted", idx, P)
    K = int(K)
    if K < 1 or P % K != 0:
        _bad("expert_out", "[T K, D]")
    T = P // K
    w_ptr = ld = 0
    if topk_weights is not None:
        topk_weights, ld = _combine_weights(topk_weights, T, K, idx)
        w_ptr = topk_weights.data_ptr()
    if out is None:
        out = _empty((T, D), dtype=dt, device=z.device)
    else:
        out = _out(out, (T, D), dt, z.device, "out")
    call = (_fast or _calls()).router_combine_fwd
    if idx == _cur_dev():
        rc = call(z.data_ptr(), _DTYPE[dt], u2p.data_ptr(), w_ptr, ld, T, K, D, out.data_ptr(),
                  _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = call(z.data_ptr(), _DTYPE[dt], u2p.data_ptr(), w_ptr, ld, T, K, D, out.data_ptr(),
                      _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_combine_fwd", rc)
    return out


def router_combine_bwd(grad_out: torch.Tensor, unpermuted_to_permuted: torch.Tensor, K: int,
                       expert_out: torch.Tensor | None = None,
                       topk_weights: torch.Tensor | None = None, *, grad_expert_out=None,
                       grad_weights=None):
    """Gradients of router_combine_fwd: (grad_expert_out [T K, D] in grad_out's
    dtype, grad_weights [T, K] float32, or None when ``expert_out`` is None).
    Rows of grad_expert_out that no choice names are left as they were."""
    g, u2p, z = grad_out, unpermuted_to_permuted, expert_out
    idx, dt = g.get_device(), g.dtype
    if idx < 0 or dt not in _DTYPE or g.dim() != 2 or not g.is_contiguous():
        g = _rows_2d(g, "grad_out", None, _DTYPE)
    dev = g.device
    T, D = g.shape
    K = int(K)
    if K < 1:
        _bad("K", "at least 1")
    P = T * K
    if u2p.get_device() != idx or u2p.dtype is not _I32 or u2p.numel() != P \
            or u2p.dim() != 1 or not u2p.is_contiguous():
        u2p = _map_1d(u2p, "unpermuted_to_permuted", idx, P)
    w_ptr = ld = z_ptr = gw_ptr = 0
    if topk_weights is not None:
        topk_weights, ld = _combine_weights(topk_weights, T, K, idx)
        w_ptr = topk_weights.data_ptr()
    if z is not None:
        if z.get_device() != idx or z.dtype is not dt or z.shape != (P, D) \
                or not z.is_contiguous():
            z = _rows_2d(z, "expert_out", idx, (dt,))
            if z.shape != (P, D):
                _bad("expert_out", f"[{P}, {D}]")
        z_ptr = z.data_ptr()
        if grad_weights is None:
            grad_weights = _empty((T, K), dtype=_F32, device=dev)
        else:
            grad_weights = _out(grad_weights, (T, K), _F32, dev, "grad_weights")
        gw_ptr = grad_weights.data_ptr()
    elif grad_weights is not None:
        raise ValueError("grad_weights needs expert_out")
    if grad_expert_out is None:
        grad_expert_out = _empty((P, D), dtype=dt, device=dev)
    else:
        grad_expert_out = _out(grad_expert_out, (P, D), dt, dev, "grad_expert_out")
    call = (_fast or _calls()).router_combine_bwd
    if idx == _cur_dev():
        rc = call(g.data_ptr(), _DTYPE[dt], u2p.data_ptr(), z_ptr, w_ptr, ld, T, K, D,
                  grad_expert_out.data_ptr(), gw_ptr, _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = call(g.data_ptr(), _DTYPE[dt], u2p.data_ptr(), z_ptr, w_ptr, ld, T, K, D,
                      grad_expert_out.data_ptr(), gw_ptr, _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_combine_bwd", rc)
    return grad_expert_out, grad_weights


# ---- the balance loss of a packed batch -----------------------------------------
def _sequences(seq_offsets, idx: int) -> tuple[int, int]:
    """(S, pointer) of a packed batch's sequence offsets [S + 1]."""
    n = seq_offsets.numel()
    if seq_offsets.get_device() != idx or seq_offsets.dtype is not _I32 \
            or seq_offsets.dim() != 1 or n < 2 or not seq_offsets.is_contiguous():
        _bad("seq_offsets", f"a contiguous int32 [S + 1] tensor on cuda:{idx}")
    return n - 1, seq_offsets.data_ptr()


def router_balance_loss_fwd(logits: torch.Tensor, topk_indices: torch.Tensor,
                            score_func: str = "softmax", coeff: float = 1.0, z_coeff: float = 0.0,
                            seq_offsets: torch.Tensor | None = None, *, loss=None,
                            tokens_per_expert=None, row_stats=None, workspace=None):
    """Load-balancing loss of each sequence of a packed batch, and the z loss, from the
    logits [T, E] and the choices [T, K] int32 (router_topk_fwd_compact's; a column
    view of a wider buffer is read in place).  ``seq_offsets`` [S + 1] int32: sequence s
    is tokens seq_offsets[s] .. seq_offsets[s + 1] - 1, other tokens are padding; None:
    all tokens are one.  Returns (loss [2] float32: balance and z loss,
    tokens_per_expert [S, E] int32, row_stats [T, 2] float32 for the backward).  The
    workspace (a uint8 CUDA tensor) is allocated here when not given."""
    x, dt, idx = logits, logits.dtype, logits.get_device()
    if idx < 0 or dt not in _DTYPE or x.dim() != 2 or not x.is_contiguous():
        x = _as_input(x, "logits", _DTYPE)
    T, E = x.shape
    dev = x.device
    choices = topk_indices
    if choices.get_device() != idx or choices.dtype is not _I32 or choices.dim() != 2 \
            or choices.shape[0] != T or choices.shape[1] < 1:
        _bad("topk_indices", f"an int32 [{T}, K] tensor on cuda:{idx}")
    ld = K = choices.shape[1]
    if not choices.is_contiguous():
        if choices.stride(1) != 1 or choices.stride(0) < K:
            choices = choices.contiguous()
        else:
            ld = choices.stride(0)
    S, seq_ptr = (1, 0) if seq_offsets is None else _sequences(seq_offsets, idx)
    loss = _empty((2,), dtype=_F32, device=dev) if loss is None \
        else _out(loss, (2,), _F32, dev, "loss")
    counts = _empty((S, E), dtype=_I32, device=dev) if tokens_per_expert is None \
        else _out(tokens_per_expert, (S, E), _I32, dev, "tokens_per_expert")
    stats = _empty((T, 2), dtype=_F32, device=dev) if row_stats is None \
        else _out(row_stats, (T, 2), _F32, dev, "row_stats")
    calls = _fast or _calls()
    if workspace is None:
        nbytes = calls.router_balance_loss_workspace_bytes(T, E, S) or 16
        workspace = _empty((nbytes,), dtype=_U8, device=dev)
    else:
        if workspace.get_device() != idx or not workspace.is_contiguous():
            _bad("workspace", f"a contiguous tensor on cuda:{idx}")
        nbytes = workspace.numel() * workspace.element_size()
    sf, coeff, z_coeff = _score(score_func), float(coeff), float(z_coeff)
    if idx == _cur_dev():
        rc = calls.router_balance_loss_fwd(
            x.data_ptr(), _DTYPE[dt], choices.data_ptr(), ld, seq_ptr, T, E, K, S, sf, coeff,
            z_coeff, loss.data_ptr(), counts.data_ptr(), stats.data_ptr(), workspace.data_ptr(),
            nbytes, _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = calls.router_balance_loss_fwd(
                x.data_ptr(), _DTYPE[dt], choices.data_ptr(), ld, seq_ptr, T, E, K, S, sf, coeff,
                z_coeff, loss.data_ptr(), counts.data_ptr(), stats.data_ptr(),
                workspace.data_ptr(), nbytes, _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_balance_loss_fwd", rc)
    return loss, counts, stats


def router_balance_loss_bwd(grad_loss: torch.Tensor, logits: torch.Tensor,
                            tokens_per_expert: torch.Tensor, row_stats: torch.Tensor, K: int,
                            score_func: str = "softmax", coeff: float = 1.0, z_coeff: float = 0.0,
                            seq_offsets: torch.Tensor | None = None, *, grad_logits=None):
    """Gradient of both losses by the logits, [T, E] in the logits' dtype; padding gets
    zeros.  ``grad_loss`` [2] float32; the other arguments are the forward's."""
    x, dt, idx = logits, logits.dtype, logits.get_device()
    if idx < 0 or dt not in _DTYPE or x.dim() != 2 or not x.is_contiguous():
        x = _as_input(x, "logits", _DTYPE)
    T, E = x.shape
    S, seq_ptr = (1, 0) if seq_offsets is None else _sequences(seq_offsets, idx)
    g, counts, stats = grad_loss, tokens_per_expert, row_stats
    if g.get_device() != idx or g.dtype is not _F32 or g.shape != (2,) or not g.is_contiguous():
        g = _vector(g, "grad_loss", idx, 2)
    if counts.get_device() != idx or counts.dtype is not _I32 or counts.shape != (S, E) \
            or not counts.is_contiguous():
        _bad("tokens_per_expert", f"a contiguous int32 [{S}, {E}] tensor on cuda:{idx}")
    if stats.get_device() != idx or stats.dtype is not _F32 or stats.shape != (T, 2) \
            or not stats.is_contiguous():
        _bad("row_stats", f"a contiguous float32 [{T}, 2] tensor on cuda:{idx}")
    out = _empty((T, E), dtype=dt, device=x.device) if grad_logits is None \
        else _out(grad_logits, (T, E), dt, x.device, "grad_logits")
    sf, K, coeff, z_coeff = _score(score_func), int(K), float(coeff), float(z_coeff)
    call = (_fast or _calls()).router_balance_loss_bwd
    if idx == _cur_dev():
        rc = call(g.data_ptr(), x.data_ptr(), _DTYPE[dt], counts.data_ptr(), stats.data_ptr(),
                  seq_ptr, T, E, K, S, sf, coeff, z_coeff, out.data_ptr(), _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = call(g.data_ptr(), x.data_ptr(), _DTYPE[dt], counts.data_ptr(),
                      stats.data_ptr(), seq_ptr, T, E, K, S, sf, coeff, z_coeff, out.data_ptr(),
                      _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_balance_loss_bwd", rc)
    return out


# ---- the norms around an expert block ------------------------------------------
_GATE_TOKEN, _GATE_VALUE = 1, 2  # 0: none


def _gate(gate, T: int, D: int, dt, idx: int):
    """(tensor, kind) of a block's gate: [T] float32, or [T, D] of the rows' type."""
    if gate.get_device() == idx:
        if gate.shape == (T,) and gate.dtype is _F32:
            return gate if gate.is_contiguous() else gate.contiguous(), _GATE_TOKEN
        if gate.shape == (T, D) and gate.dtype is dt:
            return gate if gate.is_contiguous() else gate.contiguous(), _GATE_VALUE
    _bad("gate", f"a float32 [{T}] or a {dt} [{T}, {D}] tensor on cuda:{idx}")


def _same_rows(t: torch.Tensor, name: str, shape, dt, idx: int) -> torch.Tensor:
    """A [T, D] tensor of the call's type and device."""
    if t.get_device() != idx or t.dtype is not dt or t.shape != shape:
        _bad(name, f"a {dt} {list(shape)} tensor on cuda:{idx}")
    return t if t.is_contiguous() else t.contiguous()


def router_combine_norm_fwd(expert_out: torch.Tensor, residual: torch.Tensor,
                            unpermuted_to_permuted: torch.Tensor | None = None,
                            topk_weights: torch.Tensor | None = None, *,
                            post_weight: torch.Tensor | None = None,
                            gate: torch.Tensor | None = None, residual_scale: float = 1.0,
                            pre_weight: torch.Tensor | None = None, eps: float = 1e-6,
                            save: bool = False, sum=None, normed=None, block_out=None, rstd=None):
    """The end of an expert block in one call: y, each token's weighted sum of its
    experts' outputs (as router_combine_fwd; without a map expert_out [T, D] itself), the
    RMS norm behind the block (``post_weight`` [D] float32), its gate ([T] float32 or
    [T, D]), x = residual + residual_scale gate norm(y), and the RMS norm of x before the
    next block (``pre_weight``).  Returns (x [T, D], normed [T, D] or None, y [T, D] or
    None, rstd [T, 2] float32 or None); the last two, for the backward, with
    ``save=True`` or when given."""
    res = residual
    idx, dt = res.get_device(), res.dtype
    if idx < 0 or dt not in _DTYPE or res.dim() != 2 or not res.is_contiguous():
        res = _rows_2d(res, "residual", None, _DTYPE)
    T, D = res.shape
    dev = res.device
    z, u2p = expert_out, unpermuted_to_permuted
    if z.get_device() != idx or z.dtype is not dt or z.dim() != 2 or z.shape[1] != D \
            or not z.is_contiguous():
        z = _rows_2d(z, "expert_out", idx, (dt,))
        if z.shape[1] != D:
            _bad("expert_out", f"[T K, {D}]")
    P = z.shape[0]
    K, u2p_ptr, w_ptr, ld = 1, 0, 0, 0
    if u2p is not None:
        if T > 0:
            K = P // T
        if K < 1 or P != T * K:
            _bad("expert_out", f"[{T} K, {D}]")
        if u2p.get_device() != idx or u2p.dtype is not _I32 or u2p.numel() != P \
                or u2p.dim() != 1 or not u2p.is_contiguous():
            u2p = _map_1d(u2p, "unpermuted_to_permuted", idx, P)
        u2p_ptr = u2p.data_ptr()
        if topk_weights is not None and T > 0:
            topk_weights, ld = _combine_weights(topk_weights, T, K, idx)
            w_ptr = topk_weights.data_ptr()
    else:
        if topk_weights is not None:
            raise ValueError("topk_weights needs unpermuted_to_permuted")
        if P != T:
            _bad("expert_out", f"[{T}, {D}] without a map")
    post_ptr = pre_ptr = normed_ptr = 0
    if post_weight is not None:
        post_weight = _vector(post_weight, "post_weight", idx, D)
        post_ptr = post_weight.data_ptr()
    gate_ptr = kind = 0
    if gate is not None:
        gate, kind = _gate(gate, T, D, dt, idx)
        gate_ptr = gate.data_ptr()
    if pre_weight is not None:
        pre_weight = _vector(pre_weight, "pre_weight", idx, D)
        pre_ptr = pre_weight.data_ptr()
        normed = _empty((T, D), dtype=dt, device=dev) if normed is None \
            else _out(normed, (T, D), dt, dev, "normed")
        normed_ptr = normed.data_ptr()
    elif normed is not None:
        raise ValueError("normed needs pre_weight")
    sum = _empty((T, D), dtype=dt, device=dev) if sum is None \
        else _out(sum, (T, D), dt, dev, "sum")
    block_ptr = rstd_ptr = 0
    if save or block_out is not None:
        block_out = _out(block_out, (T, D), dt, dev, "block_out")
        block_ptr = block_out.data_ptr()
    if save or rstd is not None:
        rstd = _out(rstd, (T, 2), _F32, dev, "rstd")
        rstd_ptr = rstd.data_ptr()
    call = (_fast or _calls()).router_combine_norm_fwd
    if idx == _cur_dev():
        rc = call(z.data_ptr(), _DTYPE[dt], u2p_ptr, w_ptr, ld, res.data_ptr(), post_ptr, gate_ptr,
                  kind, float(residual_scale), pre_ptr, float(eps), T, K, D, sum.data_ptr(), normed_ptr,
                  block_ptr, rstd_ptr, _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = call(z.data_ptr(), _DTYPE[dt], u2p_ptr, w_ptr, ld, res.data_ptr(), post_ptr,
                      gate_ptr, kind, float(residual_scale), pre_ptr, float(eps), T, K, D,
                      sum.data_ptr(), normed_ptr, block_ptr, rstd_ptr, _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_combine_norm_fwd", rc)
    return sum, normed, block_out, rstd


def router_combine_norm_bwd(grad_sum: torch.Tensor | None, grad_normed: torch.Tensor | None,
                            block_out: torch.Tensor | None, sum: torch.Tensor | None,
                            rstd: torch.Tensor | None, *,
                            post_weight: torch.Tensor | None = None,
                            gate: torch.Tensor | None = None, residual_scale: float = 1.0,
                            pre_weight: torch.Tensor | None = None, grad_block=None,
                            grad_residual=None, grad_gate=None, grad_post_weight=None,
                            grad_pre_weight=None, workspace=None):
    """Gradients of router_combine_norm_fwd from those of x and of the normed rows
    (``grad_sum`` may be None with a pre_weight): (grad_block [T, D], the gradient of y
    and router_combine_bwd's grad_out; grad_residual [T, D]; grad_gate like the gate;
    grad_post_weight and grad_pre_weight [D] float32), None for what the forward did
    not have.  ``block_out``, ``sum`` and ``rstd`` are the forward's; without a
    pre_weight ``sum`` and ``grad_normed`` are not read and may be None, block_out
    neither without a post_weight and a gate.  The workspace (a uint8 CUDA tensor) is
    allocated here when not given."""
    rows = grad_sum if grad_sum is not None else grad_normed
    if rows is None:
        raise ValueError("grad_sum or grad_normed must be given")
    idx, dt = rows.get_device(), rows.dtype
    if idx < 0 or dt not in _DTYPE or rows.dim() != 2:
        rows = _rows_2d(rows, "grad_sum", None, _DTYPE)
    T, D = rows.shape
    shape, dev = (T, D), rows.device
    gs_ptr = gn_ptr = x_ptr = y_ptr = rstd_ptr = 0
    post_ptr = pre_ptr = gate_ptr = kind = gpost_ptr = gpre_ptr = ggate_ptr = ws_ptr = nbytes = 0
    pre, post = pre_weight is not None, post_weight is not None
    if grad_sum is not None:
        grad_sum = _same_rows(grad_sum, "grad_sum", shape, dt, idx)
        gs_ptr = grad_sum.data_ptr()
    elif not pre:
        raise ValueError("grad_sum must be given without a pre_weight")
    if pre:
        if grad_normed is None or sum is None:
            raise ValueError("pre_weight needs grad_normed and sum")
        grad_normed = _same_rows(grad_normed, "grad_normed", shape, dt, idx)
        sum = _same_rows(sum, "sum", shape, dt, idx)
        pre_weight = _vector(pre_weight, "pre_weight", idx, D)
        grad_pre_weight = _empty((D,), dtype=_F32, device=dev) if grad_pre_weight is None \
            else _out(grad_pre_weight, (D,), _F32, dev, "grad_pre_weight")
        gn_ptr, x_ptr = grad_normed.data_ptr(), sum.data_ptr()
        pre_ptr, gpre_ptr = pre_weight.data_ptr(), grad_pre_weight.data_ptr()
    else:
        grad_pre_weight = None
    if gate is not None:
        gate, kind = _gate(gate, T, D, dt, idx)
        grad_gate = _empty(gate.shape, dtype=gate.dtype, device=dev) if grad_gate is None \
            else _out(grad_gate, tuple(gate.shape), gate.dtype, dev, "grad_gate")
        gate_ptr, ggate_ptr = gate.data_ptr(), grad_gate.data_ptr()
    else:
        grad_gate = None
    if post or kind:
        if block_out is None:
            raise ValueError("post_weight and a gate need block_out")
        block_out = _same_rows(block_out, "block_out", shape, dt, idx)
        y_ptr = block_out.data_ptr()
    if post:
        post_weight = _vector(post_weight, "post_weight", idx, D)
        grad_post_weight = _empty((D,), dtype=_F32, device=dev) if grad_post_weight is None \
            else _out(grad_post_weight, (D,), _F32, dev, "grad_post_weight")
        post_ptr, gpost_ptr = post_weight.data_ptr(), grad_post_weight.data_ptr()
    else:
        grad_post_weight = None
    calls = _fast or _calls()
    if pre or post:
        if rstd is None or rstd.get_device() != idx or rstd.dtype is not _F32 \
                or rstd.shape != (T, 2) or not rstd.is_contiguous():
            _bad("rstd", f"a contiguous float32 [{T}, 2] tensor on cuda:{idx}")
        rstd_ptr = rstd.data_ptr()
        if workspace is None:
            nbytes = calls.router_combine_norm_bwd_workspace_bytes(T, D) or 16
            workspace = _empty((nbytes,), dtype=_U8, device=dev)
        else:
            if workspace.get_device() != idx or not workspace.is_contiguous():
                _bad("workspace", f"a contiguous tensor on cuda:{idx}")
            nbytes = workspace.numel() * workspace.element_size()
        ws_ptr = workspace.data_ptr()
    grad_block = _empty(shape, dtype=dt, device=dev) if grad_block is None \
        else _out(grad_block, shape, dt, dev, "grad_block")
    grad_residual = _empty(shape, dtype=dt, device=dev) if grad_residual is None \
        else _out(grad_residual, shape, dt, dev, "grad_residual")
    args = (gs_ptr, gn_ptr, _DTYPE[dt], y_ptr, x_ptr, rstd_ptr, post_ptr, gate_ptr, kind,
            float(residual_scale), pre_ptr, T, D, grad_block.data_ptr(), grad_residual.data_ptr(),
            ggate_ptr, gpost_ptr, gpre_ptr, ws_ptr, nbytes)
    if idx == _cur_dev():
        rc = calls.router_combine_norm_bwd(*args, _raw_stream(idx))
    else:
        with torch.cuda.device(idx):
            rc = calls.router_combine_norm_bwd(*args, _raw_stream(idx))
    if rc != 0:
        raise RouterError("router_combine_norm_bwd", rc)
    return grad_block, grad_residual, grad_gate, grad_post_weight, grad_pre_weight
