"""Python binding of libpkm.so, the B200 (sm_100a) product-key memory library.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. The functions carry the names of the C entry points in include/pkm.h.
PyTorch supplies device memory and the current stream.

The library must have been built (``python product_key_memory_b200/build.py``);
importing this package raises if libpkm.so is missing. There is no CPU path.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# PKM_LIBRARY selects another build of the library (the timeout test build).
LIB_PATH = os.environ.get("PKM_LIBRARY") or os.path.join(_HERE, "libpkm.so")

PKM_F32, PKM_BF16 = 0, 1
PKM_OK = 0
PKM_OPT_PATH, PKM_OPT_SUBBATCHES = 0, 1
PKM_PATH_AUTO, PKM_PATH_TC, PKM_PATH_SIMT, PKM_PATH_SMALL_FUSED, PKM_PATH_SMALL_SPLIT = range(5)
_PATHS = {"auto": PKM_PATH_AUTO, "tc": PKM_PATH_TC, "simt": PKM_PATH_SIMT,
          "small_fused": PKM_PATH_SMALL_FUSED, "small_split": PKM_PATH_SMALL_SPLIT}
PKM_ACT_NONE, PKM_ACT_RELU, PKM_ACT_GELU, PKM_ACT_SILU = range(4)
_ACTS = {"none": PKM_ACT_NONE, "relu": PKM_ACT_RELU, "gelu": PKM_ACT_GELU, "silu": PKM_ACT_SILU}
_STATUS = {0: "PKM_OK", -1: "PKM_ERR_INVALID_ARG", -2: "PKM_ERR_UNSUPPORTED",
           -3: "PKM_ERR_WORKSPACE", -4: "PKM_ERR_CUDA", -5: "PKM_ERR_DEVICE"}

EXPORTED = ("pkm_workspace_size", "pkm_forward", "pkm_backward_values", "pkm_device_status",
            "pkm_trace_enable", "pkm_trace_read", "pkm_status_string",
            "pkm_backward_values_noalloc", "pkm_slot_usage", "pkm_backward",
            "pkm_forward_train", "pkm_backward_train", "pkm_set_option", "pkm_get_option",
            "pkm_norm_workspace_size", "pkm_layernorm_forward", "pkm_layernorm_backward",
            "pkm_adamw_step", "pkm_linear_workspace_size", "pkm_linear_forward",
            "pkm_linear_backward")


class PKMError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__("%s returned %s (%d): %s" % (fn, _STATUS.get(code, "?"), code,
                                                      pkm_status_string(code)))
        self.code = code


class pkm_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("d_model", ctypes.c_int32), ("H", ctypes.c_int32),
                ("dq", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32),
                ("v", ctypes.c_int32), ("dtype", ctypes.c_int32), ("bn_eps", ctypes.c_float)]


class pkm_norm_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("d", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("add_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class pkm_linear_shape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


class pkm_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("weight_decay", ctypes.c_float), ("lr_scale", ctypes.c_float)]


class pkm_adamw_hyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint32),
                ("zero_grad", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libpkm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("%s not built: run python product_key_memory_b200/build.py"
                              % os.path.basename(LIB_PATH))
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        S = ctypes.POINTER(pkm_shape)
        L.pkm_workspace_size.argtypes = [S, ctypes.c_int]
        L.pkm_workspace_size.restype = ctypes.c_size_t
        L.pkm_forward.argtypes = [S] + [P] * 13 + [ctypes.c_size_t, P]
        L.pkm_forward.restype = ctypes.c_int
        L.pkm_backward_values.argtypes = [S] + [P] * 7 + [ctypes.c_size_t, P]
        L.pkm_backward_values.restype = ctypes.c_int
        L.pkm_backward.argtypes = [S] + [P] * 19 + [ctypes.c_size_t, P]
        L.pkm_backward.restype = ctypes.c_int
        L.pkm_backward_train.argtypes = [S] + [P] * 19 + [ctypes.c_size_t, P]
        L.pkm_backward_train.restype = ctypes.c_int
        L.pkm_forward_train.argtypes = [S] + [P] * 6 + [ctypes.c_float] + [P] * 9 + [
            ctypes.c_size_t, P]
        L.pkm_forward_train.restype = ctypes.c_int
        L.pkm_backward_values_noalloc.argtypes = [S] + [P] * 6 + [P]
        L.pkm_backward_values_noalloc.restype = ctypes.c_int
        L.pkm_slot_usage.argtypes = [S, P, P, P, ctypes.c_size_t, P]
        L.pkm_slot_usage.restype = ctypes.c_int
        L.pkm_device_status.argtypes = [P, P]
        L.pkm_device_status.restype = ctypes.c_int
        L.pkm_trace_enable.argtypes = [ctypes.c_int]
        L.pkm_trace_enable.restype = ctypes.c_int
        L.pkm_trace_read.argtypes = [ctypes.c_int, P, ctypes.c_int, P, P]
        L.pkm_trace_read.restype = ctypes.c_int
        L.pkm_set_option.argtypes = [ctypes.c_int, ctypes.c_int]
        L.pkm_set_option.restype = ctypes.c_int
        L.pkm_get_option.argtypes = [ctypes.c_int]
        L.pkm_get_option.restype = ctypes.c_int
        N = ctypes.POINTER(pkm_norm_shape)
        L.pkm_norm_workspace_size.argtypes = [N]
        L.pkm_norm_workspace_size.restype = ctypes.c_size_t
        L.pkm_layernorm_forward.argtypes = [N] + [P] * 9
        L.pkm_layernorm_forward.restype = ctypes.c_int
        L.pkm_layernorm_backward.argtypes = [N] + [P] * 10 + [ctypes.c_size_t, P]
        L.pkm_layernorm_backward.restype = ctypes.c_int
        D = ctypes.POINTER(pkm_linear_shape)
        L.pkm_linear_workspace_size.argtypes = [D, ctypes.c_int]
        L.pkm_linear_workspace_size.restype = ctypes.c_size_t
        L.pkm_linear_forward.argtypes = [D] + [P] * 7 + [ctypes.c_size_t, P]
        L.pkm_linear_forward.restype = ctypes.c_int
        L.pkm_linear_backward.argtypes = [D] + [P] * 8 + [ctypes.c_size_t, P]
        L.pkm_linear_backward.restype = ctypes.c_int
        L.pkm_adamw_step.argtypes = [ctypes.POINTER(pkm_adamw_tensor), ctypes.c_int64,
                                     ctypes.POINTER(pkm_adamw_hyper), P, P]
        L.pkm_adamw_step.restype = ctypes.c_int
        L.pkm_status_string.argtypes = [ctypes.c_int]
        L.pkm_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


lib()  # fail loudly at import when the library is missing


def pkm_status_string(code: int) -> str:
    return lib().pkm_status_string(int(code)).decode()


def pkm_set_option(option: int, value: int) -> None:
    rc = lib().pkm_set_option(int(option), int(value))
    if rc != PKM_OK:
        raise PKMError("pkm_set_option", rc)


def pkm_get_option(option: int) -> int:
    rc = int(lib().pkm_get_option(int(option)))
    if rc < 0:
        raise PKMError("pkm_get_option", rc)
    return rc


class options:
    """Context manager that sets the library's implementation switches and restores
    them on exit: ``with options(path="simt"): ...`` (path: "auto", "tc", "simt",
    "small_fused" or "small_split"; subbatches: 1..4)."""

    def __init__(self, path: Optional[str] = None, subbatches: Optional[int] = None):
        self.want = {}
        if path is not None:
            self.want[PKM_OPT_PATH] = _PATHS[path]
        if subbatches is not None:
            self.want[PKM_OPT_SUBBATCHES] = int(subbatches)

    def __enter__(self):
        self.old = {o: pkm_get_option(o) for o in self.want}
        for o, v in self.want.items():
            pkm_set_option(o, v)
        return self

    def __exit__(self, *exc):
        for o, v in self.old.items():
            pkm_set_option(o, v)


def make_shape(B, d_model, H, dq, n, k, v, dtype, bn_eps=1e-5) -> pkm_shape:
    dt = dtype if isinstance(dtype, int) else (PKM_BF16 if dtype == torch.bfloat16 else PKM_F32)
    return pkm_shape(int(B), int(d_model), int(H), int(dq), int(n), int(k), int(v), dt,
                     float(bn_eps))


def pkm_workspace_size(shape: pkm_shape, for_backward: bool = False) -> int:
    return int(lib().pkm_workspace_size(ctypes.byref(shape), int(bool(for_backward))))


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libpkm takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libpkm takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def alloc_workspace(shape: pkm_shape, for_backward: bool = False,
                    device=None) -> torch.Tensor:
    n = pkm_workspace_size(shape, for_backward)
    if n == 0:
        raise PKMError("pkm_workspace_size", -1)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def pkm_forward(x: torch.Tensor, W_q: torch.Tensor, bn_mean: torch.Tensor,
                bn_var: torch.Tensor, bn_gamma: torch.Tensor, bn_beta: torch.Tensor,
                subkeys: torch.Tensor, values: torch.Tensor, k: int, bn_eps: float = 1e-5,
                out: Optional[torch.Tensor] = None, indices: Optional[torch.Tensor] = None,
                weights: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                want_scores: bool = True, workspace: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor,
                                      Optional[torch.Tensor]]:
    """Run the PKM forward on the current CUDA stream.

    x [B][d_model], W_q [H*dq][d_model], BN vectors [H*dq] fp32, subkeys [H][2][n][dq/2],
    values [n*n][v] -- x, W_q, subkeys, values all fp32 or all bf16.
    Returns (out [B][v] fp32, indices [B][H][k] int32, weights [B][H][k] fp32,
    scores [B][H][k] fp32 or None). Missing outputs are allocated here.
    """
    B, d = x.shape
    H, two, n, half = subkeys.shape
    if two != 2:
        raise ValueError("subkeys must be [H][2][n][dq/2]")
    v = values.shape[1]
    shape = make_shape(B, d, H, 2 * half, n, k, v, x.dtype, bn_eps)
    dev = x.device
    if out is None:
        out = torch.empty(B, v, dtype=torch.float32, device=dev)
    if indices is None:
        indices = torch.empty(B, H, k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(B, H, k, dtype=torch.float32, device=dev)
    if scores is None and want_scores:
        scores = torch.empty(B, H, k, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(shape, False, dev)
    rc = lib().pkm_forward(ctypes.byref(shape), _ptr(x), _ptr(W_q), _ptr(bn_mean), _ptr(bn_var),
                           _ptr(bn_gamma), _ptr(bn_beta), _ptr(subkeys), _ptr(values), _ptr(out),
                           _ptr(indices), _ptr(weights), _ptr(scores), _ptr(workspace),
                           workspace.numel(), _stream(stream))
    if rc != PKM_OK:
        raise PKMError("pkm_forward", rc)
    return out, indices, weights, scores


def pkm_backward_values(values: torch.Tensor, indices: torch.Tensor, weights: torch.Tensor,
                        grad_out: torch.Tensor, grad_values: torch.Tensor,
                        grad_scores: Optional[torch.Tensor], n: int,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Sparse value backward. grad_values [n*n][v] fp32 is accumulated into;
    grad_scores [B][H][k] fp32 is overwritten (may be None)."""
    B, H, k = indices.shape
    v = values.shape[1]
    shape = make_shape(B, 0, H, 0, n, k, v, values.dtype)
    if workspace is None:
        workspace = alloc_workspace(shape, True, values.device)
    rc = lib().pkm_backward_values(ctypes.byref(shape), _ptr(values), _ptr(indices),
                                   _ptr(weights), _ptr(grad_out), _ptr(grad_values),
                                   _ptr(grad_scores), _ptr(workspace), workspace.numel(),
                                   _stream(stream))
    if rc != PKM_OK:
        raise PKMError("pkm_backward_values", rc)
    return grad_values, grad_scores


def pkm_forward_train(x: torch.Tensor, W_q: torch.Tensor, bn_running_mean: torch.Tensor,
                      bn_running_var: torch.Tensor, bn_gamma: torch.Tensor,
                      bn_beta: torch.Tensor, subkeys: torch.Tensor, values: torch.Tensor, k: int,
                      momentum: float = 0.1, bn_eps: float = 1e-5,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """Forward with BatchNorm in training mode. Updates bn_running_mean/var in place;
    returns (out, indices, weights, scores, batch_mean, batch_var)."""
    B, d = x.shape
    H, _, n, half = subkeys.shape
    v = values.shape[1]
    F = H * 2 * half
    shape = make_shape(B, d, H, 2 * half, n, k, v, x.dtype, bn_eps)
    dev = x.device
    if workspace is None:
        nb = int(lib().pkm_workspace_size(ctypes.byref(shape), 4))
        if nb == 0:
            raise PKMError("pkm_workspace_size", -1)
        workspace = torch.empty(nb, dtype=torch.uint8, device=dev)
    out = torch.empty(B, v, dtype=torch.float32, device=dev)
    idx = torch.empty(B, H, k, dtype=torch.int32, device=dev)
    wts = torch.empty(B, H, k, dtype=torch.float32, device=dev)
    scs = torch.empty(B, H, k, dtype=torch.float32, device=dev)
    bm = torch.empty(F, dtype=torch.float32, device=dev)
    bv = torch.empty(F, dtype=torch.float32, device=dev)
    rc = lib().pkm_forward_train(ctypes.byref(shape), _ptr(x), _ptr(W_q), _ptr(bn_running_mean),
                                 _ptr(bn_running_var), _ptr(bn_gamma), _ptr(bn_beta),
                                 ctypes.c_float(momentum), _ptr(subkeys), _ptr(values), _ptr(out),
                                 _ptr(idx), _ptr(wts), _ptr(scs), _ptr(bm), _ptr(bv),
                                 _ptr(workspace), workspace.numel(), _stream(stream))
    if rc != PKM_OK:
        raise PKMError("pkm_forward_train", rc)
    return out, idx, wts, scs, bm, bv


def pkm_backward(x: torch.Tensor, W_q: torch.Tensor, bn_mean: torch.Tensor,
                 bn_var: torch.Tensor, bn_gamma: torch.Tensor, bn_beta: torch.Tensor,
                 subkeys: torch.Tensor, values: torch.Tensor, indices: torch.Tensor,
                 weights: torch.Tensor, grad_out: torch.Tensor, grads: dict,
                 bn_eps: float = 1e-5, workspace: Optional[torch.Tensor] = None, stream=None,
                 bn_training: bool = False):
    """Full backward of the layer with the forward's picks held fixed.

    ``grads`` maps any of x [B][d], W_q [H*dq][d], bn_gamma, bn_beta [H*dq],
    subkeys [H][2][n][dq/2], values [n*n][v], scores [B][H][k] to fp32 device
    tensors; missing entries are not computed. values is accumulated into, the
    others are overwritten. With bn_training, bn_mean / bn_var are the batch
    statistics pkm_forward_train returned (pkm_backward_train)."""
    B, d = x.shape
    H, _, n, half = subkeys.shape
    k = indices.shape[2]
    v = values.shape[1]
    shape = make_shape(B, d, H, 2 * half, n, k, v, x.dtype, bn_eps)
    if workspace is None:
        nb = int(lib().pkm_workspace_size(ctypes.byref(shape), 3))
        if nb == 0:
            raise PKMError("pkm_workspace_size", -1)
        workspace = torch.empty(nb, dtype=torch.uint8, device=x.device)
    g = grads
    fn = lib().pkm_backward_train if bn_training else lib().pkm_backward
    rc = fn(ctypes.byref(shape), _ptr(x), _ptr(W_q), _ptr(bn_mean), _ptr(bn_var),
            _ptr(bn_gamma), _ptr(bn_beta), _ptr(subkeys), _ptr(values), _ptr(indices),
            _ptr(weights), _ptr(grad_out), _ptr(g.get("x")), _ptr(g.get("W_q")),
            _ptr(g.get("bn_gamma")), _ptr(g.get("bn_beta")), _ptr(g.get("subkeys")),
            _ptr(g.get("values")), _ptr(g.get("scores")), _ptr(workspace), workspace.numel(),
            _stream(stream))
    if rc != PKM_OK:
        raise PKMError("pkm_backward_train" if bn_training else "pkm_backward", rc)
    return grads


def pkm_backward_values_noalloc(values: torch.Tensor, indices: torch.Tensor,
                                weights: torch.Tensor, grad_out: torch.Tensor,
                                grad_values: torch.Tensor, grad_scores: Optional[torch.Tensor],
                                n: int, stream=None):
    """pkm_backward_values with the library's fixed device scratch instead of a
    workspace (for callers that cannot allocate; limits in include/pkm.h)."""
    B, H, k = indices.shape
    v = values.shape[1]
    shape = make_shape(B, 0, H, 0, n, k, v, values.dtype)
    rc = lib().pkm_backward_values_noalloc(ctypes.byref(shape), _ptr(values), _ptr(indices),
                                           _ptr(weights), _ptr(grad_out), _ptr(grad_values),
                                           _ptr(grad_scores), _stream(stream))
    if rc != PKM_OK:
        raise PKMError("pkm_backward_values_noalloc", rc)
    return grad_values, grad_scores


def pkm_slot_usage(indices: torch.Tensor, n: int, hits: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Distinct slots among indices [B][H][k] (device int64 tensor of one element)."""
    B, H, k = indices.shape
    shape = make_shape(B, 0, H, 0, n, k, 8, PKM_F32)
    if hits is None:
        hits = torch.empty(1, dtype=torch.int64, device=indices.device)
    if workspace is None:
        nb = int(lib().pkm_workspace_size(ctypes.byref(shape), 2))
        if nb == 0:
            raise PKMError("pkm_workspace_size", -1)
        workspace = torch.empty(nb, dtype=torch.uint8, device=indices.device)
    rc = lib().pkm_slot_usage(ctypes.byref(shape), _ptr(indices), _ptr(hits), _ptr(workspace),
                              workspace.numel(), _stream(stream))
    if rc != PKM_OK:
        raise PKMError("pkm_slot_usage", rc)
    return hits


def pkm_device_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return (and clear) the workspace's device status."""
    return int(lib().pkm_device_status(_ptr(workspace), _stream(stream)))


def pkm_trace_enable(on: bool = True) -> None:
    """Record CUDA events at stage boundaries of every following call."""
    lib().pkm_trace_enable(int(bool(on)))


def pkm_trace_read(pass_: int = 0, max_stages: int = 4):
    """(per-stage milliseconds summed over traced calls, traced calls, kernel launches)
    for pass 0 (forward) or 1 (backward); waits for the events and resets."""
    ms = (ctypes.c_double * max_stages)()
    calls = ctypes.c_int64(0)
    launches = ctypes.c_int64(0)
    rc = lib().pkm_trace_read(int(pass_), ms, max_stages, ctypes.byref(calls),
                              ctypes.byref(launches))
    if rc != PKM_OK:
        raise PKMError("pkm_trace_read", rc)
    return list(ms), int(calls.value), int(launches.value)


# ---------------------------------------------------------------------------------------
# The transformer block around the layer. These calls check the tensors they are given
# (device, type, shape, contiguity: ValueError) and run on the device of their first
# tensor, whichever device is current. With a `stream` other than the current one the inputs have
# to be ready there and to live until it has read them, and results are ready on it.
# ---------------------------------------------------------------------------------------
_DTYPES = {torch.float32: PKM_F32, torch.bfloat16: PKM_BF16}


def _dtype(t) -> int:
    """pkm_dtype of a torch type (or a pkm_dtype itself)."""
    if isinstance(t, int):
        return t
    if t not in _DTYPES:
        raise ValueError("libpkm takes float32 and bfloat16, not %s" % t)
    return _DTYPES[t]


def _check(name: str, t: torch.Tensor, shape, dtype, device) -> None:
    """t is a contiguous device tensor of this shape, type (None: fp32 or bf16) and device."""
    kind = t.dtype
    if (t.shape == shape and (kind is dtype or (dtype is None and kind in _DTYPES)) and
            t.device == device and t.is_cuda and t.is_contiguous()):
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is None:
        _dtype(kind)
    elif kind != dtype:
        raise ValueError("%s: %s, expected %s" % (name, kind, dtype))
    if not t.is_cuda:
        raise ValueError("%s: libpkm takes device tensors" % name)
    if t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    raise ValueError("%s: libpkm takes contiguous tensors" % name)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda i: torch.cuda.current_stream(i).cuda_stream)


class _Call:
    """The device and stream of one call: makes `device` current while it lasts, and a `stream`
    that is not the current one too: what the call allocates then comes from that stream's
    memory, which no work queued elsewhere still uses."""
    __slots__ = ("device", "given", "handle", "guard", "caller")

    def __init__(self, device: torch.device, stream):
        if stream is not None and stream.device != device:
            raise ValueError("stream is on %s, not on %s" % (stream.device, device))
        self.device, self.given, self.guard, self.caller = device, stream, None, None

    def __enter__(self):
        index = self.device.index
        self.handle = _raw_stream(index)
        if self.given is not None and self.given.cuda_stream != self.handle:
            self.handle = self.given.cuda_stream
            self.caller = torch.cuda.current_stream(index)
            self.guard = torch.cuda.stream(self.given)
            self.guard.__enter__()
        elif _current_device() != index:
            self.guard = torch.cuda.device(index)
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def empty(self, like: torch.Tensor, shape, dtype, result: bool = True) -> torch.Tensor:
        """An uninitialised tensor beside `like` (the forms that cost the host least). A result is
        the caller's from then on: its memory waits for the work of the caller's stream when it
        is dropped."""
        if dtype is not like.dtype:
            t = like.new_empty(shape, dtype=dtype)
        elif shape == like.shape:
            t = torch.empty_like(like)
        else:
            t = like.new_empty(shape)
        if result and self.caller is not None:
            t.record_stream(self.caller)
        return t


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def make_norm_shape(rows, d, x_dtype=PKM_F32, add_dtype=PKM_F32, y_dtype=PKM_F32,
                    grad_dtype=PKM_F32, eps=1e-5) -> pkm_norm_shape:
    return pkm_norm_shape(int(rows), int(d), _dtype(x_dtype), _dtype(add_dtype), _dtype(y_dtype),
                          _dtype(grad_dtype), float(eps))


@functools.lru_cache(maxsize=1024)
def _norm_ref(*fields):
    """(make_norm_shape(*fields) by reference, workspace bytes): sizes and types only."""
    shape = make_norm_shape(*fields)
    ref = ctypes.byref(shape)
    return ref, int(lib().pkm_norm_workspace_size(ref))


def alloc_norm_workspace(shape: pkm_norm_shape, device=None) -> torch.Tensor:
    """Scratch of pkm_layernorm_backward for this many rows of this width."""
    n = int(lib().pkm_norm_workspace_size(ctypes.byref(shape)))
    if n == 0:
        raise PKMError("pkm_norm_workspace_size", -1)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def pkm_layernorm_forward(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor],
                          add: Optional[torch.Tensor] = None, eps: float = 1e-5,
                          out_dtype: Optional[torch.dtype] = None, want_stats: bool = True,
                          out: Optional[torch.Tensor] = None,
                          sum_out: Optional[torch.Tensor] = None, stream=None):
    """Layer norm of the rows of x + add: (y, h, mean, rstd).

    x [rows][d] and add [rows][d] are fp32 or bf16 each, gamma and beta [d] fp32 (beta may
    be None). h is x + add in x's type (x itself without add): the new residual stream. y has
    type out_dtype (x's by default). mean and rstd [rows] fp32 are what
    pkm_layernorm_backward takes; None unless want_stats. out and sum_out receive y and h
    and may be x or add themselves (in place) where the types are equal."""
    if x.dim() != 2:
        raise ValueError("x must be [rows][d]")
    rows, d = x.shape
    dev = x.device
    _check("x", x, (rows, d), None, dev)
    _check("gamma", gamma, (d,), torch.float32, dev)
    if beta is not None:
        _check("beta", beta, (d,), torch.float32, dev)
    if add is not None:
        _check("add", add, (rows, d), None, dev)
    elif sum_out is not None:
        raise ValueError("sum_out without add")
    if out is not None:
        _check("out", out, (rows, d), out_dtype, dev)
        out_dtype = out.dtype
    if sum_out is not None:
        _check("sum_out", sum_out, (rows, d), x.dtype, dev)
    out_dtype = out_dtype or x.dtype
    ref, _ = _norm_ref(rows, d, x.dtype, PKM_F32 if add is None else add.dtype, out_dtype, PKM_F32,
                       eps)
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty(x, (rows, d), out_dtype)
        if sum_out is None and add is not None:
            sum_out = c.empty(x, (rows, d), x.dtype)
        mean = c.empty(gamma, (rows,), torch.float32) if want_stats else None
        rstd = c.empty(gamma, (rows,), torch.float32) if want_stats else None
        rc = lib().pkm_layernorm_forward(ref, _addr(x), _addr(add), _addr(gamma),
                                         _addr(beta), _addr(out), _addr(sum_out), _addr(mean),
                                         _addr(rstd), c.handle)
    if rc != PKM_OK:
        raise PKMError("pkm_layernorm_forward", rc)
    return out, x if add is None else sum_out, mean, rstd


def pkm_layernorm_backward(grad_y: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                           rstd: torch.Tensor, gamma: torch.Tensor,
                           grad_sum: Optional[torch.Tensor] = None,
                           grad_dtype: Optional[torch.dtype] = None,
                           grad_x: Optional[torch.Tensor] = None,
                           grad_gamma: Optional[torch.Tensor] = None,
                           grad_beta: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward of pkm_layernorm_forward: (grad_x, grad_gamma, grad_beta).

    grad_y [rows][d] fp32 or bf16; x, mean, rstd: the forward's h, mean and rstd; grad_sum
    [rows][d] fp32 or bf16: the gradient that reaches h past the norm (added to grad_x).
    grad_x has type grad_dtype (grad_y's by default) and may be grad_y, grad_sum or x itself;
    grad_gamma and grad_beta [d] are fp32 and overwritten."""
    if x.dim() != 2:
        raise ValueError("x must be [rows][d]")
    rows, d = x.shape
    dev = x.device
    _check("x", x, (rows, d), None, dev)
    _check("grad_y", grad_y, (rows, d), None, dev)
    _check("mean", mean, (rows,), torch.float32, dev)
    _check("rstd", rstd, (rows,), torch.float32, dev)
    _check("gamma", gamma, (d,), torch.float32, dev)
    if grad_sum is not None:
        _check("grad_sum", grad_sum, (rows, d), None, dev)
    if grad_x is not None:
        _check("grad_x", grad_x, (rows, d), grad_dtype, dev)
        grad_dtype = grad_x.dtype
    grad_dtype = grad_dtype or grad_y.dtype
    for name, t in (("grad_gamma", grad_gamma), ("grad_beta", grad_beta)):
        if t is not None:
            _check(name, t, (d,), torch.float32, dev)
    ref, need = _norm_ref(rows, d, x.dtype, PKM_F32 if grad_sum is None else grad_sum.dtype,
                          grad_y.dtype, grad_dtype)
    with _Call(dev, stream) as c:
        if grad_x is None:
            grad_x = c.empty(x, (rows, d), grad_dtype)
        if grad_gamma is None:
            grad_gamma = c.empty(gamma, (d,), torch.float32)
        if grad_beta is None:
            grad_beta = c.empty(gamma, (d,), torch.float32)
        if workspace is None:
            workspace = c.empty(x, (max(need, 1),), torch.uint8, result=False)
        ws, nbytes = _given_workspace(c, workspace)
        rc = lib().pkm_layernorm_backward(ref, _addr(grad_y), _addr(x),
                                          _addr(mean), _addr(rstd), _addr(gamma), _addr(grad_sum),
                                          _addr(grad_x), _addr(grad_gamma), _addr(grad_beta),
                                          _addr(ws), nbytes, c.handle)
    if rc != PKM_OK:
        raise PKMError("pkm_layernorm_backward", rc)
    return grad_x, grad_gamma, grad_beta


ADAMW_BLOCK = 256      # elements that share a scale of 8-bit states


def alloc_adamw_state(param: torch.Tensor, bits: int = 32) -> dict:
    """The initial states of one parameter as the entries make_adamw_tensors takes: m and v in
    fp32, or (bits=8) as torch.float8_e4m3fn codes with m_scale and v_scale."""
    if bits not in (32, 8):
        raise ValueError("bits is 32 or 8")
    kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
    state = {k: torch.zeros(param.shape, dtype=kind, device=param.device) for k in ("m", "v")}
    if bits == 8:
        blocks = -(-param.numel() // ADAMW_BLOCK)
        for k in ("m_scale", "v_scale"):
            state[k] = torch.zeros(blocks, dtype=torch.float32, device=param.device)
    return state


class AdamWTensors:
    """The list pkm_adamw_step works through (make_adamw_tensors): holds its tensors."""

    def __init__(self, array, tensors, device):
        self.array, self.tensors, self.device = array, tensors, device

    def __len__(self):
        return len(self.array)


def make_adamw_tensors(tensors) -> AdamWTensors:
    """The list of an AdamW step, made once for tensors that stay where they are.

    Each entry is a dict: param (fp32 or bf16, updated in place), grad (fp32 or bf16 of its
    shape), m and v (fp32, or torch.float8_e4m3fn with m_scale and v_scale [ceil(n / 256)]
    fp32; v then holds the second moment's square root), optionally master (fp32, the copy
    of a bf16 param that carries it), weight_decay (0) and lr_scale (1). All tensors are
    contiguous, on one device and distinct."""
    array = (pkm_adamw_tensor * len(tensors))()
    device = tensors[0]["param"].device if len(tensors) else torch.device("cuda")
    kept, spans = [], []
    for i, t in enumerate(tensors):
        p = t["param"]
        n, where = p.numel(), "tensor %d: " % i
        _check(where + "param", p, p.shape, None, device)
        _check(where + "grad", t["grad"], p.shape, None, device)
        bits = 8 if t["m"].dtype == torch.float8_e4m3fn else 32
        kind = torch.float8_e4m3fn if bits == 8 else torch.float32
        for k in ("m", "v"):
            _check(where + k, t[k], p.shape, kind, device)
        for k in ("m_scale", "v_scale"):
            if (t.get(k) is not None) != (bits == 8):
                raise ValueError(where + "%s goes with 8-bit states" % k)
            if bits == 8:
                _check(where + k, t[k], (-(-n // ADAMW_BLOCK),), torch.float32, device)
        if t.get("master") is not None:
            if p.dtype != torch.bfloat16:
                raise ValueError(where + "master goes with a bf16 param")
            _check(where + "master", t["master"], p.shape, torch.float32, device)
        a = array[i]
        for k in ("param", "grad", "master", "m", "v", "m_scale", "v_scale"):
            x = t.get(k)
            if x is not None:
                setattr(a, k, x.data_ptr())
                kept.append(x)
                if x.numel():
                    spans.append((x.data_ptr(), x.data_ptr() + x.numel() * x.element_size(),
                                  where + k))
        a.n, a.param_dtype, a.grad_dtype = n, _dtype(p.dtype), _dtype(t["grad"].dtype)
        a.state_bits = bits
        a.weight_decay = float(t.get("weight_decay", 0.0))
        a.lr_scale = float(t.get("lr_scale", 1.0))
    spans.sort()
    for (_, end, first), (begin, _, second) in zip(spans, spans[1:]):
        if begin < end:
            raise ValueError("%s and %s overlap" % (first, second))
    return AdamWTensors(array, kept, device)


def pkm_adamw_step(tensors: AdamWTensors, lr: float, step: int, betas=(0.9, 0.999),
                   eps: float = 1e-8, grad_scale: float = 1.0, zero_grad: bool = False,
                   seed: int = 0, dyn: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW step over a list from make_adamw_tensors: parameters, masters and states are
    updated in place, gradients cleared with zero_grad. step counts from 1. dyn: three
    device fp32 [lr, step, grad_scale] that the step reads in the place of the arguments
    when it runs (for captured steps)."""
    if not isinstance(tensors, AdamWTensors):
        raise ValueError("pkm_adamw_step takes a list from make_adamw_tensors")
    if dyn is not None:
        _check("dyn", dyn, (3,), torch.float32, tensors.device)
    h = pkm_adamw_hyper(float(lr), float(betas[0]), float(betas[1]), float(eps),
                        float(grad_scale), int(step), int(seed) & 0xffffffff, int(bool(zero_grad)))
    if len(tensors):
        with _Call(tensors.device, stream) as c:
            rc = lib().pkm_adamw_step(tensors.array, len(tensors), ctypes.byref(h), _addr(dyn),
                                      c.handle)
    else:
        rc = lib().pkm_adamw_step(None, 0, ctypes.byref(h), None, None)
    if rc != PKM_OK:
        raise PKMError("pkm_adamw_step", rc)


def _activation(name) -> int:
    if isinstance(name, int):
        return name
    if name not in _ACTS:
        raise ValueError("activation is one of %s" % ", ".join(sorted(_ACTS)))
    return _ACTS[name]


def make_linear_shape(M, N, K, dtype, out_dtype=None, activation="none") -> pkm_linear_shape:
    """Sizes of a dense layer: x [M][K], W [N][K] of dtype, y (in the backward grad_x) of
    out_dtype (dtype by default)."""
    return pkm_linear_shape(int(M), int(N), int(K), _dtype(dtype),
                            _dtype(dtype if out_dtype is None else out_dtype),
                            _activation(activation))


def alloc_linear_workspace(shape: pkm_linear_shape, for_backward: bool = False,
                           device=None) -> torch.Tensor:
    n = int(lib().pkm_linear_workspace_size(ctypes.byref(shape), int(bool(for_backward))))
    if n == 0:
        raise PKMError("pkm_linear_workspace_size", -1)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _given_workspace(c: _Call, workspace: torch.Tensor):
    if not workspace.is_contiguous() or workspace.device != c.device:
        raise ValueError("workspace must be contiguous and on %s" % c.device)
    return workspace, workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=1024)
def _linear_ref(for_backward, *fields):
    """(make_linear_shape(*fields) by reference, workspace bytes): sizes and types only."""
    shape = make_linear_shape(*fields)
    ref = ctypes.byref(shape)
    return ref, int(lib().pkm_linear_workspace_size(ref, for_backward))


def _linear_workspace(c: _Call, x, workspace, need: int):
    """(workspace, bytes): the caller's, or one for this call."""
    if workspace is None:
        return c.empty(x, (max(need, 1),), torch.uint8, result=False), need
    return _given_workspace(c, workspace)


def _linear_operands(x: torch.Tensor, W: torch.Tensor):
    if x.dim() != 2 or W.dim() != 2:
        raise ValueError("x must be [M][K] and W [N][K]")
    (M, K), N, dev = x.shape, W.shape[0], x.device
    _check("x", x, (M, K), None, dev)
    _check("W", W, (N, K), x.dtype, dev)
    return M, N, K, dev


def pkm_linear_forward(x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
                       residual: Optional[torch.Tensor] = None, activation: str = "none",
                       out_dtype: Optional[torch.dtype] = None, want_pre: bool = False,
                       out: Optional[torch.Tensor] = None, pre: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """Dense layer: (y, pre) with pre = x W^T + bias and y = activation(pre) + residual.

    x [M][K] and W [N][K] both fp32 or both bf16, bias [N] fp32, activation "none", "relu",
    "gelu" (exact) or "silu". y and residual [M][N] have type out_dtype (x's by default);
    residual may be out itself. pre [M][N] of x's type is what pkm_linear_backward takes
    (None unless given or want_pre)."""
    M, N, K, dev = _linear_operands(x, W)
    act = _activation(activation)
    if bias is not None:
        _check("bias", bias, (N,), torch.float32, dev)
    if out is not None:
        _check("out", out, (M, N), out_dtype, dev)
        out_dtype = out.dtype
    if residual is not None:
        _check("residual", residual, (M, N), out_dtype, dev)
        out_dtype = residual.dtype
    out_dtype = out_dtype or x.dtype
    if pre is not None:
        _check("pre", pre, (M, N), x.dtype, dev)
    ref, need = _linear_ref(0, M, N, K, x.dtype, out_dtype, act)
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty(x, (M, N), out_dtype)
        if pre is None and want_pre:
            pre = c.empty(x, (M, N), x.dtype)
        ws, nbytes = _linear_workspace(c, x, workspace, need)
        rc = lib().pkm_linear_forward(ref, _addr(x), _addr(W), _addr(bias),
                                      _addr(residual), _addr(out), _addr(pre),
                                      _addr(ws), nbytes, c.handle)
    if rc != PKM_OK:
        raise PKMError("pkm_linear_forward", rc)
    return out, pre


def pkm_linear_backward(x: torch.Tensor, W: torch.Tensor, grad_y: torch.Tensor, grads: dict,
                        pre: Optional[torch.Tensor] = None, activation: str = "none",
                        workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Backward of pkm_linear_forward.

    ``grads`` maps any of x [M][K] (fp32 or bf16), W [N][K] fp32 and bias [N] fp32 to device
    tensors, overwritten; missing entries are not computed. grad_y [M][N] has x's type, and
    so has pre, the forward's (needed with an activation). The residual's gradient is grad_y."""
    M, N, K, dev = _linear_operands(x, W)
    act = _activation(activation)
    _check("grad_y", grad_y, (M, N), x.dtype, dev)
    if pre is not None:
        _check("pre", pre, (M, N), x.dtype, dev)
    unknown = set(grads) - {"x", "W", "bias"}
    if unknown:
        raise ValueError("grads takes x, W and bias, not %s" % ", ".join(sorted(unknown)))
    gx, gW, gb = (grads.get(k) for k in ("x", "W", "bias"))
    if gx is not None:
        _check("grads['x']", gx, (M, K), None, dev)
    if gW is not None:
        _check("grads['W']", gW, (N, K), torch.float32, dev)
    if gb is not None:
        _check("grads['bias']", gb, (N,), torch.float32, dev)
    ref, need = _linear_ref(1, M, N, K, x.dtype, x.dtype if gx is None else gx.dtype, act)
    with _Call(dev, stream) as c:
        ws, nbytes = _linear_workspace(c, x, workspace, need)
        rc = lib().pkm_linear_backward(ref, _addr(x), _addr(W), _addr(grad_y),
                                       _addr(pre), _addr(gx), _addr(gW), _addr(gb),
                                       _addr(ws), nbytes, c.handle)
    if rc != PKM_OK:
        raise PKMError("pkm_linear_backward", rc)
    return grads
