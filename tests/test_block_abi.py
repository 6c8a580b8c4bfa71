"""Host-side checks of the transformer-block entry points: sizes and refusals, before any CUDA call
(these run without a GPU)."""
import ctypes
import math

import pytest
import torch

import product_key_memory_b200 as P

OK = ctypes.c_void_p(1 << 20)          # looks like an aligned device address
ODD = ctypes.c_void_p((1 << 20) + 8)


def _norm(**kw):
    base = dict(rows=5, d=64)
    base.update(kw)
    return P.make_norm_shape(**base)


def _forward(s, **kw):
    a = dict(x=OK, add=None, gamma=OK, beta=OK, y=OK, sum=None, mean=OK, rstd=OK)
    a.update(kw)
    return P.lib().pkm_layernorm_forward(ctypes.byref(s) if s else None, *a.values(), None)


def _backward(s, ws=OK, nbytes=1 << 40, **kw):
    a = dict(gy=OK, x=OK, mean=OK, rstd=OK, gamma=OK, gsum=None, gx=OK, gg=OK, gb=OK)
    a.update(kw)
    return P.lib().pkm_layernorm_backward(ctypes.byref(s) if s else None, *a.values(), ws, nbytes,
                                          None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(d=0), -1), (dict(d=-8), -1), (dict(d=16385), -2),
    (dict(rows=1 << 31), -2), (dict(x_dtype=2), -1), (dict(y_dtype=-1), -1)])
def test_norm_sizes_refused(kw, code):
    s = _norm(**kw)
    assert _forward(s) == code and _backward(s) == code
    if "x_dtype" not in kw and "y_dtype" not in kw:
        assert P.lib().pkm_norm_workspace_size(ctypes.byref(s)) == 0


def test_norm_arguments_refused():
    s = _norm()
    assert _forward(None) == -1 and _backward(None) == -1
    for name in ("x", "gamma", "y"):
        assert _forward(s, **{name: None}) == -1, name
    assert _forward(s, add=OK) == -1 and _forward(s, sum=OK) == -1      # both or neither
    for eps in (-1e-5, math.nan, math.inf):
        assert _forward(_norm(eps=eps)) == -1
    assert _forward(_norm(add_dtype=5), add=OK, sum=OK) == -1
    for name in ("gy", "x", "mean", "rstd", "gamma", "gx"):
        assert _backward(s, **{name: None}) == -1, name
    assert _backward(_norm(grad_dtype=3)) == -1
    for name in ("x", "gamma", "beta", "y", "mean", "rstd"):
        assert _forward(s, **{name: ODD}) == -2, name
    for name in ("gy", "x", "mean", "rstd", "gamma", "gsum", "gx", "gg", "gb"):
        assert _backward(s, **{name: ODD}) == -2, name
    need = int(P.lib().pkm_norm_workspace_size(ctypes.byref(s)))
    assert need >= 2 * 64 * 4
    assert _backward(s, nbytes=need - 1) == -3 and _backward(s, ws=None) == -3
    assert _backward(s, ws=ctypes.c_void_p((1 << 20) + 128)) == -3


def test_norm_no_rows_returns_without_a_gpu():
    s = _norm(rows=0)
    assert _forward(s, x=None, y=None, mean=None, rstd=None) == 0
    assert _backward(s, gy=None, x=None, mean=None, rstd=None, gx=None, gg=None, gb=None) == 0


def test_norm_binding_checks_tensors():
    x, v = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError):
        P.pkm_layernorm_forward(x, v, v)                      # host tensors
    with pytest.raises(ValueError):
        P.pkm_layernorm_forward(torch.zeros(4, 2, 4), v, v)
    with pytest.raises(ValueError):
        P.make_norm_shape(4, 8, torch.float16)
    with pytest.raises(P.PKMError):
        P.alloc_norm_workspace(P.make_norm_shape(4, 0))
