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


def _adamw(t=None, h=None, count=1, dyn=None, tensors=True):
    a = P.pkm_adamw_tensor(param=OK.value, grad=OK.value, m=OK.value, v=OK.value, n=100,
                           param_dtype=0, grad_dtype=0, state_bits=32, weight_decay=0.1,
                           lr_scale=1.0)
    for k, x in (t or {}).items():
        setattr(a, k, x)
    b = P.pkm_adamw_hyper(lr=1e-3, beta1=0.9, beta2=0.98, eps=1e-8, grad_scale=1.0, step=1)
    for k, x in (h or {}).items():
        setattr(b, k, x)
    return P.lib().pkm_adamw_step(ctypes.byref(a) if tensors else None, count, ctypes.byref(b), dyn,
                                  None)


@pytest.mark.parametrize("t,code", [
    (dict(param=None), -1), (dict(grad=None), -1), (dict(m=None), -1), (dict(v=None), -1),
    (dict(n=-1), -1), (dict(n=1 << 38), -2), (dict(param_dtype=2), -1), (dict(grad_dtype=-1), -1),
    (dict(state_bits=16), -1), (dict(state_bits=8), -1),
    (dict(state_bits=8, m_scale=OK.value), -1), (dict(m_scale=OK.value), -1),
    (dict(master=OK.value), -1), (dict(weight_decay=-0.1), -1),
    (dict(weight_decay=math.nan), -1), (dict(lr_scale=-1.0), -1), (dict(lr_scale=math.inf), -1),
    (dict(param=ODD.value), -2), (dict(grad=ODD.value), -2), (dict(m=ODD.value), -2),
    (dict(v=ODD.value), -2),
    (dict(state_bits=8, m_scale=ODD.value, v_scale=OK.value), -2),
    (dict(param_dtype=1, master=ODD.value), -2)])
def test_adamw_tensor_refused(t, code):
    assert _adamw(t) == code


@pytest.mark.parametrize("h", [
    dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
    dict(beta2=1.0), dict(beta2=math.nan), dict(eps=0.0), dict(eps=math.nan), dict(eps=-1.0),
    dict(grad_scale=math.inf), dict(grad_scale=math.nan), dict(step=0), dict(step=-3),
    dict(zero_grad=2)])
def test_adamw_hyper_refused(h):
    assert _adamw(h=h) == -1


def test_adamw_call_refused():
    assert _adamw(count=-1) == -1 and _adamw(tensors=False) == -1
    assert _adamw(dyn=ctypes.c_void_p((1 << 20) + 2)) == -2
    assert P.lib().pkm_adamw_step(None, 0, None, None, None) == -1
    assert _adamw(count=0, tensors=False) == 0            # an empty list
    assert _adamw(dict(n=0, param=None)) == 0             # an empty tensor


def test_adamw_binding_checks_tensors():
    x = torch.zeros(8)
    with pytest.raises(ValueError):
        P.make_adamw_tensors([dict(param=x, grad=x, m=x, v=x)])       # host tensors
    with pytest.raises(ValueError):
        P.pkm_adamw_step([dict(param=x)], lr=1e-3, step=1)
    with pytest.raises(ValueError):
        P.alloc_adamw_state(x, 16)
    s = P.alloc_adamw_state(torch.zeros(300), 8)
    assert s["m"].dtype == torch.float8_e4m3fn and s["v_scale"].shape == (2,)


def _linear(**kw):
    base = dict(M=100, N=72, K=80, dtype=1, out_dtype=1, activation=0)
    base.update(kw)
    return P.pkm_linear_shape(**base)


def _linear_forward(s, ws=OK, nbytes=1 << 60, **kw):
    a = dict(x=OK, W=OK, bias=None, residual=None, y=OK, pre=None)
    a.update(kw)
    return P.lib().pkm_linear_forward(ctypes.byref(s) if s else None, *a.values(), ws, nbytes, None)


def _linear_backward(s, ws=OK, nbytes=1 << 60, **kw):
    a = dict(x=OK, W=OK, gy=OK, pre=None, gx=OK, gW=OK, gb=OK)
    a.update(kw)
    return P.lib().pkm_linear_backward(ctypes.byref(s) if s else None, *a.values(), ws, nbytes,
                                       None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(K=-8), -1), (dict(dtype=2), -1),
    (dict(out_dtype=-1), -1), (dict(activation=4), -1), (dict(activation=-1), -1),
    (dict(M=(1 << 31) - 1), -2), (dict(N=(1 << 20) + 1), -2), (dict(K=(1 << 20) + 1), -2),
    (dict(M=1 << 20, N=1 << 18), -2), (dict(M=1 << 20, K=1 << 18), -2)])
def test_linear_sizes_refused(kw, code):
    s = _linear(**kw)
    assert P.lib().pkm_linear_workspace_size(ctypes.byref(s), 0) == 0
    assert P.lib().pkm_linear_workspace_size(ctypes.byref(s), 1) == 0
    assert _linear_forward(s) == code and _linear_backward(s, pre=OK) == code


@pytest.mark.parametrize("dtype", [0, 1])
def test_linear_arguments_refused(dtype):
    s = _linear(dtype=dtype)
    assert _linear_forward(None) == -1 and _linear_backward(None) == -1
    for name in ("x", "W", "y"):
        assert _linear_forward(s, **{name: None}) == -1, name
    for name in ("x", "W", "gy"):
        assert _linear_backward(s, **{name: None}) == -1, name
    assert _linear_backward(_linear(dtype=dtype, activation=2)) == -1       # pre is missing
    for name in ("x", "W", "bias", "residual", "y", "pre"):
        assert _linear_forward(s, **{name: ODD}) == -2, name
    for name in ("x", "W", "gy", "pre", "gx", "gW", "gb"):
        assert _linear_backward(s, **{name: ODD}) == -2, name
    for back, call in ((0, _linear_forward), (1, _linear_backward)):
        need = int(P.lib().pkm_linear_workspace_size(ctypes.byref(s), back))
        assert need >= 256
        assert call(s, nbytes=need - 1) == -3 and call(s, ws=None) == -3
        assert call(s, ws=ctypes.c_void_p((1 << 20) + 128)) == -3


def test_linear_no_rows_returns_without_a_gpu():
    s = _linear(M=0, activation=2)
    for back in (0, 1):
        assert P.lib().pkm_linear_workspace_size(ctypes.byref(s), back) == 256
    assert _linear_forward(s, x=None, y=None) == 0
    assert _linear_backward(s, x=None, gy=None, gx=None, gW=None, gb=None) == 0


def test_linear_workspace_holds_the_planes():
    """fp32 operands: three bf16 planes each, rows padded to 8; bf16 rows of 16-byte multiples are
    used in place."""
    def size(back, **kw):
        return int(P.lib().pkm_linear_workspace_size(ctypes.byref(_linear(**kw)), back))
    even = dict(M=9472, N=512)            # 74 tiles of 256 x 256: one for each pair of CTAs
    assert size(0, K=1024, **even) == 256
    assert size(0, dtype=0, K=1024, **even) == 256 + 3 * 2 * (9472 + 512) * 1024
    assert size(0, K=1001, **even) == 256 + 2 * (9472 + 512) * 1008
    assert size(1, activation=2, K=1024, **even) >= 2 * 2 * 9472 * 512
    # few tiles: cut along K, two fp32 parts of 256 x 256 for each pair that has a range
    cut = size(0, M=256, N=256, K=6400) - 256
    assert cut and cut % (2 * 256 * 256 * 4) == 0 and cut <= 74 * 2 * 256 * 256 * 4


def test_linear_binding_checks_tensors():
    x, W = torch.zeros(4, 8), torch.zeros(3, 8)
    for call in (lambda: P.pkm_linear_forward(x, W), lambda: P.pkm_linear_forward(x, W[0]),
                 lambda: P.pkm_linear_forward(x, W, activation="tanh"),
                 lambda: P.pkm_linear_backward(x, W, torch.zeros(4, 3), {}),
                 lambda: P.make_linear_shape(4, 3, 8, torch.float16)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(P.PKMError):
        P.alloc_linear_workspace(P.make_linear_shape(4, 0, 8, torch.bfloat16))


def _at(*places):
    """Aligned addresses, `places` in units of 64 KiB (more than any array below)."""
    return [ctypes.c_void_p((1 << 24) + (p << 16)) for p in places]


@pytest.mark.parametrize("a,b,code", [
    ("y", "gamma", -1), ("y", "beta", -1), ("y", "sum", -1), ("y", "mean", -1), ("y", "rstd", -1),
    ("sum", "gamma", -1), ("sum", "rstd", -1), ("mean", "rstd", -1), ("mean", "x", -1),
    ("rstd", "add", -1), ("mean", "gamma", -1), ("rstd", "beta", -1)])
def test_norm_forward_overlaps_refused(a, b, code):
    names = ("x", "add", "gamma", "beta", "y", "sum", "mean", "rstd")
    arrays = dict(zip(names, _at(*range(8))))
    arrays[a] = ctypes.c_void_p(arrays[b].value)
    assert _forward(_norm(), **arrays) == code


def test_norm_in_place_needs_the_same_array_and_type():
    names = ("x", "add", "gamma", "beta", "y", "sum", "mean", "rstd")
    for out, t in (("y", dict(y_dtype=1)), ("sum", dict(add_dtype=1))):
        for given in ("x", "add"):
            arrays = dict(zip(names, _at(*range(8))))
            arrays[out] = ctypes.c_void_p(arrays[given].value + 64 * 4)      # a row further
            assert _forward(_norm(), **arrays) == -1, (out, given)
            arrays[out] = ctypes.c_void_p(arrays[given].value)
            if (out, given) != ("sum", "x"):                                  # always of one type
                assert _forward(_norm(**t), **arrays) == -1, (out, given)
    names = ("gy", "x", "mean", "rstd", "gamma", "gsum", "gx", "gg", "gb")
    for given in ("gy", "x", "gsum"):
        arrays = dict(zip(names, _at(*range(9))))
        arrays["gx"] = ctypes.c_void_p(arrays[given].value + 64 * 4)
        assert _backward(_norm(), ws=_at(20)[0], **arrays) == -1, given
        arrays["gx"] = ctypes.c_void_p(arrays[given].value)
        assert _backward(_norm(grad_dtype=1), ws=_at(20)[0], **arrays) == -1, given


@pytest.mark.parametrize("a,b", [
    ("gx", "mean"), ("gx", "rstd"), ("gx", "gamma"), ("gx", "gg"), ("gx", "gb"), ("gg", "gb"),
    ("gg", "gy"), ("gb", "x"), ("gg", "gsum"), ("gg", "gamma"), ("gb", "mean")])
def test_norm_backward_overlaps_refused(a, b):
    names = ("gy", "x", "mean", "rstd", "gamma", "gsum", "gx", "gg", "gb")
    arrays = dict(zip(names, _at(*range(9))))
    arrays[a] = ctypes.c_void_p(arrays[b].value)
    assert _backward(_norm(), ws=_at(20)[0], **arrays) == -1
    for name in names:
        arrays = dict(zip(names, _at(*range(9))))
        assert _backward(_norm(), ws=arrays[name], **arrays) == -1, name


@pytest.mark.parametrize("M", [3, 100])
@pytest.mark.parametrize("dtype", [0, 1])
def test_linear_overlaps_refused(M, dtype):
    s = _linear(M=M, N=80, K=80, dtype=dtype, out_dtype=dtype, activation=2)
    names = ("x", "W", "bias", "residual", "y", "pre")
    for a, b in (("y", "x"), ("y", "W"), ("y", "bias"), ("y", "pre"), ("pre", "x"), ("pre", "W"),
                 ("pre", "bias"), ("pre", "residual")):
        arrays = dict(zip(names, _at(*range(6))))
        arrays[a] = ctypes.c_void_p(arrays[b].value)
        assert _linear_forward(s, ws=_at(20)[0], **arrays) == -1, (a, b)
    arrays = dict(zip(names, _at(*range(6))))
    arrays["y"] = ctypes.c_void_p(arrays["residual"].value + 16)          # partly
    assert _linear_forward(s, ws=_at(20)[0], **arrays) == -1
    for name in names:
        arrays = dict(zip(names, _at(*range(6))))
        assert _linear_forward(s, ws=arrays[name], **arrays) == -1, name
    names = ("x", "W", "gy", "pre", "gx", "gW", "gb")
    for a in ("gx", "gW", "gb"):
        for b in names:
            if a == b:
                continue
            arrays = dict(zip(names, _at(*range(7))))
            arrays[a] = ctypes.c_void_p(arrays[b].value)
            assert _linear_backward(s, ws=_at(200)[0], **arrays) == -1, (a, b)
    for name in names:
        arrays = dict(zip(names, _at(*range(7))))
        assert _linear_backward(s, ws=arrays[name], **arrays) == -1, name


@pytest.mark.parametrize("d", [8, 40, 64, 65, 1024, 2001])
def test_norm_workspace_serves_fewer_rows(d):
    sizes = [int(P.lib().pkm_norm_workspace_size(ctypes.byref(_norm(rows=r, d=d))))
             for r in list(range(3000)) + [20000, 1 << 30]]
    assert sizes == sorted(sizes)
