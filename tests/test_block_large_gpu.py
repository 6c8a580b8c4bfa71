"""The transformer-block operators on arrays of more than 2^31 elements: the first, middle and last rows
against 64 bits, with the bounds of the operators' own tests."""
import pytest
import torch

from block_ref import BF16, F32, U, adamw, assert_within, half_step, layernorm_backward
from test_layernorm_gpu import K as KU, _check_forward as check_norm
from test_linear_gpu import _product_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _room():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _some(rows):
    return torch.tensor([0, 1, rows // 2, rows - 3, rows - 2, rows - 1], device="cuda")


@pytest.mark.parametrize("d", [1032, 1031])
def test_norm(d):
    import product_key_memory_b200 as P
    rows = (1 << 31) // d + 1005
    x = torch.empty(rows, d, device="cuda", dtype=BF16).normal_()
    gamma, beta = torch.rand(d, device="cuda") + 0.5, torch.rand(d, device="cuda")
    y, _, mean, rstd = P.pkm_layernorm_forward(x, gamma, beta)
    i = _some(rows)
    check_norm(x[i], None, gamma, beta, 1e-5, (y[i], x[i], mean[i], rstd[i]))
    gy = y.normal_()
    gx, _, gb = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma)
    want, _, _ = layernorm_backward(gy[i], x[i], mean[i], rstd[i], gamma, None)
    xhat = (x[i].double() - mean[i].double()[:, None]) * rstd[i].double()[:, None]
    t = gy[i].double() * gamma.double()
    size = t.abs() + t.abs().mean(1, keepdim=True) + xhat.abs() * (t * xhat).abs().mean(1, keepdim=True)
    bound = KU * U * rstd[i].double()[:, None] * size
    assert_within("grad_x", gx[i], want, bound + half_step(BF16) * (want.abs() + bound))
    parts = gy.split(1 << 17)
    assert_within("grad_beta", gb, sum(p.double().sum(0) for p in parts),
                  (KU + rows) * U * sum(p.double().abs().sum(0) for p in parts))


@pytest.mark.parametrize("kind,K", [(BF16, 8), (F32, 9)])
def test_dense(kind, K):
    import product_key_memory_b200 as P
    N = 1030
    M = (1 << 31) // N + 777
    x = torch.empty(M, K, device="cuda").normal_().to(kind)
    W = torch.randn(N, K, device="cuda").to(kind)
    y, _ = P.pkm_linear_forward(x, W, out_dtype=BF16)
    i = _some(M)

    def check(name, got, a, b, terms):
        want = a.double() @ b.double()
        bound = _product_bound(a.double().abs() @ b.double().abs(), terms, 6, 2.0 ** -22)
        assert_within(name, got, want, bound + half_step(got.dtype) * (want.abs() + bound))
    check("y", y[i], x[i], W.t(), K)
    if kind == F32:
        return
    gy = y.normal_()
    g = dict(x=torch.empty(M, K, device="cuda"), W=torch.empty(N, K, device="cuda"))
    P.pkm_linear_backward(x, W, gy, g)
    check("grad_x", g["x"][i], gy[i], W, N)
    want = sum(a.double().t() @ b.double() for a, b in zip(gy.split(1 << 17), x.split(1 << 17)))
    # M = 2^21 terms, taken out every 256 of them: 2^13 roundings, 2^13 2^-24 of the sum's size at most
    size = sum(a.double().abs().t() @ b.double().abs() for a, b in zip(gy.split(1 << 17), x.split(1 << 17)))
    assert_within("grad_W", g["W"], want, 2.0 ** -10 * size)


def test_adamw():
    import product_key_memory_b200 as P
    n = (1 << 31) + 2077
    p = torch.empty(n, device="cuda", dtype=BF16).normal_()
    g = torch.empty(n, device="cuda", dtype=BF16).normal_()
    t = dict(param=p, grad=g, **P.alloc_adamw_state(p, 32))
    hyper = dict(lr=1e-3, step=1, betas=(0.9, 0.98), eps=1e-8, grad_scale=0.5, seed=0)
    spans = [(0, 5000), (n // 2, n // 2 + 5000), (n - 5000, n)]
    before = [{k: t[k][a:b].clone() for k in ("param", "grad", "m", "v")} for a, b in spans]
    P.pkm_adamw_step(P.make_adamw_tensors([t]), **hyper)
    for (a, b), old in zip(spans, before):
        want = adamw(old, hyper, 0)
        assert torch.equal(t["m"][a:b], want["m"]) and torch.equal(t["v"][a:b], want["v"])
        e = want["bound"]
        assert_within("param", p[a:b], want["param"], e + half_step(BF16) * (want["param"].abs() + e))
