"""Layer norm and its backward on the GPU against a plain 64-bit implementation, element by
element, with bounds counted in roundings.

Forward. The row's sum is made of per-thread chains of at most 64 additions and a tree
or a chain over at most 16 warps: at most 64 + 5 + 16 roundings, each of at most U = 2^-24 of
the partial sums' magnitude, so the mean is off by at most 85 U mean|h|; the centred value
adds one rounding, the variance as many as the mean, halved by the square root; rstd,
its product, gamma and beta one rounding each. Together, with K = 200 for all chains,
  |err| <= K U (mean|h| rstd |gamma| + |y - beta|) + U |beta| + (half a step of y's type) |y|.
Backward, the same chains for the two row sums, and 85 + rows for a column sum:
  |err grad_x| <= K U rstd (|t| + mean|t| + |xhat| mean|t xhat|) + U |grad_sum| + half step,
  |err grad_gamma| <= (K + rows) U sum |grad_y| (|x| + |mean|) rstd
(xhat = (x - mean) rstd carries a rounding of x - mean relative to that difference and of
the product), grad_beta alike with sum |grad_y|.
"""
import pytest
import torch

from block_ref import (BF16, F32, U, assert_within, guarded, half_step, layernorm,
                       layernorm_backward)

pytestmark = pytest.mark.gpu
K = 200.0


def _data(rows, d, xt, at, seed=0, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (rn(rows, d) * scale + 0.3).to(xt)
    add = None if at is None else (rn(rows, d) * 0.5).to(at)
    return x, add, 1 + 0.2 * rn(d), 0.2 * rn(d), rn


def _check_forward(x, add, gamma, beta, eps, got):
    y, h, mean, rstd = got
    rh, rm, rr, ry = layernorm(x, add, gamma, beta, eps)
    assert torch.equal(h, rh)
    hd = rh.double()
    level = hd.abs().mean(1, keepdim=True)
    flat = ry if beta is None else ry - beta.double()
    bound = K * U * (level * rr[:, None] * gamma.double().abs() + flat.abs())
    if beta is not None:
        bound = bound + U * beta.double().abs()
    assert_within("y", y, ry, bound + half_step(y.dtype) * (ry.abs() + bound))
    if mean is not None:
        assert_within("mean", mean, rm, K * U * level[:, 0])
        # var is off by K U (var + level sqrt(var)): half of that, relative, in rstd
        var = (hd - rm[:, None]).square().mean(1)
        rel = K * U * (1 + level[:, 0] * var.sqrt() / (var + eps))
        assert_within("rstd", rstd, rr, rel * rr)


WIDTHS = [1, 2, 7, 8, 24, 64, 65, 72, 255, 256, 264, 512, 777, 1000, 1001, 1024, 1600, 2048, 2056,
          4096, 4097, 4104, 8192, 16377, 16384]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5, 700])
def test_forward_widths(rows, d):
    import product_key_memory_b200 as P
    types = [(F32, BF16, BF16), (BF16, F32, BF16), (BF16, None, F32), (F32, F32, F32),
             (F32, None, BF16), (BF16, BF16, F32)]
    xt, at, yt = types[(d + rows) % len(types)]
    x, add, gamma, beta, _ = _data(rows, d, xt, at, seed=d)
    out, check_out = guarded((rows, d), yt)
    h, check_sum = guarded((rows, d), xt)
    got = P.pkm_layernorm_forward(x, gamma, beta, add=add, out=out,
                                  sum_out=None if add is None else h)
    _check_forward(x, add, gamma, beta, 1e-5, got)
    check_out()
    check_sum()


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("at", [None, F32, BF16])
@pytest.mark.parametrize("yt", [F32, BF16])
def test_forward_types(xt, at, yt):
    import product_key_memory_b200 as P
    for rows, d in ((3, 200), (1300, 96), (40, 333)):
        x, add, gamma, beta, _ = _data(rows, d, xt, at, seed=rows)
        got = P.pkm_layernorm_forward(x, gamma, beta, add=add, out_dtype=yt, want_stats=rows != 3)
        assert got[0].dtype == yt and got[1].dtype == xt and (got[2] is None) == (rows == 3)
        _check_forward(x, add, gamma, beta, 1e-5, got)


def test_forward_no_bias_large_offset_constant_and_eps():
    import product_key_memory_b200 as P
    x, add, gamma, beta, _ = _data(65, 1024, F32, None)
    _check_forward(x, None, gamma, None, 1e-5, P.pkm_layernorm_forward(x, gamma, None))
    x = x + 1000.0                        # the mean is a thousand times the deviation
    _check_forward(x, None, gamma, beta, 1e-5, P.pkm_layernorm_forward(x, gamma, beta))
    x = torch.full((4, 1024), 0.5, device="cuda")
    y, _, mean, rstd = P.pkm_layernorm_forward(x, gamma, beta, eps=1e-2)
    assert torch.equal(y, beta.expand_as(y)) and bool((mean == 0.5).all())
    assert_within("rstd", rstd, torch.full((4,), 10.0, device="cuda").double(),
                  torch.full((4,), 10 * 4 * U, device="cuda").double())


def test_forward_in_place():
    import product_key_memory_b200 as P
    x, add, gamma, beta, _ = _data(300, 1000, BF16, BF16)
    want = P.pkm_layernorm_forward(x, gamma, beta, add=add)
    xs, ad = x.clone(), add.clone()
    y, h, _, _ = P.pkm_layernorm_forward(xs, gamma, beta, add=ad, out=ad, sum_out=xs)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    assert y.data_ptr() == ad.data_ptr() and h.data_ptr() == xs.data_ptr()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_non_finite_row_stays_its_own(value):
    import product_key_memory_b200 as P
    for rows, d in ((40, 64), (40, 1001), (2000, 512), (7, 4096)):
        x, _, gamma, beta, rn = _data(rows, d, F32, None)
        want = P.pkm_layernorm_forward(x, gamma, beta)
        x[3, d // 2] = value
        got = P.pkm_layernorm_forward(x, gamma, beta)
        keep = torch.arange(rows, device="cuda") != 3
        assert torch.equal(got[0][keep], want[0][keep]) and bool(got[0][3].isnan().all())
        gy = rn(rows, d)
        gx, _, gb = P.pkm_layernorm_backward(gy, x, got[2], got[3], gamma)
        assert bool(gx[3].isnan().all()) and bool(gx[keep].isfinite().all())
        assert bool(gb.isfinite().all())


def _check_backward(gy, x, mean, rstd, gamma, gsum, got):
    gx, gg, gb = got
    rx, rg, rb = layernorm_backward(gy, x, mean, rstd, gamma, gsum)
    rows = x.shape[0]
    xd, md, rd, gd = x.double(), mean.double()[:, None], rstd.double()[:, None], gy.double()
    xhat, t = (xd - md) * rd, gd * gamma.double()
    size = t.abs() + t.abs().mean(1, keepdim=True)
    size = size + xhat.abs() * (t * xhat).abs().mean(1, keepdim=True)
    bound = K * U * rd * size
    if gsum is not None:
        bound = bound + U * gsum.double().abs()
    assert_within("grad_x", gx, rx, bound + half_step(gx.dtype) * (rx.abs() + bound))
    assert_within("grad_gamma", gg, rg,
                  (K + rows) * U * (gd.abs() * (xd.abs() + md.abs()) * rd).sum(0))
    assert_within("grad_beta", gb, rb, (K + rows) * U * gd.abs().sum(0))


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5, 700])
def test_backward_widths(rows, d):
    import product_key_memory_b200 as P
    types = [(F32, F32, None, BF16), (BF16, F32, BF16, BF16), (F32, BF16, F32, F32),
             (BF16, BF16, None, BF16), (F32, F32, F32, F32)]
    xt, gt, st, ot = types[(d + rows) % len(types)]
    x, gsum, gamma, beta, rn = _data(rows, d, xt, st, seed=d + 1)
    gy = rn(rows, d).to(gt)
    _, _, mean, rstd = P.pkm_layernorm_forward(x, gamma, beta)
    gx, check_x = guarded((rows, d), ot)
    gg, check_g = guarded((d,), F32)
    gb, check_b = guarded((d,), F32)
    got = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma, grad_sum=gsum, grad_x=gx,
                                   grad_gamma=gg, grad_beta=gb)
    _check_backward(gy, x, mean, rstd, gamma, gsum, got)
    check_x()
    check_g()
    check_b()


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("st", [None, F32, BF16])
@pytest.mark.parametrize("ot", [F32, BF16])
def test_backward_types(xt, gt, st, ot):
    import product_key_memory_b200 as P
    for rows, d in ((3000, 40), (50, 800), (40, 333)):
        x, gsum, gamma, beta, rn = _data(rows, d, xt, st, seed=rows)
        gy = rn(rows, d).to(gt)
        _, _, mean, rstd = P.pkm_layernorm_forward(x, gamma, beta)
        got = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma, grad_sum=gsum, grad_dtype=ot)
        assert got[0].dtype == ot
        _check_backward(gy, x, mean, rstd, gamma, gsum, got)
        again = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma, grad_sum=gsum, grad_dtype=ot)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_backward_in_place_and_dirty_workspace():
    import product_key_memory_b200 as P
    x, gsum, gamma, beta, rn = _data(300, 1000, BF16, F32)
    gy = rn(300, 1000)
    _, _, mean, rstd = P.pkm_layernorm_forward(x, gamma, beta)
    want = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma, grad_sum=gsum)
    ws = P.alloc_norm_workspace(P.make_norm_shape(300, 1000), "cuda")
    ws.fill_(255)
    for target in ("gy", "gsum"):
        a, b = gy.clone(), gsum.clone()
        got = P.pkm_layernorm_backward(a, x, mean, rstd, gamma, grad_sum=b, workspace=ws,
                                       grad_x=a if target == "gy" else b)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_backward_against_differences():
    """A central difference of sum(y * gy) along a random direction, in 64 bits through the
    plain forward, against <grad, direction> of the kernel's gradients."""
    import product_key_memory_b200 as P
    x, _, gamma, beta, rn = _data(6, 130, F32, None)
    gy = rn(6, 130)
    _, _, mean, rstd = P.pkm_layernorm_forward(x, gamma, beta)
    gx, gg, gb = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma)
    dx, dg, db = rn(6, 130).double(), rn(130).double(), rn(130).double()

    def loss(e):
        h = x.double() + e * dx
        c = h - h.mean(1, keepdim=True)
        y = c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        return ((y * (gamma.double() + e * dg) + beta.double() + e * db) * gy.double()).sum()

    e = 1e-5
    want = (loss(e) - loss(-e)) / (2 * e)
    got = (gx.double() * dx).sum() + (gg.double() * dg).sum() + (gb.double() * db).sum()
    size = (gx.double() * dx).abs().sum() + (gg.double() * dg).abs().sum() + \
        (gb.double() * db).abs().sum()
    # K U of each term's magnitude; the difference itself is good to e^2 and 2^-52 / e
    assert abs(got - want) <= K * U * size + 1e-7 * size


def test_no_rows():
    import product_key_memory_b200 as P
    x = torch.empty(0, 64, device="cuda")
    gamma = torch.ones(64, device="cuda")
    y, h, mean, rstd = P.pkm_layernorm_forward(x, gamma, gamma)
    assert y.shape == (0, 64) and mean.shape == (0,)
    gg = torch.full((64,), 3.0, device="cuda")
    gb = gg.clone()
    P.pkm_layernorm_backward(x, x, mean, rstd, gamma, grad_gamma=gg, grad_beta=gb)
    assert not bool(gg.any()) and not bool(gb.any())


def test_another_stream_and_captured_graph():
    import product_key_memory_b200 as P
    x, add, gamma, beta, rn = _data(500, 1024, BF16, F32)
    gy = rn(500, 1024)
    want = P.pkm_layernorm_forward(x, gamma, beta, add=add)
    wantb = P.pkm_layernorm_backward(gy, want[1], want[2], want[3], gamma)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = P.pkm_layernorm_forward(x, gamma, beta, add=add, stream=side)
    gotb = P.pkm_layernorm_backward(gy, got[1], got[2], got[3], gamma, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + gotb, want + wantb))
    ws = P.alloc_norm_workspace(P.make_norm_shape(500, 1024), "cuda")
    xs, gs = x.clone(), gy.clone()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = P.pkm_layernorm_forward(xs, gamma, beta, add=add)
            gotb = P.pkm_layernorm_backward(gs, got[1], got[2], got[3], gamma, workspace=ws)
    xs.zero_()
    gs.zero_()
    graph.replay()
    torch.cuda.synchronize()
    xs.copy_(x)
    gs.copy_(gy)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + gotb, want + wantb))


@pytest.mark.parametrize("rows,d", [(3000, 100), (5000, 255), (4000, 65), (6000, 33), (3000, 257),
                                    (900, 1001), (700, 2001), (500, 5001), (300, 8191), (200, 16383)])
@pytest.mark.parametrize("kinds", [(F32, F32, F32, F32), (BF16, BF16, None, BF16), (F32, BF16, BF16, F32)])
def test_backward_many_rows_of_odd_widths(rows, d, kinds):
    """Several rows a group and a block, all numbers of groups a block holds, and every place in a
    16-byte block for a row to begin."""
    import product_key_memory_b200 as P
    xt, gt, st, ot = kinds
    x, gsum, gamma, beta, rn = _data(rows, d, xt, st, seed=d + 2)
    gy = rn(rows, d).to(gt)
    _, _, mean, rstd = P.pkm_layernorm_forward(x, gamma, beta)
    gx, check_x = guarded((rows, d), ot)
    got = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma, grad_sum=gsum, grad_x=gx)
    _check_backward(gy, x, mean, rstd, gamma, gsum, got)
    check_x()
    a = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma, grad_sum=gsum, grad_dtype=ot)
    assert all(torch.equal(p, q) for p, q in zip(a, got))


@pytest.mark.parametrize("d", [129, 257, 301, 511, 513, 2001, 8191])
@pytest.mark.parametrize("rows", [3, 900])
def test_forward_odd_widths(rows, d):
    import product_key_memory_b200 as P
    types = [(F32, BF16, BF16), (BF16, F32, BF16), (BF16, None, F32), (F32, None, F32)]
    xt, at, yt = types[(d // 2 + rows) % len(types)]
    x, add, gamma, beta, _ = _data(rows, d, xt, at, seed=d + 3)
    out, check = guarded((rows, d), yt)
    got = P.pkm_layernorm_forward(x, gamma, beta, add=add, out=out)
    _check_forward(x, add, gamma, beta, 1e-5, got)
    check()


@pytest.mark.parametrize("d", [64, 65, 520, 777, 1024, 1600, 4104, 5001, 8200, 16384])
@pytest.mark.parametrize("rows", [5, 400])
@pytest.mark.parametrize("xt,offset", [(F32, 1000.0), (F32, -30.0), (BF16, 30.0)])
def test_backward_rows_far_from_zero(d, rows, xt, offset):
    """Rows whose mean is many deviations: xhat is the difference x - mean, rounded relative to
    itself, times rstd, so the column sums' terms are good relative to |grad_y xhat|, whatever
    the mean."""
    import product_key_memory_b200 as P
    x, _, gamma, beta, rn = _data(rows, d, F32, None, seed=d + 4, scale=1.0)
    x = (x + offset).to(xt)
    gy = rn(rows, d)
    _, _, mean, rstd = P.pkm_layernorm_forward(x, gamma, beta)
    got = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma)
    _check_backward(gy, x, mean, rstd, gamma, None, got)
    _, rg, _ = layernorm_backward(gy, x, mean, rstd, gamma, None)
    xhat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    # A term has two roundings of xhat and one of its product (or none, fused), the sum `rows` at most.
    assert_within("grad_gamma", got[1], rg, (rows + 3) * U * (gy.double() * xhat).abs().sum(0))


@pytest.mark.parametrize("d", [64, 333, 1000, 5001])
def test_backward_over_x(d):
    import product_key_memory_b200 as P
    x, gsum, gamma, beta, rn = _data(300, d, BF16, F32, seed=d)
    gy = rn(300, d)
    _, _, mean, rstd = P.pkm_layernorm_forward(x, gamma, beta)
    want = P.pkm_layernorm_backward(gy, x, mean, rstd, gamma, grad_sum=gsum, grad_dtype=BF16)
    a = x.clone()
    got = P.pkm_layernorm_backward(gy, a, mean, rstd, gamma, grad_sum=gsum, grad_x=a)
    assert got[0].data_ptr() == a.data_ptr() and all(torch.equal(p, q) for p, q in zip(got, want))
    with pytest.raises(P.PKMError):                        # two results in one array
        P.pkm_layernorm_forward(x, gamma, beta, add=gsum, out=a, sum_out=a)
    W = torch.ones(d, d, device="cuda", dtype=BF16)
    for kw in (dict(out=x), dict(pre=x), dict(out=a, pre=a)):
        with pytest.raises(P.PKMError):
            P.pkm_linear_forward(x, W, **kw)
