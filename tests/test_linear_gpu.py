"""The dense layer and its backward on the GPU against a plain 64-bit implementation, element by
element.

A product of K terms accumulates in fp32, 16 terms a step: each step may cut the running sum to
24 bits (2^-23 of its size, which is at most S = sum |a b|), with `pairs` steps for each 16 terms
where operands are planes (6 in fp32 layers, 3 for a backward with an activation), and at most 16
parts are added at the end. Planes: an fp32 value is its three planes to 2^-24, and the
products left out, mid lo, lo mid and lo lo, are at most 2 * 2^-25 + 2^-32 of S. So
  |err of a product| <= E = S (2^-23 (pairs K / 16 + 16) + cut),  cut = 2^-22 or 0.
Activations have slopes below 1.13 in size, second derivatives below 0.8, and cost at most 8
roundings of their result and argument; bias, residual and the output round once each.
"""
import pytest
import torch

from block_ref import (BF16, F32, U, act, act_slope, assert_within, guarded, half_step)

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "silu"]


def _product_bound(S, K, pairs, cut):
    return S * (2.0 ** -23 * (pairs * K / 16 + 16) + cut)


def _data(M, N, K, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * M + 3 * N + K)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return rn(M, K).to(kind), (rn(N, K) * K ** -0.5).to(kind), rn


def _check_forward(x, W, bias, residual, name, y, pre):
    f32 = x.dtype == F32
    K = x.shape[1]
    xd, wd = x.double(), W.double()
    rpre = xd @ wd.t()
    bound = _product_bound(xd.abs() @ wd.abs().t(), K, 6 if f32 else 1, 2.0 ** -22 if f32 else 0)
    if bias is not None:
        rpre = rpre + bias.double()
        bound = bound + U * rpre.abs()
    if pre is not None:
        assert pre.dtype == x.dtype
        assert_within("pre", pre, rpre, bound + half_step(x.dtype) * (rpre.abs() + bound))
    ry = act(rpre, name)
    b = 1.13 * bound
    if name == "relu":
        b = bound
    if name in ("gelu", "silu"):
        b = b + 8 * U * (ry.abs() + rpre.abs() * 0.5 * (rpre.abs() < 12))
    if residual is not None:
        ry = ry + residual.double()
        b = b + U * ry.abs()
    assert_within("y", y, ry, b + half_step(y.dtype) * (ry.abs() + b))


# (M, N, K): single rows and small batches, odd sizes, one of each tile and split, widths of one.
SIZES = [(1, 1, 1), (1, 4096, 1024), (2, 33, 65), (3, 100, 1000), (5, 7, 24), (8, 515, 1001),
         (9, 64, 64), (9, 1, 3000), (16, 130, 72), (33, 515, 1001), (64, 4096, 1024), (129, 257, 8),
         (128, 64, 6400), (300, 1600, 264), (777, 515, 1001), (1500, 1536, 136), (2048, 2048, 192),
         (2100, 2056, 200), (2049, 2305, 77)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kind", [BF16, F32])
def test_forward_sizes(M, N, K, kind):
    import product_key_memory_b200 as P
    x, W, rn = _data(M, N, K, kind)
    i = M + N + K + (kind == F32)
    name = ACTS[i % 4]
    yt = F32 if i % 3 == 0 else kind
    bias = rn(N) if i % 2 else None
    residual = rn(M, N).to(yt) if i % 5 < 3 else None
    out, check_out = guarded((M, N), yt)
    pre, check_pre = guarded((M, N), kind)
    shape = P.make_linear_shape(M, N, K, kind, yt, name)
    ws = P.alloc_linear_workspace(shape, False, "cuda").fill_(255)
    P.pkm_linear_forward(x, W, bias, residual, name, out=out, pre=pre, workspace=ws)
    assert P.pkm_device_status(ws) == 0
    _check_forward(x, W, bias, residual, name, out, pre)
    check_out()
    check_pre()


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("yt", [BF16, F32])
@pytest.mark.parametrize("name", ACTS)
def test_forward_types_and_activations(kind, yt, name):
    import product_key_memory_b200 as P
    for M, N, K in ((4, 72, 80), (40, 72, 80), (200, 131, 96)):
        x, W, rn = _data(M, N, K, kind, seed=5)
        x = x * 3
        bias, residual = rn(N), rn(M, N).to(yt)
        y, pre = P.pkm_linear_forward(x, W, bias, residual, name, want_pre=M != 40)
        assert y.dtype == yt and (pre is None) == (M == 40)
        _check_forward(x, W, bias, residual, name, y, pre)
        y2, _ = P.pkm_linear_forward(x, W, None, None, name, out_dtype=yt)
        _check_forward(x, W, None, None, name, y2, None)


# Few rows: every number of row tiles and of shares of K, ragged in all three sizes, and the two
# sides of each kernel's limits.
FEW = [(5, 40, 8), (5, 1, 24), (6, 4096, 1024), (8, 16, 136), (9, 1600, 6400), (12, 33, 2056),
       (13, 515, 264), (16, 100, 4096), (16, 2400, 520), (17, 100, 264), (24, 4100, 4104),
       (31, 33, 40), (32, 515, 4096), (32, 4096, 1024), (33, 64, 512)]


@pytest.mark.parametrize("M,N,K", FEW)
@pytest.mark.parametrize("yt", [BF16, F32])
def test_forward_few_rows(M, N, K, yt):
    import product_key_memory_b200 as P
    x, W, rn = _data(M, N, K, BF16, seed=4)
    name = ACTS[(M + N) % 4]
    bias = rn(N)
    residual = rn(M, N).to(yt) if M % 2 else None
    out, check_out = guarded((M, N), yt)
    pre, check_pre = guarded((M, N), BF16)
    shape = P.make_linear_shape(M, N, K, BF16, yt, name)
    ws = P.alloc_linear_workspace(shape, False, "cuda").fill_(255)
    P.pkm_linear_forward(x, W, bias, residual, name, out=out, pre=pre, workspace=ws)
    assert P.pkm_device_status(ws) == 0
    _check_forward(x, W, bias, residual, name, out, pre)
    check_out()
    check_pre()
    x[M // 2] = float("inf")                       # the other rows stay as they are
    again, _ = P.pkm_linear_forward(x, W, bias, residual, name, out_dtype=yt)
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(again[keep], out[keep])


def test_forward_residual_in_place_and_repeatable():
    import product_key_memory_b200 as P
    for M in (6, 20, 700):
        x, W, rn = _data(M, 264, 512, BF16)
        residual = rn(M, 264).to(BF16)
        want, _ = P.pkm_linear_forward(x, W, None, residual, "gelu")
        again, _ = P.pkm_linear_forward(x, W, None, residual, "gelu")
        buf = residual.clone()
        got, _ = P.pkm_linear_forward(x, W, None, buf, "gelu", out=buf)
        assert got.data_ptr() == buf.data_ptr()
        assert torch.equal(got, want) and torch.equal(again, want)


@pytest.mark.parametrize("kind", [BF16, F32])
def test_a_non_finite_row_stays_its_own(kind):
    """Rows of a tile share MMAs; a row of x with a NaN or an infinity does not reach the others,
    nor does what lies behind the last row or column."""
    import product_key_memory_b200 as P
    for M, N, K in ((5, 40, 72), (150, 70, 100), (2100, 2056, 72)):
        x, W, rn = _data(M, N, K, kind, seed=1)
        want, _ = P.pkm_linear_forward(x, W, activation="silu")
        for value in (float("nan"), float("inf")):
            bad = x.clone()
            bad[3, K // 2] = value
            got, _ = P.pkm_linear_forward(bad, W, activation="silu")
            keep = torch.arange(M, device="cuda") != 3
            assert torch.equal(got[keep], want[keep])
            plain = act(bad[3:4].double() @ W.double().t(), "silu")
            assert not bool(got[3][~plain[0].isfinite()].isfinite().logical_and(
                plain[0][~plain[0].isfinite()].isnan()).any())


def _check_backward(x, W, gy, pre, name, grads):
    f32 = x.dtype == F32
    M, K = x.shape
    N = W.shape[0]
    xd, wd, gd = x.double(), W.double(), gy.double()
    slope = act_slope(pre.double(), name) if name != "none" else torch.ones_like(gd)
    d = gd * slope
    # d itself: the slope's 8 roundings (of 1.13, and of its argument) and the product's
    dd = gd.abs() * 10 * U * 1.13 if name in ("gelu", "silu") else U * d.abs()
    pairs = 6 if f32 else (3 if name != "none" else 1)
    cut = 2.0 ** -22 if f32 or name != "none" else 0.0
    if "x" in grads:
        gx = grads["x"]
        one = not f32 and name != "none" and gx.dtype == BF16      # d rounded to bf16
        c = half_step(BF16) if one else cut
        b = _product_bound(d.abs() @ wd.abs(), N, 1 if one else pairs, c) + dd @ wd.abs()
        r = d @ wd
        assert_within("grad_x", gx, r, b + half_step(gx.dtype) * (r.abs() + b))
    if "W" in grads:
        b = _product_bound(d.abs().t() @ xd.abs(), M, pairs, cut) + dd.t() @ xd.abs()
        assert_within("grad_W", grads["W"], d.t() @ xd, b)
    if "bias" in grads:
        b = (M + 16) * U * d.abs().sum(0) + dd.sum(0)
        assert_within("grad_bias", grads["bias"], d.sum(0), b)


BACK = [(1, 1, 1), (1, 64, 72), (2, 33, 65), (7, 515, 1001), (16, 130, 72), (64, 4096, 1024),
        (129, 257, 8), (300, 1600, 264), (777, 515, 1001), (3000, 72, 80), (520, 2048, 1536),
        (2100, 2056, 1000), (2049, 2305, 77),
        (1700, 2562, 2600)]                    # rounds of whole tiles, the last one's cut


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("kind", [BF16, F32])
def test_backward_sizes(M, N, K, kind):
    import product_key_memory_b200 as P
    x, W, rn = _data(M, N, K, kind)
    i = M + N + K + (kind == F32)
    name = ACTS[i % 4]
    gx, check_x = guarded((M, K), F32 if i % 3 == 0 else kind)
    gW, check_W = guarded((N, K), F32)
    gb, check_b = guarded((N,), F32)
    pre = rn(M, N).to(kind) if name != "none" else None
    gy = rn(M, N).to(kind)
    shape = P.make_linear_shape(M, N, K, kind, gx.dtype, name)
    ws = P.alloc_linear_workspace(shape, True, "cuda").fill_(255)
    grads = dict(x=gx, W=gW, bias=gb)
    P.pkm_linear_backward(x, W, gy, grads, pre=pre, activation=name, workspace=ws)
    assert P.pkm_device_status(ws) == 0
    _check_backward(x, W, gy, pre, name, grads)
    check_x()
    check_W()
    check_b()


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("name", ACTS)
def test_backward_types_and_subsets(kind, xt, name):
    import product_key_memory_b200 as P
    M, N, K = 210, 136, 88
    x, W, rn = _data(M, N, K, kind, seed=2)
    pre = rn(M, N).to(kind)
    gy = rn(M, N).to(kind)
    full = dict(x=torch.empty(M, K, device="cuda", dtype=xt), W=torch.empty(N, K, device="cuda"),
                bias=torch.empty(N, device="cuda"))
    P.pkm_linear_backward(x, W, gy, full, pre=pre, activation=name)
    _check_backward(x, W, gy, pre, name, full)
    for keys in (("x",), ("W",), ("bias",), ("W", "bias")):
        some = {k: torch.full_like(full[k], 9.0) for k in keys}
        P.pkm_linear_backward(x, W, gy, some, pre=pre, activation=name)
        for k in keys:
            # the same products whatever else is asked for; without x, out_dtype plays no part
            assert torch.equal(some[k], full[k]), k


@pytest.mark.parametrize("name", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(2, 1101, 72), (33, 360, 464), (130, 513, 200), (700, 1304, 520)])
def test_bf16_grad_x_is_its_own_rounding(name, M, N, K):
    """d enters a bf16 grad_x as two planes, d to 2^-16 (each plane leaves at most half a step of
    bf16, 2^-8, of what it stands for), so a result is the 64-bit one to its own half step and
    _check_backward's other terms; d as one plane would be another 2^-8 of each product."""
    import product_key_memory_b200 as P
    x, W, rn = _data(M, N, K, BF16, seed=6)
    pre, gy = rn(M, N).to(BF16), rn(M, N).to(BF16)
    d = gy.double() * act_slope(pre.double(), name)
    dd = gy.double().abs() * 10 * U * 1.13 if name != "relu" else U * d.abs()
    b = _product_bound(d.abs() @ W.double().abs(), N, 2, 2.0 ** -16) + dd @ W.double().abs()
    r = d @ W.double()
    both = dict(x=torch.empty_like(x), W=torch.empty(N, K, device="cuda"))
    alone = dict(x=torch.empty_like(x))
    for grads in (both, alone):
        P.pkm_linear_backward(x, W, gy, grads, pre=pre, activation=name)
        assert_within("grad_x", grads["x"], r, b + half_step(BF16) * (r.abs() + b))
    assert torch.equal(both["x"], alone["x"])


def test_backward_against_differences():
    """Central differences of sum(y gy) in 64 bits against the kernel's gradients along random
    directions, gelu."""
    import product_key_memory_b200 as P
    M, N, K = 50, 70, 90
    x, W, rn = _data(M, N, K, F32, seed=3)
    bias, gy = rn(N), rn(M, N)
    _, pre = P.pkm_linear_forward(x, W, bias, activation="gelu", want_pre=True)
    grads = dict(x=torch.empty_like(x), W=torch.empty_like(W), bias=torch.empty_like(bias))
    P.pkm_linear_backward(x, W, gy, grads, pre=pre, activation="gelu")
    dirs = dict(x=rn(M, K).double(), W=rn(N, K).double() * K ** -0.5, bias=rn(N).double())

    def loss(e):
        p = (x.double() + e * dirs["x"]) @ (W.double() + e * dirs["W"]).t()
        return (act(p + bias.double() + e * dirs["bias"], "gelu") * gy.double()).sum()

    e = 1e-5
    want = (loss(e) - loss(-e)) / (2 * e)
    got = sum((grads[k].double() * dirs[k]).sum() for k in dirs)
    size = sum((grads[k].double() * dirs[k]).abs().sum() for k in dirs)
    # products of 90 terms: 2^-23 (6 * 90 / 16 + 16) + 2^-22 of terms a few times their sum;
    # the difference's third-order term e^2
    assert abs(got - want) <= 1e-4 * size


def test_no_rows():
    import product_key_memory_b200 as P
    x, W = torch.empty(0, 40, device="cuda"), torch.ones(24, 40, device="cuda")
    y, pre = P.pkm_linear_forward(x, W, want_pre=True)
    assert y.shape == (0, 24) and pre.shape == (0, 24)
    g = dict(x=torch.empty(0, 40, device="cuda"), W=torch.ones(24, 40, device="cuda"),
             bias=torch.ones(24, device="cuda"))
    P.pkm_linear_backward(x, W, y, g)
    assert not bool(g["W"].any()) and not bool(g["bias"].any())


def test_another_stream_two_at_once_and_captured_graph():
    import product_key_memory_b200 as P
    cases = []
    for M in (4, 600, 2100):
        x, W, rn = _data(M, 2056, 512, BF16)
        gy = rn(M, 2056).to(BF16)
        cases.append((x, W, rn(2056), gy))

    def both(x, W, bias, gy, stream=None, spaces=(None, None)):
        y, pre = P.pkm_linear_forward(x, W, bias, activation="gelu", want_pre=True, stream=stream,
                                      workspace=spaces[0])
        g = dict(x=torch.empty_like(x), W=torch.empty(W.shape, device="cuda"),
                 bias=torch.empty_like(bias))
        P.pkm_linear_backward(x, W, gy, g, pre=pre, activation="gelu", stream=stream,
                              workspace=spaces[1])
        return [y, pre, g["x"], g["W"], g["bias"]]
    want = [both(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [both(*c, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    for c, w in zip(cases, want):
        fixed = [t.clone() for t in c]
        side = streams[0]
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = both(*fixed)
        for t in fixed:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, s in zip(fixed, c):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, w))


def _all_bf16(limit):
    """Every bf16 value v of 2^-60 < |v| < limit: exact as an operand of any type."""
    v = torch.arange(0, 1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(BF16)
    return v[(v.float().abs() < limit) & (v.float().abs() > 2.0 ** -60)]


@pytest.mark.parametrize("name,limit", [("gelu", 13.0), ("silu", 86.0)])
@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("as_weights", [False, True])
def test_activations_relative_to_themselves(name, limit, kind, as_weights):
    """fp32 results of gelu and silu on every bf16 value (pre is that value: one product with 1): within
    2^-19 of themselves, however small. Of the polynomial 1.2e-7 (2 U); t 3 U, the polynomial's
    steps 4 U, t and the exponential 2^-22 (4 U) and its correction 2 U, products and sums 4 U: 19
    of 32 U. The slopes' two terms may cancel, each is as good."""
    import product_key_memory_b200 as P
    v = _all_bf16(limit)
    n = v.numel()
    one = torch.ones(1, 1, device="cuda", dtype=kind)
    col = v.to(kind)[:, None].contiguous()
    x, W = (one, col) if as_weights else (col, one)
    y, pre = P.pkm_linear_forward(x, W, activation=name, out_dtype=F32, want_pre=True)
    assert torch.equal(pre.flatten(), v.to(kind))
    want = act(v.double(), name)
    assert_within("y", y.flatten(), want, 2.0 ** -19 * want.abs())
    if as_weights:
        return
    for r in (40, 8):                                       # rounded to bf16: whole tiles, few rows
        xb = v[: n // r * r].view(r, -1).t().contiguous() if r == 40 else v[:r].view(r, 1)
        Wb = torch.eye(r, device="cuda", dtype=BF16) if r == 40 else torch.ones(8, 1, device="cuda", dtype=BF16)
        yb, _ = P.pkm_linear_forward(xb.to(BF16), Wb, activation=name)
        wb = act((xb.double() @ Wb.double().t()), name)
        assert_within("bf16 y", yb, wb, (half_step(BF16) + 2.0 ** -15) * wb.abs() + 2.0 ** -126)
    g = dict(bias=torch.empty(n, device="cuda"))            # a column each: the sum of one slope
    ones = torch.ones(1, n, device="cuda", dtype=kind)
    P.pkm_linear_backward(one, torch.ones(n, 1, device="cuda", dtype=kind), ones, g,
                          pre=v.to(kind)[None].contiguous(), activation=name)
    d = v.double()
    s = torch.sigmoid(d)
    terms = (0.5 * torch.special.erfc(-d * 0.5 ** 0.5), d * torch.exp(-0.5 * d * d) * 0.3989422804014327) \
        if name == "gelu" else (s, s * d * torch.sigmoid(-d))
    assert_within("slope", g["bias"], act_slope(d, name), 2.0 ** -19 * (terms[0].abs() + terms[1].abs()))


def _norm_error(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


# The tensor cores cut the running sum by 2^-25 of it on average at each step of 16 terms; it is
# taken out every 4 K blocks, 16 steps, over which it grows like the root of their number: 10.7
# steps' worth, 10.7 * 2^-25 = 3.2e-7 of the part and so of the sum. At most 128 takings and parts
# add their roundings' root mean square, sqrt(128) * 2^-25 * 0.6 / 3 (partial sums grow alike) =
# 0.7e-7. What planes leave out and their own roundings are 2^-24 each in single terms, below
# 0.1e-7 of the sum of 264 and more. A product of planes left out would be 2e-6 or more, a taking
# half as often 6.4e-7.
LONG_SUM = 4e-7


@pytest.mark.parametrize("K", [264, 1001, 4096])
@pytest.mark.parametrize("rows,cols", [(300, 520), (2400, 2100)])       # cut along K; whole tiles too
@pytest.mark.parametrize("kind", [BF16, F32])
def test_long_sums_in_fp32(K, rows, cols, kind):
    """fp32 results as whole arrays: the forward over K, grad_x over N, grad_W over M."""
    import product_key_memory_b200 as P
    x, W, rn = _data(rows, cols, K, kind, seed=8)
    y, _ = P.pkm_linear_forward(x, W, out_dtype=F32)
    assert _norm_error(y, x.double() @ W.double().t()) < LONG_SUM
    for name in ("none", "relu"):                        # relu: d takes planes, its slope is exact
        for M, N, k in ((rows, K, cols), (K, cols, rows)):   # the long sum is N's, then M's
            x, W, rn = _data(M, N, k, kind, seed=9)
            gy, pre = rn(M, N).to(kind), rn(M, N).to(kind)
            d = gy.double() * act_slope(pre.double(), name) if name != "none" else gy.double()
            g = dict(x=torch.empty(M, k, device="cuda"), W=torch.empty(N, k, device="cuda"))
            P.pkm_linear_backward(x, W, gy, g, pre=pre if name != "none" else None, activation=name)
            assert _norm_error(g["x"], d @ W.double()) < LONG_SUM
            assert _norm_error(g["W"], d.t() @ x.double()) < LONG_SUM


def test_bf16_results_of_very_long_sums():
    """Sums of 65,536 positive terms on whole tiles, forward and grad_x, against the 64-bit sums
    rounded to bf16. Cuts towards zero all have one sign. Taken out every 16 steps they are at most
    16 * 2^-24 = 1e-6 of a sum, 0.07 of 2^16; the sums have a deviation of 107, so a step of bf16
    (256, 2^-8 of them) is crossed by at most 0.07 * 0.4 / 107 of them: 1e-6 on the mean. Never
    taken out, 4096 cuts of 2^-25 on average of a running sum that is half of the result are 6e-5,
    4 of 2^16: some 2e-5 on the mean."""
    import product_key_memory_b200 as P
    M, wide, K = 40, 75 * 256, 1 << 16                # 75 tiles: 74 whole ones
    g = torch.Generator(device="cuda").manual_seed(11)
    W = torch.rand(wide, K, generator=g, device="cuda", dtype=BF16) + 0.5
    x = torch.rand(M, K, generator=g, device="cuda").to(BF16) + 0.5
    ref = torch.cat([x.double() @ w.double().t() for w in W.chunk(16)], 1)

    def off(y):
        return abs(float((y.double() / ref.to(BF16).double() - 1).mean()))
    y, _ = P.pkm_linear_forward(x, W)
    assert off(y) < 1.5e-6
    gx = torch.empty(M, wide, device="cuda", dtype=BF16)
    Wt = W.t().contiguous()
    P.pkm_linear_backward(torch.empty(M, wide, device="cuda", dtype=BF16), Wt, x, dict(x=gx))
    assert off(gx) < 1.5e-6


@pytest.mark.parametrize("M", [40, 700])
def test_the_largest_fp32_values(M):
    """Finite values above the largest bf16 (3.39e38), which would round to infinity there."""
    import product_key_memory_b200 as P
    N, K = 72, 136
    x, W, rn = _data(M, N, K, F32, seed=12)
    gy = rn(M, N)
    x[::3, 5] = 3.4e38
    x[1::3, 7] = -3.4028e38
    gy[3::5, 9] = 3.3999e38
    W = W * 2.0 ** -20
    y, _ = P.pkm_linear_forward(x, W)
    _check_forward(x, W, None, None, "none", y, None)
    g = dict(x=torch.empty(M, K, device="cuda"))
    P.pkm_linear_backward(x, W, gy, g)
    _check_backward(x, W, gy, None, "none", g)
    g = dict(W=torch.empty(N, K, device="cuda"))
    small = gy.clamp(-8, 8) * 2.0 ** -20
    P.pkm_linear_backward(x, W, small, g)
    _check_backward(x, W, small, None, "none", g)
    assert all(bool(t.isfinite().all()) for t in (y, g["W"]))


# Small fp32 layers: each height of a tile (16, 32, 64 rows), one to eight shares of K, shares that end
# inside a step, widths next to a tile's 64, and both sides of the limit to the tensor cores.
SMALL_F32 = [(9, 1, 1), (9, 63, 4351), (16, 64, 33), (17, 65, 31), (32, 129, 300), (33, 40, 1000),
             (64, 64, 64), (65, 200, 8), (100, 33, 2000), (500, 100, 129), (777, 93, 320),
             (1200, 70, 40), (300, 400, 264), (512, 512, 512), (600, 600, 600), (58, 3136, 40)]


@pytest.mark.parametrize("M,N,K", SMALL_F32)
@pytest.mark.parametrize("name", ACTS)
def test_small_fp32_layers(M, N, K, name):
    import product_key_memory_b200 as P
    x, W, rn = _data(M, N, K, F32, seed=13)
    yt, xt = ((F32, BF16), (BF16, F32), (F32, F32))[(M + N) % 3]
    bias, residual = rn(N), rn(M, N).to(yt)
    out, check_out = guarded((M, N), yt)
    pre, check_pre = guarded((M, N), F32)
    ws = P.alloc_linear_workspace(P.make_linear_shape(M, N, K, F32, yt, name)).fill_(255)
    P.pkm_linear_forward(x, W, bias, residual, name, out=out, pre=pre, workspace=ws)
    assert P.pkm_device_status(ws) == 0
    _check_forward(x, W, bias, residual, name, out, pre)
    again, _ = P.pkm_linear_forward(x, W, bias, residual.clone(), name, out_dtype=yt)
    assert torch.equal(again, out)
    check_out()
    check_pre()
    gy, pre = rn(M, N), rn(M, N) if name != "none" else None
    gx, check_x = guarded((M, K), xt)
    gW, check_W = guarded((N, K), F32)
    gb, check_b = guarded((N,), F32)
    ws = P.alloc_linear_workspace(P.make_linear_shape(M, N, K, F32, xt, name), True).fill_(255)
    grads = dict(x=gx, W=gW, bias=gb)
    P.pkm_linear_backward(x, W, gy, grads, pre=pre, activation=name, workspace=ws)
    assert P.pkm_device_status(ws) == 0
    _check_backward(x, W, gy, pre, name, grads)
    for check in (check_x, check_W, check_b):
        check()
    for keys in (("x",), ("W",), ("bias",), ("x", "bias")):
        some = {k: torch.full_like(grads[k], 9.0) for k in keys}
        P.pkm_linear_backward(x, W, gy, some, pre=pre, activation=name)
        assert all(torch.equal(some[k], grads[k]) for k in keys), keys


def test_small_fp32_layers_on_streams_and_in_a_graph():
    import product_key_memory_b200 as P
    x, W, rn = _data(200, 136, 500, F32, seed=14)
    gy = rn(200, 136)

    def both(stream=None):
        y, pre = P.pkm_linear_forward(x, W, activation="silu", want_pre=True, stream=stream)
        g = dict(x=torch.empty_like(x), W=torch.empty_like(W), bias=torch.empty(136, device="cuda"))
        P.pkm_linear_backward(x, W, gy, g, pre=pre, activation="silu", stream=stream)
        return [y, pre, *g.values()]
    want = both()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [both(s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    with torch.cuda.stream(streams[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            out = both()
    for t in out:
        t.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    bad = x.clone()
    bad[7, 3] = float("nan")
    y, _ = P.pkm_linear_forward(bad, W, activation="silu")
    keep = torch.arange(200, device="cuda") != 7
    assert torch.equal(y[keep], want[0][keep]) and bool(y[7].isnan().all())
