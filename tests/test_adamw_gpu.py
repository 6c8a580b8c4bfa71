"""AdamW over lists of tensors on the GPU: states bit for bit against the formula evaluated step by
step in fp32 (codes and scales of 8-bit states included, but for second moments within the
root's error of the middle of two codes), parameters against 64 bits within
the roundings counted in block_ref.adamw."""
import pytest
import torch

from block_ref import BF16, F32, adamw, assert_within, guarded, half_step

pytestmark = pytest.mark.gpu
HYPER = dict(lr=3e-3, step=7, betas=(0.9, 0.98), eps=1e-8, grad_scale=0.5, seed=99)
KEYS = ("param", "grad", "master", "m", "v", "m_scale", "v_scale")


def _tensor(P, n, pt, gt, bits, master=False, seed=0, fresh=False, wd=0.1, lr_scale=1.0):
    """One entry with warm states (made by two steps of the plain form), inside sentinels."""
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + n)
    rn = lambda: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    checks = []

    def put(t):
        out, check = guarded(t.shape, t.dtype if t.dtype != torch.float8_e4m3fn else torch.uint8)
        checks.append(check)
        out = out if t.dtype != torch.float8_e4m3fn else out.view(torch.float8_e4m3fn)
        out.copy_(t)
        return out
    full = rn()
    t = dict(param=put(full.to(pt)), grad=put((rn() * 1e-2).to(gt)), weight_decay=wd,
             lr_scale=lr_scale)
    if master:
        t["master"] = put(full)
    state = P.alloc_adamw_state(t["param"], bits)
    for step in ((1, 2) if not fresh else ()):
        new = adamw(dict(t, **state, grad=rn() * 1e-2), dict(HYPER, step=step), 0)
        state = {k: new[k] for k in state}
    t.update({k: put(x) for k, x in state.items()})
    return t, checks


def _bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _equal(a, b):
    return bool(((_bits(a) == _bits(b)) | (a.float().isnan() & b.float().isnan())).all())


def _copy(t):
    return {k: (v.clone() if torch.is_tensor(v) else v) for k, v in t.items()}


def _check(t, before, hyper, index, zero=False):
    want = adamw(before, hyper, index)
    for k in ("m", "v", "m_scale", "v_scale"):
        if k in want:
            same = (_bits(t[k]) == _bits(want[k])) | (t[k].float().isnan() & want[k].float().isnan())
            if k == "v" and "v_edge" in want:
                same |= want["v_edge"] & ((_bits(t[k]).int() - _bits(want[k]).int()).abs() <= 1)
            assert bool(same.all()), "%s of tensor %d (n %d)" % (k, index, t[k].numel())
    if t.get("master") is not None:
        assert_within("master", t["master"], want["param"], want["bound"])
        assert torch.equal(t["param"], t["master"].to(t["param"].dtype))
    else:
        b = want["bound"]
        if t["param"].dtype != F32:
            b = b + half_step(t["param"].dtype) * (want["param"].abs() + b)
        assert_within("param", t["param"], want["param"], b)
    if zero:
        assert not bool(t["grad"].any())
    else:
        assert torch.equal(t["grad"], before["grad"])


SIZES = [1, 2, 7, 8, 255, 256, 257, 511, 2047, 2048, 2049, 5000, 100003]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,master", [(F32, False), (BF16, False), (BF16, True)])
@pytest.mark.parametrize("gt", [F32, BF16])
def test_sizes_and_types(bits, pt, master, gt):
    import product_key_memory_b200 as P
    made = [_tensor(P, n, pt, gt, bits, master, seed=i) for i, n in enumerate(SIZES)]
    ts = [t for t, _ in made]
    zero = gt == BF16
    before = [_copy(t) for t in ts]
    P.pkm_adamw_step(P.make_adamw_tensors(ts), zero_grad=zero, **HYPER)
    for i, t in enumerate(ts):
        _check(t, before[i], HYPER, i, zero)
    for _, checks in made:
        for c in checks:
            c()


def test_first_steps_from_zero_states():
    import product_key_memory_b200 as P
    ts = [_tensor(P, n, F32, F32, bits, seed=n, fresh=True)[0] for n in (300, 4097) for bits in (32, 8)]
    lst = P.make_adamw_tensors(ts)
    for step in range(1, 6):
        hyper = dict(HYPER, step=step, grad_scale=1.0)
        for i, t in enumerate(ts):
            t["grad"].copy_(torch.randn(t["grad"].numel(), device="cuda") * 10.0 ** -step)
        before = [_copy(t) for t in ts]
        P.pkm_adamw_step(lst, **hyper)
        for i, t in enumerate(ts):
            _check(t, before[i], hyper, i)


def test_every_code_of_a_long_tensor():
    """Roots are rounded to nearest before their dither, so every code of the second moment is the
    plain form's, however near to the middle of two codes its value lies."""
    import product_key_memory_b200 as P
    ts = [_tensor(P, n, F32, F32, 8, seed=n)[0] for n in (8 << 20, (4 << 20) + 77)]
    before = [_copy(t) for t in ts]
    P.pkm_adamw_step(P.make_adamw_tensors(ts), **HYPER)
    for i, t in enumerate(ts):
        want = adamw(before[i], HYPER, i)
        for k in ("m", "v", "m_scale", "v_scale"):
            assert _equal(t[k], want[k]), k


def test_mixed_long_list():
    """More tensors than one launch takes, of every kind, empty ones among them."""
    import product_key_memory_b200 as P
    ts = []
    for i in range(600):
        pt, master = [(F32, False), (BF16, False), (BF16, True)][i % 3]
        ts.append(_tensor(P, (i * 37) % 900 if i % 50 else 0, pt, [F32, BF16][i % 2],
                          [32, 8][(i // 2) % 2], master, seed=i, wd=0.01 * (i % 3),
                          lr_scale=[1.0, 0.25][i % 2])[0])
    before = [_copy(t) for t in ts]
    P.pkm_adamw_step(P.make_adamw_tensors(ts), **HYPER)
    for i, t in enumerate(ts):
        if t["param"].numel():
            _check(t, before[i], HYPER, i)


def test_extreme_values_in_8_bits():
    """Blocks of zeros, of one value, at the scales' borders, of tiny and of huge values."""
    import product_key_memory_b200 as P
    t, _ = _tensor(P, 256 * 13, F32, F32, 8, fresh=True)
    g = t["grad"].view(13, 256)
    g[0] = 0
    g[1] = 1.0
    g[2] *= 1e-30
    g[3] *= 1e15
    g[4] = 0
    g[4, 17] = -3.0
    g[5] = 448.0 / (0.1 * 0.5)             # largest m at, just below and just above 448
    g[6] = 448.0 / (0.1 * 0.5) * (1 + 2.0 ** -20)
    g[7] = 448.0 / (0.1 * 0.5) * (1 - 2.0 ** -20)
    g[8] = torch.logspace(-30, 3, 256, device="cuda")
    g[9] = torch.logspace(-7, 0, 256, device="cuda")
    g[10] = 1e-38
    g[11] *= 1e-20
    lst = P.make_adamw_tensors([t])
    for step in (1, 2, 3):
        before = _copy(t)
        P.pkm_adamw_step(lst, **dict(HYPER, step=step))
        _check(t, before, dict(HYPER, step=step), 0)
    assert bool((t["param"].view(13, 256)[0] == 0).logical_not().all())   # decay only, no NaN
    assert bool(t["param"].isfinite().all())


@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_gradients_stay_in_their_block(bits):
    import product_key_memory_b200 as P
    for value in (float("inf"), float("nan")):
        t, _ = _tensor(P, 1000, F32, F32, bits)
        t["grad"][300] = value
        before = _copy(t)
        P.pkm_adamw_step(P.make_adamw_tensors([t]), **HYPER)
        want = adamw(before, HYPER, 0)
        for k in ("m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
            assert _equal(t[k], want[k])
        bad = torch.zeros(1000, dtype=torch.bool, device="cuda")
        bad[300] = True
        assert bool(t["param"][~bad].isfinite().all())
        lost = t["m"].float().isnan() if bits == 8 else ~t["m"].isfinite()
        if bits == 8:
            bad[256:512] = True
        assert torch.equal(lost, bad)


def test_a_moment_that_is_a_code_stays_that_code():
    """With beta2 = 0 the new r is |g|: a gradient of codes times a power of two comes back as
    it is whatever the dither, but for powers of two, which may go one code down."""
    import product_key_memory_b200 as P
    codes = torch.arange(0, 127, dtype=torch.uint8, device="cuda")
    two = ((codes & 7) == 0) & (codes > 8)        # the codes below lie half as far apart
    two = two.repeat(40)[:256 * 19]
    codes = codes.repeat(40)[:256 * 19]
    g = codes.view(torch.float8_e4m3fn).float() * 2.0 ** -12
    t = dict(param=torch.zeros_like(g), grad=g, **P.alloc_adamw_state(g, 8))
    lst = P.make_adamw_tensors([t])
    for step in range(1, 9):
        P.pkm_adamw_step(lst, lr=0.0, step=step, betas=(0.0, 0.0), seed=step)
        m, v = (t[k].float() * t[k + "_scale"].repeat_interleave(256) for k in ("m", "v"))
        assert torch.equal(m, g) and torch.equal(v[~two], g[~two])
        assert bool(((v[two] == g[two]) | (v[two] == g[two] * (15 / 16))).all())


def test_a_moment_without_gradients_decays_at_its_rate():
    """The 8-bit moment falls at the rate of the 32-bit one on average (rounding to nearest
    would hold it)."""
    import product_key_memory_b200 as P
    n = 1 << 16
    p = torch.zeros(n, device="cuda")
    t = dict(param=p, grad=torch.zeros(n, device="cuda"), **P.alloc_adamw_state(p, 8))
    t["grad"].copy_(torch.rand(n, device="cuda") + 0.5)
    lst = P.make_adamw_tensors([t])
    P.pkm_adamw_step(lst, lr=0.0, step=1, betas=(0.0, 0.5), seed=5)
    r0 = (t["v"].float() * t["v_scale"].repeat_interleave(256)).double()
    t["grad"].zero_()
    for step in range(2, 202):
        P.pkm_adamw_step(lst, lr=0.0, step=step, betas=(0.9, 0.999), seed=5)
    r1 = (t["v"].float() * t["v_scale"].repeat_interleave(256)).double()
    # Each element's r falls by 0.999^(200/2) = 0.9048 on average. The dither's noise per step is
    # at most sqrt(5e-4 * step size 1/8) of r, over 200 steps below 12 % of an element and
    # below 0.12 / 2^8 of the mean over 2^16: five of those and the 1e-3 of drift of r^2. An
    # element that passes a power of two on its way (log2(1 / 0.9048) = 14.4 % of them) may
    # be one code, 1/16, further down there.
    ratio = (r1.sum() / r0.sum()).item()
    noise = 5 * 0.12 / 256 + 1e-3
    assert -0.144 / 16 - noise < ratio - 0.999 ** 100 < noise


def test_deterministic_and_seeded():
    import product_key_memory_b200 as P
    a, _ = _tensor(P, 70000, BF16, F32, 8, True)
    b, c = _copy(a), _copy(a)
    P.pkm_adamw_step(P.make_adamw_tensors([a]), **HYPER)
    P.pkm_adamw_step(P.make_adamw_tensors([b]), **HYPER)
    P.pkm_adamw_step(P.make_adamw_tensors([c]), **dict(HYPER, seed=100))
    assert all(_equal(a[k], b[k]) for k in KEYS)
    assert not _equal(a["v"], c["v"]) and _equal(a["m"], c["m"])


def test_device_hyper_parameters_and_captured_step():
    import product_key_memory_b200 as P
    ts = [_tensor(P, n, BF16, F32, bits, True, seed=n)[0] for n in (3000, 9) for bits in (32, 8)]
    ref = [_copy(t) for t in ts]
    dyn = torch.zeros(3, device="cuda")
    lst, rlst = P.make_adamw_tensors(ts), P.make_adamw_tensors(ref)
    hyper = dict(betas=HYPER["betas"], eps=HYPER["eps"], seed=3)
    start = [_copy(t) for t in ts]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            P.pkm_adamw_step(lst, lr=123.0, step=1, dyn=dyn, **hyper)
    torch.cuda.synchronize()
    assert all(_equal(t[k], s[k]) for t, s in zip(ts, start) for k in s if torch.is_tensor(s[k]))
    for step, lr, gs in ((5, 2.0 ** -9, 1.0), (6, 2.0 ** -8, 0.25), (5000, 2.0 ** -9, 1.0)):
        dyn.copy_(torch.tensor([lr, float(step), gs]))
        before = [_copy(t) for t in ts]
        graph.replay()
        P.pkm_adamw_step(rlst, lr=lr, step=step, grad_scale=gs, **hyper)
        torch.cuda.synchronize()
        full = dict(hyper, lr=lr, step=step, grad_scale=gs)
        for i, (t, r) in enumerate(zip(ts, ref)):
            _check(t, before[i], full, i)
            assert all(_equal(t[k], r[k]) for k in ("m", "v"))
            for k in r:      # the next step starts from the same values on both sides
                if torch.is_tensor(r[k]):
                    r[k].copy_(t[k])


def test_another_stream():
    import product_key_memory_b200 as P
    t, _ = _tensor(P, 50000, F32, F32, 32)
    before = _copy(t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    P.pkm_adamw_step(P.make_adamw_tensors([t]), stream=side, **HYPER)
    side.synchronize()
    _check(t, before, HYPER, 0)


def test_empty_list():
    import product_key_memory_b200 as P
    P.pkm_adamw_step(P.make_adamw_tensors([]), **HYPER)


def test_overlap_refused():
    import product_key_memory_b200 as P
    t, _ = _tensor(P, 512, F32, F32, 32)
    with pytest.raises(ValueError, match="overlap"):
        P.make_adamw_tensors([t, t])
    with pytest.raises(ValueError, match="overlap"):
        P.make_adamw_tensors([dict(t, v=t["m"])])
