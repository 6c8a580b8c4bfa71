"""Plain implementations in 64 bits of the transformer-block operators, and helpers of their tests."""
import torch

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24            # half a step of fp32, relative
SENTINEL = 7.0            # held exactly by every type, bytes too


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def guarded(shape, dtype, device="cuda", pad=64):
    """A contiguous tensor of `shape` with `pad` sentinel elements before and behind it: (tensor,
    check), check() asserts that the sentinels are as they were."""
    n = 1
    for s in shape:
        n *= s
    flat = torch.full((n + 2 * pad,), SENTINEL, dtype=dtype, device=device)
    t = flat[pad:pad + n].view(shape)

    def check():
        assert bool((flat[:pad].float() == SENTINEL).all()), "written before the start"
        assert bool((flat[pad + n:].float() == SENTINEL).all()), "written past the end"
    return t, check


def assert_within(name, got, ref, bound):
    """|got - ref| <= bound element by element (got widened to 64 bits)."""
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = int((err - bound).nan_to_num(float("inf")).argmax())
        raise AssertionError("%s: %d of %d outside; worst at %d: got %r, want %r, bound %r" % (
            name, int(bad.sum()), bad.numel(), i, got.double().flatten()[i].item(),
            ref.flatten()[i].item(), bound.expand_as(ref).flatten()[i].item()))


def layernorm(x, add, gamma, beta, eps):
    """(h as stored, mean, rstd, y), 64 bits from the stored h on."""
    h = x if add is None else (x.float() + add.float()).to(x.dtype)
    hd = h.double()
    mean = hd.mean(1)
    c = hd - mean[:, None]
    rstd = (c.square().mean(1) + eps).rsqrt()
    y = c * rstd[:, None] * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return h, mean, rstd, y


def layernorm_backward(gy, x, mean, rstd, gamma, gsum):
    gy, x, mean, rstd, gamma = (t.double() for t in (gy, x, mean, rstd, gamma))
    xhat = (x - mean[:, None]) * rstd[:, None]
    t = gy * gamma
    gx = rstd[:, None] * (t - t.mean(1, keepdim=True) - xhat * (t * xhat).mean(1, keepdim=True))
    if gsum is not None:
        gx = gx + gsum.double()
    return gx, (gy * xhat).sum(0), gy.sum(0)


# ------------------------------------------------------------------------------- AdamW
MASK = 0xffffffff


def mix32(h):
    """MurmurHash3's 32-bit finaliser on a tensor of int64 (or an int) below 2^32."""
    h = h ^ (h >> 16)
    h = (h * 0x85ebca6b) & MASK
    h = h ^ (h >> 13)
    h = (h * 0xc2b2ae35) & MASK
    return h ^ (h >> 16)


def block_scale(t):
    """Power-of-two scale of each 256 elements, by comparisons with every candidate."""
    n = t.numel()
    full = torch.zeros(-(-n // 256) * 256, dtype=torch.float64, device=t.device)
    full[:n] = t.double()
    most = full.view(-1, 256).abs().amax(1)
    steps = torch.arange(-100, 121, device=t.device)
    powers = torch.ldexp(torch.ones(221, dtype=torch.float64, device=t.device), steps)
    ok = most[:, None] <= 448 * powers[None]
    s = powers[ok.int().argmax(1)].float()
    return torch.where(most.isfinite(), s, torch.full_like(s, float("nan")))


def adamw(t, hyper, index):
    """One step of one tensor (a dict as make_adamw_tensors takes it): the new m, v (and codes
    and scales) step by step in fp32, and (param, bound) in 64 bits."""
    lr, step, (b1, b2), eps, gs, seed = (hyper[k] for k in
                                         ("lr", "step", "betas", "eps", "grad_scale", "seed"))
    n = t["param"].numel()
    eight = t.get("m_scale") is not None
    lr = lr * t.get("lr_scale", 1.0)
    g = t["grad"].flatten().float() * gs
    m, v = t["m"].flatten().float(), t["v"].flatten().float()
    if eight:
        m = m * t["m_scale"].repeat_interleave(256)[:n]
        v = (v * t["v_scale"].repeat_interleave(256)[:n]).square()
    p = (t["param"] if t.get("master") is None else t["master"]).flatten().double()
    md, gd = m.double(), g.double()
    big = b1 * md.abs() + (1 - b1) * gd.abs()
    mn = b1 * m + (1 - b1) * g
    vn = b2 * v + (1 - b2) * g * g
    vd = b2 * v.double() + (1 - b2) * gd.square()
    den = (vd / (1 - b2 ** step)).sqrt() + eps
    over = lr / (1 - b1 ** step)
    wd = t.get("weight_decay", 0.0)
    pd = p * (1 - lr * wd) - over * (b1 * md + (1 - b1) * gd) / den
    # Roundings: keep, its product and the subtraction (3 U of |p|); m 3, v 4 halved by the root
    # plus its own, root, denominator 2, quotient, step, product: 16 U of the update's size
    # with m's two terms apart, and the subtraction's own of the update.
    bound = 3 * U * p.abs() + 17 * U * over * big / den
    out = {"param": pd, "bound": bound}
    if not eight:
        out["m"], out["v"] = mn, vn
        return out
    r = vn.sqrt()
    out["m_scale"], out["v_scale"] = block_scale(mn), block_scale(r)
    out["m"] = (mn / out["m_scale"].repeat_interleave(256)[:n]).to(torch.float8_e4m3fn)
    q = r / out["v_scale"].repeat_interleave(256)[:n]
    key = mix32(mix32((seed + 0x9e3779b9 * step) & MASK) ^ ((0x9e3779b9 * index) & MASK))
    i = torch.arange(n, device=q.device)
    h = mix32((i // 2) ^ key)
    b = torch.where(i % 2 == 0, h & 0xffff, h >> 16).double()
    ulp = torch.ldexp(torch.ones_like(b), (torch.frexp(q.double())[1] - 1).clamp(min=-6) - 3)
    near = (q + (ulp * (b - 32767.5) / 65536).float()).clamp(2.0 ** -9, 448.0)
    out["v"] = torch.where(q > 0, near, q).to(torch.float8_e4m3fn)
    # The kernel's root is good to 2^-22: 2^-18 of a code at most (16 steps an octave), so a
    # value this near to the middle of two codes may go to either, and one this near to a power
    # of two may have the dither of the other side (half or twice as wide).
    at = torch.ldexp(torch.ones_like(b), (torch.frexp(near.double())[1] - 1).clamp(min=-6) - 3)
    part = near.double() / at
    power = ((torch.frexp(q.double())[0] * 2 - 1.5).abs() - 0.5).abs() < 2.0 ** -20
    out["v_edge"] = (((part - part.floor() - 0.5).abs() < 2.0 ** -16) | power) & (q > 0)
    return out


# ------------------------------------------------------------------------------- dense layer
def act(t, name):
    if name == "relu":
        return torch.where(t <= 0, torch.zeros_like(t), t)
    if name == "gelu":
        return 0.5 * t * torch.special.erfc(-t * 0.5 ** 0.5)
    if name == "silu":
        return t * torch.sigmoid(t)
    return t


def act_slope(t, name):
    if name == "relu":
        return (t > 0).to(t.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-t * 0.5 ** 0.5) + \
            t * torch.exp(-0.5 * t * t) * 0.3989422804014327
    if name == "silu":
        s = torch.sigmoid(t)
        return s * (1 + t * (1 - s))
    return torch.ones_like(t)
