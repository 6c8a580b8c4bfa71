"""Plain implementations in 64 bits of the transformer-block operators, and helpers of their tests."""
import torch

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24            # half a step of fp32, relative
SENTINEL = 7.25


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
