"""The transformer-block operators together with the memory layer, as a model's step uses them:

  n1 = LN1(x)            m = memory(n1)          n2, h = LN2(x + m)
  u = gelu(n2 W1^T + b1)                         y = u W2^T + b2 + h

forward, backward from grad_y, and AdamW on every parameter; against 64-bit autograd with the
memory's picks held fixed, and the step captured in a graph against the eager one.

Tolerances (relative, 2-norm). fp32: a product of K <= 256 terms is within 2^-23 (6 K / 16 + 16)
<= 1.34e-5 of sum |a b|, which for terms of random sign is about 0.64 sqrt(K) <= 10.2 times the
result: 1.4e-4 of it at most, were every step cut alike. Seven products lie on the longest way
(q, W1, W2 forward; W2, W1, the memory's and q's backward); norms, softmax and gelu hand
relative errors on with a factor near 1 and add a few 2^-24: 7 * 1.4e-4 = 1e-3.
bf16: each of the eleven stored intermediates is off by at most 2^-9 of its own size, and the
operands are the oracle's: 11 * 2^-9 = 0.0215 if all add up in one direction.
"""
import pytest
import torch

from block_ref import BF16, F32, adamw, assert_within, half_step

pytestmark = pytest.mark.gpu
B, D, H, DQ, N, K, FF = 130, 128, 2, 32, 32, 8, 256
EPS = 1e-5


def _model(kind):
    g = torch.Generator(device="cuda").manual_seed(11)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    p = dict(gamma1=1 + 0.1 * rn(D), beta1=0.1 * rn(D), gamma2=1 + 0.1 * rn(D), beta2=0.1 * rn(D),
             W_q=(rn(H * DQ, D) * D ** -0.5).to(kind), bn_gamma=1 + 0.1 * rn(H * DQ),
             bn_beta=0.1 * rn(H * DQ), subkeys=(rn(H, 2, N, DQ // 2) * 0.5).to(kind),
             values=rn(N * N, D).to(kind), W1=(rn(FF, D) * D ** -0.5).to(kind), b1=0.1 * rn(FF),
             W2=(rn(D, FF) * FF ** -0.5).to(kind), b2=0.1 * rn(D))
    bn = dict(mean=0.1 * rn(H * DQ), var=1 + 0.1 * rn(H * DQ).abs())
    return p, bn, rn


class Step:
    """One training step on fixed buffers."""

    def __init__(self, kind, p, bn, x, gy, bits):
        import product_key_memory_b200 as P
        self.P, self.p, self.bn, self.x, self.gy = P, p, bn, x, gy
        self.g = {k: torch.zeros(t.shape, device="cuda") for k, t in p.items()}
        self.state = []
        for k, t in p.items():
            e = dict(param=t, grad=self.g[k], weight_decay=0.01 if t.dim() > 1 else 0.0,
                     **P.alloc_adamw_state(t, bits if t.numel() >= 4096 else 32))
            if t.dtype == BF16:
                e["master"] = t.float()
            self.state.append(e)
        self.list = P.make_adamw_tensors(self.state)
        self.dyn = torch.zeros(3, device="cuda")
        self.kind = kind
        shape = P.make_shape(B, D, H, DQ, N, K, D, kind)
        self.fws = P.alloc_workspace(shape, False, "cuda")
        import ctypes
        nb = int(P.lib().pkm_workspace_size(ctypes.byref(shape), 3))
        self.bws = torch.zeros(nb, dtype=torch.uint8, device="cuda")

    def forward(self):
        P, p = self.P, self.p
        self.n1, _, self.mu1, self.rs1 = P.pkm_layernorm_forward(self.x, p["gamma1"], p["beta1"],
                                                                 eps=EPS)
        self.m, self.idx, self.wt, _ = P.pkm_forward(
            self.n1, p["W_q"], self.bn["mean"], self.bn["var"], p["bn_gamma"], p["bn_beta"],
            p["subkeys"], p["values"], k=K, want_scores=False, workspace=self.fws)
        self.n2, self.h, self.mu2, self.rs2 = P.pkm_layernorm_forward(
            self.x, p["gamma2"], p["beta2"], add=self.m, eps=EPS)
        self.u, self.pre = P.pkm_linear_forward(self.n2, p["W1"], p["b1"], activation="gelu",
                                                want_pre=True)
        self.y, _ = P.pkm_linear_forward(self.u, p["W2"], p["b2"], residual=self.h)
        return self.y

    def backward(self):
        P, p, g = self.P, self.p, self.g
        du = torch.empty_like(self.u)
        P.pkm_linear_backward(self.u, p["W2"], self.gy, dict(x=du, W=g["W2"], bias=g["b2"]))
        dn2 = torch.empty_like(self.n2)
        P.pkm_linear_backward(self.n2, p["W1"], du, dict(x=dn2, W=g["W1"], bias=g["b1"]),
                              pre=self.pre, activation="gelu")
        dh, _, _ = P.pkm_layernorm_backward(dn2, self.h, self.mu2, self.rs2, p["gamma2"],
                                            grad_sum=self.gy, grad_dtype=self.kind,
                                            grad_gamma=g["gamma2"], grad_beta=g["beta2"])
        dn1 = torch.empty(B, D, device="cuda")
        grads = dict(x=dn1, **{k: g[k] for k in ("W_q", "bn_gamma", "bn_beta", "subkeys",
                                                 "values")})
        P.pkm_backward(self.n1, p["W_q"], self.bn["mean"], self.bn["var"], p["bn_gamma"],
                       p["bn_beta"], p["subkeys"], p["values"], self.idx, self.wt, dh, grads,
                       bn_eps=EPS, workspace=self.bws)
        self.dx, _, _ = P.pkm_layernorm_backward(dn1, self.x, self.mu1, self.rs1, p["gamma1"],
                                                 grad_sum=dh, grad_dtype=F32,
                                                 grad_gamma=g["gamma1"], grad_beta=g["beta1"])

    def update(self, t, lr):
        self.P.pkm_adamw_step(self.list, lr=lr, step=t, zero_grad=True, seed=5)


def _reference(s):
    """y, and the gradients of sum(y gy), in 64 bits with the picks of the step's forward."""
    p = {k: t.double().requires_grad_(True) for k, t in s.p.items()}
    x = s.x.double().requires_grad_(True)
    ln = torch.nn.functional.layer_norm
    n1 = ln(x, (D,), p["gamma1"], p["beta1"], EPS)
    q = n1 @ p["W_q"].t()
    q = (q - s.bn["mean"].double()) / (s.bn["var"].double() + EPS).sqrt() * p["bn_gamma"] + p["bn_beta"]
    q = q.view(B, H, 2, DQ // 2)
    idx = s.idx.long()
    heads = torch.arange(H, device="cuda").view(1, H, 1)
    k1 = p["subkeys"][heads, 0, idx // N]
    k2 = p["subkeys"][heads, 1, idx % N]
    score = (q[:, :, 0, None] * k1).sum(-1) + (q[:, :, 1, None] * k2).sum(-1)
    m = (score.softmax(-1)[..., None] * p["values"][idx]).sum((1, 2))
    h = x + m
    n2 = ln(h, (D,), p["gamma2"], p["beta2"], EPS)
    u = torch.nn.functional.gelu(n2 @ p["W1"].t() + p["b1"])
    y = u @ p["W2"].t() + p["b2"] + h
    (y * s.gy.double()).sum().backward()
    return y.detach(), x.grad, {k: t.grad for k, t in p.items()}


@pytest.mark.parametrize("kind,bits", [(F32, 32), (BF16, 32), (BF16, 8)])
def test_steps_of_a_block(kind, bits):
    p, bn, rn = _model(kind)
    s = Step(kind, p, bn, rn(B, D).to(kind), rn(B, D).to(kind), bits)
    tol = 1e-3 if kind == F32 else 11 * 2.0 ** -9
    for t in (1, 2):
        y = s.forward()
        s.backward()
        ry, rdx, rg = _reference(s)
        off = lambda a, r: float((a.double() - r).norm() / r.norm())  # noqa: E731
        assert off(y, ry) <= tol
        assert off(s.dx, rdx) <= tol
        for k, r in rg.items():
            assert off(s.g[k], r) <= tol, k
        hyper = dict(lr=1e-3, step=t, betas=(0.9, 0.999), eps=1e-8, grad_scale=1.0, seed=5)
        want = [adamw(e, hyper, i) for i, e in enumerate(s.state)]
        s.update(t, 1e-3)
        for k, e, w in zip(s.p, s.state, want):
            carrier = e.get("master", e["param"]).flatten()
            if e["param"].dtype == F32 or "master" in e:
                assert_within(k, carrier, w["param"], w["bound"] + half_step(F32) * w["param"].abs())
            if "master" in e:
                assert torch.equal(e["param"], e["master"].to(BF16))
            assert not bool(e["grad"].any()), k


def test_a_captured_step_is_the_eager_one():
    results = []
    for captured in (False, True):
        p, bn, rn = _model(BF16)
        s = Step(BF16, p, bn, rn(B, D).to(BF16), rn(B, D).to(BF16), 8)
        rows = torch.tensor([[1e-3, 1.0, 1.0], [5e-4, 2.0, 1.0], [2e-4, 3.0, 0.5]], device="cuda")

        def step():
            s.forward()
            s.backward()
            s.P.pkm_adamw_step(s.list, lr=0.0, step=1, zero_grad=True, seed=5, dyn=s.dyn)

        if captured:
            before = [{k: v.clone() for k, v in e.items() if torch.is_tensor(v)} for e in s.state]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            s.dyn.copy_(rows[0])
            with torch.cuda.stream(side):
                step()                               # warm-up; its changes are taken back
            torch.cuda.current_stream().wait_stream(side)
            for e, b in zip(s.state, before):
                for k, v in b.items():
                    e[k].copy_(v)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for r in rows:
            s.dyn.copy_(r)
            graph.replay() if captured else step()
        torch.cuda.synchronize()
        results.append((s.p, s.y.clone(), s.dx.clone()))
    (p0, y0, d0), (p1, y1, d1) = results
    assert torch.equal(y0, y1) and torch.equal(d0, d1)
    for k in p0:
        assert torch.equal(p0[k], p1[k]), k
