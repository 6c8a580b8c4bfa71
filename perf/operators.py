"""Operators of the transformer block around a product-key memory layer: what is timed, and the plain
form that the kernels are compared with.

Layer norm with the residual addition before it, the dense (feed-forward) layer with bias, activation
and residual in its epilogue, both with their backward passes, and the AdamW step over a list of
tensors with states in 32 or in 8 bits. Sizes are those of the memory layers this repository runs
(d_model 1024 and 1600, 4096 and 16384 tokens, 512^2 slots) and of a feed-forward layer four times as
wide, with generic odd ones.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
TYPES = {F32: torch.float32, BF16: torch.bfloat16}
LR, BETA1, BETA2, EPS, DECAY, GRAD_SCALE, SEED = 1e-3, 0.9, 0.98, 1e-8, 0.01, 0.5, 1234
BLOCK = 256              # elements that share a scale of 8-bit states
SMALL = 4096             # tensors below this keep 32-bit states
LARGEST_ADAMW = 512 * 512 * 1024
LARGEST_ROWS = 16384 * 1600
LARGEST_PRODUCT = 4096 * 1600 * 6400


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One token being generated: the residual stream in bf16, the memory layer's fp32 output added.
        dict(name="ln_fwd_1_token", op="ln_fwd", rows=1, d=1024, x=BF16, add=F32, y=BF16, stats=False),
        # The 16384-token training batch: fp32 residual stream, bf16 input for the next layer.
        dict(name="ln_fwd_16384x1024", op="ln_fwd", rows=16384, d=1024, x=F32, add=F32, y=BF16, stats=True),
        # The wide model's backward: the memory layer's fp32 input gradient, the bf16 residual stream.
        dict(name="ln_bwd_16384x1600", op="ln_bwd", rows=16384, d=1600, x=BF16, g=F32, add=BF16, gx=BF16),
        # A ragged batch of an odd width, all in fp32, no residual gradient.
        dict(name="ln_bwd_777x1001", op="ln_bwd", rows=777, d=1001, x=F32, g=F32, add="", gx=F32),
        # The whole 512^2 layer: bf16 weights with fp32 masters, gradients cleared for the next step.
        dict(name="adamw32_512_layer", op="adamw", d=1024, H=4, dq=512, n=512, v=1024, vectors=0,
             param=BF16, master=True, grad=F32, bits=32, zero=True),
        # The same layer with 8-bit states and no masters: what a memory-bound training run keeps.
        dict(name="adamw8_512_layer", op="adamw", d=1024, H=4, dq=512, n=512, v=1024, vectors=0,
             param=BF16, master=False, grad=F32, bits=8, zero=False),
        # Only the norms and biases of a 12-block model: many short fp32 tensors.
        dict(name="adamw32_vectors", op="adamw", d=1024, H=0, dq=0, n=0, v=0, vectors=48,
             param=F32, master=False, grad=F32, bits=32, zero=False),
        # One token through the first feed-forward matrix.
        dict(name="linear_fwd_1_token", op="linear_fwd", M=1, K=1024, N=4096, x=BF16, y=BF16, act="gelu",
             bias=True, residual=False, pre=False),
        # The training batch through the first feed-forward matrix; the backward pass wants `pre`.
        dict(name="linear_fwd_16384x4096", op="linear_fwd", M=16384, K=1024, N=4096, x=BF16, y=BF16,
             act="gelu", bias=True, residual=False, pre=True),
        # Odd sizes in fp32 with everything in the epilogue.
        dict(name="linear_fwd_777x515_f32", op="linear_fwd", M=777, K=1001, N=515, x=F32, y=F32, act="silu",
             bias=True, residual=True, pre=False),
        # The wide model's first feed-forward matrix: every gradient.
        dict(name="linear_bwd_4096x6400", op="linear_bwd", M=4096, K=1600, N=6400, x=BF16, gx=BF16, act="gelu",
             bias=True),
        # A ragged batch through the second feed-forward matrix (no activation).
        dict(name="linear_bwd_777x1024", op="linear_bwd", M=777, K=4096, N=1024, x=BF16, gx=F32, act="none",
             bias=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A width: any number in three of ten draws, else a multiple of 8."""
    w = _log(rng, low, high)
    return w if rng.random() < 0.3 else max(8, w // 8 * 8)


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "adamw", "linear_fwd", "linear_bwd"])
    kind = lambda: rng.choice([F32, BF16])  # noqa: E731
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("ln_fwd", "ln_bwd"):
        d = _width(rng, 32, 8192)
        rows = _log(rng, 1, min(32768, LARGEST_ROWS // d))
        add = rng.choice(["", F32, BF16])
        if op == "ln_fwd":
            return dict(op=op, rows=rows, d=d, x=kind(), add=add, y=kind(), stats=flag())
        return dict(op=op, rows=rows, d=d, x=kind(), g=kind(), add=add, gx=kind())
    if op == "adamw":
        n, v = _log(rng, 4, 512), 8 * _log(rng, 4, 128)
        param = kind()
        return dict(op=op, d=_width(rng, 32, 1600), H=rng.randint(1, 4), dq=2 * _log(rng, 4, 256), n=n, v=v,
                    vectors=rng.randint(0, 30), param=param, master=param == BF16 and flag(), grad=kind(),
                    bits=rng.choice([32, 8]), zero=flag())
    K, N = _width(rng, 32, 6400), _width(rng, 32, 6400)
    M = _log(rng, 1, max(1, min(16384, LARGEST_PRODUCT // (2 * K * N))))
    case = dict(op=op, M=M, K=K, N=N, x=kind(), act=rng.choice(["none", "relu", "gelu", "silu"]), bias=flag())
    if op == "linear_fwd":
        return dict(case, y=kind(), residual=flag(), pre=flag())
    return dict(case, gx=kind())


# ------------------------------------------------------------------------------------ inputs
def _tensors(case):
    """(elements, row length, type of the parameter, weight decay) of an AdamW case's tensors."""
    some = []
    if case["n"]:
        F, kind = case["H"] * case["dq"], case["param"]
        some += [(F * case["d"], case["d"], kind, DECAY), (F, F, F32, 0.0), (F, F, F32, 0.0),
                 (F * case["n"], case["dq"] // 2, kind, DECAY), (case["n"] ** 2 * case["v"], case["v"], kind, 0.0)]
    widths = (1, 1, 4, 1)  # a block's norm weight and bias, its two feed-forward biases
    some += [(case["d"] * widths[i % 4], case["d"], F32, 0.0) for i in range(case["vectors"])]
    return some


def _blocks(t):
    """t as rows of BLOCK values, the last row filled up with zeros."""
    short = -t.numel() % BLOCK
    return torch.cat([t, t.new_zeros(short)]).view(-1, BLOCK) if short else t.view(-1, BLOCK)


def _power(exponent):
    """2^exponent in fp32 (exponents of normal numbers), from its bits."""
    return ((exponent.int() + 127) << 23).view(torch.float32)


def _scale(t):
    """The smallest power of two s >= 2^-100 with |t| <= 448 s over each block (NaN if that is not finite)."""
    most = _blocks(t).abs().amax(1)
    mantissa, exponent = torch.frexp(most)                   # most = mantissa 2^exponent, mantissa in [1/2, 1)
    exponent = exponent - 9 + (mantissa > 0.875).int()       # 448 = 0.875 2^9
    s = torch.where(most == 0, torch.full_like(most, 2.0 ** -100), _power(exponent.clamp(min=-100)))
    return torch.where(torch.isfinite(most), s, torch.full_like(s, math.nan))


def _spread(scale, n):
    return scale[:, None].expand(-1, BLOCK).reshape(-1)[:n]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]

    def normal(shape, kind, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(TYPES[kind])

    s = {"case": case}
    if op in ("ln_fwd", "ln_bwd"):
        rows, d = case["rows"], case["d"]
        s["x"] = (torch.randn(rows, d, generator=g, device="cuda") * 1.5 + 0.3).to(TYPES[case["x"]])
        s["gamma"] = 1 + normal(d, F32, 0.2)
        s["beta"] = normal(d, F32, 0.2)
        s["add"] = normal((rows, d), case["add"], 0.5) if case["add"] else None
        if op == "ln_bwd":
            s["g"] = normal((rows, d), case["g"])
            xd = s["x"].double()
            s["mean"] = xd.mean(1).float()
            s["rstd"] = (xd.var(1, unbiased=False) + 1e-5).rsqrt().float()
    elif op == "adamw":
        s["tensors"] = []
        for n, row, kind, decay in _tensors(case):
            # Rows that the batch did not touch have no gradient, as in the memory's value table.
            hit = torch.rand(-(-n // row), generator=g, device="cuda") < 0.7
            grad = (torch.randn(n, generator=g, device="cuda").view(-1, row) * hit[:, None]).view(-1) * 1e-2
            value = torch.randn(n, generator=g, device="cuda") / 16
            m = torch.randn(n, generator=g, device="cuda") * 2e-3
            r = (torch.randn(n, generator=g, device="cuda") * 2e-3 + 4e-3).abs()      # sqrt of the second moment
            t = {"param": value.to(TYPES[kind]), "grad": grad.to(TYPES[case["grad"]]), "decay": decay, "master": None}
            if kind == BF16 and case["master"]:
                t["master"] = value
            if case["bits"] == 8 and n >= SMALL:
                for key, w in (("m", m), ("v", r)):
                    t[key + "_scale"] = _scale(w)
                    t[key] = (w / _spread(t[key + "_scale"], n)).to(torch.float8_e4m3fn)
            else:
                t["m"], t["v"] = m, r * r
            s["tensors"].append(t)
        s["step"] = 1000
    else:
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = normal((M, K), case["x"])
        s["W"] = normal((N, K), case["x"], K ** -0.5)
        s["bias"] = normal(N, F32, 0.1) if case["bias"] else None
        if op == "linear_fwd":
            s["residual"] = normal((M, N), case["y"]) if case["residual"] else None
        else:
            s["pre"] = normal((M, N), case["x"]) if case["act"] != "none" else None
            s["g"] = normal((M, N), case["x"])
            s["grads"] = {"x": torch.empty(M, K, device="cuda", dtype=TYPES[case["gx"]]),
                          "W": torch.empty(N, K, device="cuda")}
            if case["bias"]:
                s["grads"]["bias"] = torch.empty(N, device="cuda")
    if own:  # what a program keeps beside its tensors: the list of parameters, the scratch of its layers
        import product_key_memory_b200 as P
        if op == "adamw":
            s["list"] = P.make_adamw_tensors([
                dict(param=t["param"], grad=t["grad"], master=t["master"], m=t["m"], v=t["v"],
                     m_scale=t.get("m_scale"), v_scale=t.get("v_scale"), weight_decay=t["decay"]) for t in s["tensors"]])
        elif op == "ln_bwd":
            s["workspace"] = P.alloc_norm_workspace(P.make_norm_shape(case["rows"], case["d"]), "cuda")
        elif op != "ln_fwd":
            shape = P.make_linear_shape(M, N, K, TYPES[case["x"]], TYPES[case["y" if op == "linear_fwd" else "gx"]], case["act"])
            s["workspace"] = P.alloc_linear_workspace(shape, op == "linear_bwd", "cuda")
    return s


# ------------------------------------------------------------------------------------ one pass
def _act(t, act):
    if act == "relu":
        return torch.where(t <= 0, torch.zeros_like(t), t)
    if act == "gelu":
        return 0.5 * t * (1 + torch.erf(t * 0.5 ** 0.5))
    if act == "silu":
        return t / (1 + torch.exp(-t))
    return t


def _act_slope(t, act):
    if act == "relu":
        return (t > 0).to(t.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(t * 0.5 ** 0.5)) + t * torch.exp(-0.5 * t * t) * (2 * math.pi) ** -0.5
    s = 1 / (1 + torch.exp(-t))
    return s * (1 + t * (1 - s))


def _mix(h):
    """A 32-bit mixing function (MurmurHash3's finaliser) on numbers held in 64 bits."""
    h = h ^ (h >> 16)
    h = (h * 0x85ebca6b) & 0xffffffff
    h = h ^ (h >> 13)
    h = (h * 0xc2b2ae35) & 0xffffffff
    return h ^ (h >> 16)


def _dither(n, step, index, device, dtype):
    """Element i's offset in (-1/2, 1/2): 16 bits of a hash of its pair, by the call's seed, step and list position."""
    key = _mix((SEED + 0x9e3779b9 * step) & 0xffffffff)
    key = _mix(key ^ (index * 0x9e3779b9 & 0xffffffff))
    h = _mix(torch.arange((n + 1) // 2, device=device) ^ key)
    return (torch.stack([h & 0xffff, h >> 16], 1).view(-1)[:n].to(dtype) - 32767.5) / 65536


def _adamw_plain(t, step, index, zero):
    n = t["param"].numel()
    eight = "m_scale" in t
    lr_over = LR / (1 - BETA1 ** step)
    root = (1 - BETA2 ** step) ** -0.5
    p = t["param"].float() if t["master"] is None else t["master"]
    g = t["grad"].float() * GRAD_SCALE
    m, v = t["m"].float(), t["v"].float()
    if eight:
        m = m * _spread(t["m_scale"], n)
        v = (v * _spread(t["v_scale"], n)).square()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    r = v.sqrt()
    p = p * (1 - LR * t["decay"]) - lr_over * (m / (r * root + EPS))
    if eight:
        t["m_scale"].copy_(_scale(m))
        t["v_scale"].copy_(_scale(r))
        t["m"].copy_((m / _spread(t["m_scale"], n)).to(torch.float8_e4m3fn))
        q = r / _spread(t["v_scale"], n)
        ulp = _power((torch.frexp(q)[1] - 1).clamp(min=-6) - 3)  # e4m3's step at q
        near = q + ulp * _dither(n, step, index, q.device, q.dtype)
        t["v"].copy_(torch.where(q > 0, near.clamp(2.0 ** -9, 448.0), q).to(torch.float8_e4m3fn))
    else:
        t["m"].copy_(m)
        t["v"].copy_(v)
    if t["master"] is not None:
        t["master"].copy_(p)
    t["param"].copy_(p.to(t["param"].dtype))
    if zero:
        t["grad"].zero_()


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "ln_fwd":
        x = s["x"] if s["add"] is None else (s["x"].float() + s["add"].float()).to(s["x"].dtype)
        h = x.float()
        mean = h.mean(1, keepdim=True)
        c = h - mean
        rstd = 1 / (c.square().mean(1, keepdim=True) + 1e-5).sqrt()
        y = (c * rstd * s["gamma"] + s["beta"]).to(TYPES[case["y"]])
        return [y, x if s["add"] is not None else None] + ([mean[:, 0], rstd[:, 0]] if case["stats"] else [])
    if op == "ln_bwd":
        g = s["g"].float()
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        t = g * s["gamma"]
        gx = s["rstd"][:, None] * (t - t.mean(1, keepdim=True) - xhat * (t * xhat).mean(1, keepdim=True))
        if s["add"] is not None:
            gx = gx + s["add"].float()
        return [gx.to(TYPES[case["gx"]]), (g * xhat).sum(0), g.sum(0)]
    if op == "adamw":
        [_adamw_plain(t, s["step"], i, case["zero"]) for i, t in enumerate(s["tensors"])]
        return _adamw_outputs(s)
    x, W = s["x"].float(), s["W"].float()
    if op == "linear_fwd":
        pre = x @ W.t()
        if s["bias"] is not None:
            pre = pre + s["bias"]
        y = _act(pre, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return [y.to(TYPES[case["y"]]), pre.to(s["x"].dtype) if case["pre"] else None]
    t = s["g"].float()
    if s["pre"] is not None:
        t = t * _act_slope(s["pre"].float(), case["act"])
    return [(t @ W).to(TYPES[case["gx"]]), t.t() @ x, t.sum(0) if case["bias"] else None]


def _adamw_outputs(s):
    keys = ("param", "master", "m", "v", "m_scale", "v_scale") + (("grad",) if s["case"]["zero"] else ())
    big = [t for t in s["tensors"] if t["param"].numel() >= SMALL]
    few = (big or s["tensors"])[:5] + (s["tensors"][-1:] if len(s["tensors"]) > 5 else [])
    return [{k: t[k] for k in keys if t.get(k) is not None} for t in few]


def run(state):
    if not own:
        return _run_plain(state)
    import product_key_memory_b200 as P
    s, case = state, state["case"]
    op = case["op"]
    if op == "ln_fwd":
        y, x, mean, rstd = P.pkm_layernorm_forward(s["x"], s["gamma"], s["beta"], add=s["add"], eps=1e-5,
                                                   out_dtype=TYPES[case["y"]], want_stats=case["stats"])
        return [y, x if s["add"] is not None else None] + ([mean, rstd] if case["stats"] else [])
    if op == "ln_bwd":
        return list(P.pkm_layernorm_backward(s["g"], s["x"], s["mean"], s["rstd"], s["gamma"], grad_sum=s["add"],
                                             grad_dtype=TYPES[case["gx"]], workspace=s["workspace"]))
    if op == "adamw":
        P.pkm_adamw_step(s["list"], lr=LR, step=s["step"], betas=(BETA1, BETA2), eps=EPS, grad_scale=GRAD_SCALE,
                         zero_grad=case["zero"], seed=SEED)
        return _adamw_outputs(s)
    if op == "linear_fwd":
        y, pre = P.pkm_linear_forward(s["x"], s["W"], bias=s["bias"], residual=s["residual"], activation=case["act"],
                                      out_dtype=TYPES[case["y"]], want_pre=case["pre"], workspace=s["workspace"])
        return [y, pre]
    P.pkm_linear_backward(s["x"], s["W"], s["g"], s["grads"], pre=s["pre"], activation=case["act"],
                          workspace=s["workspace"])
    return [s["grads"]["x"], s["grads"]["W"], s["grads"].get("bias")]


# ------------------------------------------------------------------------------------ work
def work(case):
    size = lambda kind: {F32: 4, BF16: 2}.get(kind, 0)  # noqa: E731
    op = case["op"]
    if op == "ln_fwd":
        n = case["rows"] * case["d"]
        each = size(case["x"]) + size(case["add"]) + size(case["y"]) + (size(case["x"]) if case["add"] else 0)
        return {"bytes": n * each + 8 * case["d"] + (8 * case["rows"] if case["stats"] else 0), "flops": 8 * n}
    if op == "ln_bwd":
        n = case["rows"] * case["d"]
        each = size(case["x"]) + size(case["g"]) + size(case["add"]) + size(case["gx"])
        return {"bytes": n * each + 12 * case["d"] + 8 * case["rows"], "flops": 14 * n}
    if op == "adamw":
        total = flops = 0
        for n, _, kind, _ in _tensors(case):
            master = kind == BF16 and case["master"]
            each = size(kind) * (1 if master else 2) + (8 if master else 0)
            each += size(case["grad"]) * (2 if case["zero"] else 1)
            each += 4 + 16 / BLOCK if case["bits"] == 8 and n >= SMALL else 16
            total += n * each
            flops += 16 * n
        return {"bytes": total, "flops": flops}
    M, K, N, e = case["M"], case["K"], case["N"], size(case["x"])
    if op == "linear_fwd":
        out = size(case["y"]) * (2 if case["residual"] else 1) + (e if case["pre"] else 0)
        return {"bytes": e * (M * K + N * K) + M * N * out + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    read = e * (M * K + N * K + M * N * (1 if case["act"] == "none" else 2))
    return {"bytes": read + size(case["gx"]) * M * K + 4 * N * K + (4 * N if case["bias"] else 0), "flops": 4 * M * N * K}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    def adamw(t, step, index, zero):
        n, out = t["param"].numel(), {}
        eight = "m_scale" in t
        read = lambda k: t[k].double() * _spread(t[k + "_scale"].double(), n) if eight else t[k].double()  # noqa: E731
        g = t["grad"].double() * GRAD_SCALE
        m = BETA1 * read("m") + (1 - BETA1) * g
        v = read("v").square() if eight else read("v")
        v = BETA2 * v + (1 - BETA2) * g.square()
        p = (t["param"] if t["master"] is None else t["master"]).double()
        out["param"] = p - LR * t["decay"] * p - LR / (1 - BETA1 ** step) * m / (v.sqrt() / math.sqrt(1 - BETA2 ** step) + EPS)
        if t["master"] is not None:
            out["master"] = out["param"]
        if eight:
            for key, w in (("m", m), ("v", v.sqrt())):
                exponent = torch.ceil(torch.log2(_blocks(w).abs().amax(1) / 448)).clamp(min=-100)
                out[key + "_scale"] = torch.exp2(exponent)
                q = w / _spread(out[key + "_scale"], n)
                at = torch.exp2(torch.floor(torch.log2(q.abs())).clamp(min=-6) - 3)
                if key == "v":
                    near = torch.round(q / at + _dither(n, step, index, q.device, q.dtype)) * at
                    out[key] = torch.where(q > 0, near.clamp(2.0 ** -9, 448.0), q)
                else:
                    out[key] = torch.round(q / at) * at
        else:
            out["m"], out["v"] = m, v
        if zero:
            out["grad"] = torch.zeros_like(g)
        return out

    s = prepare(case, seed)
    op = case["op"]
    if op == "ln_fwd":
        x = s["x"] if s["add"] is None else (s["x"].float() + s["add"].float()).to(s["x"].dtype)
        h = x.double()
        var, mean = torch.var_mean(h, 1, unbiased=False, keepdim=True)
        rstd = (var + 1e-5).rsqrt()
        y = (h - mean) * rstd * s["gamma"].double() + s["beta"].double()
        return [y, x.double() if s["add"] is not None else None] + ([mean[:, 0], rstd[:, 0]] if case["stats"] else [])
    if op == "ln_bwd":
        g, r = s["g"].double(), s["rstd"].double()[:, None]
        xhat = (s["x"].double() - s["mean"].double()[:, None]) * r
        t = g * s["gamma"].double()
        gx = r * (t - t.mean(1, keepdim=True)) - r * xhat * (t * xhat).mean(1, keepdim=True)
        if s["add"] is not None:
            gx = gx + s["add"].double()
        return [gx, torch.einsum("rd,rd->d", g, xhat), g.sum(0)]
    if op == "adamw":
        big = [i for i, t in enumerate(s["tensors"]) if t["param"].numel() >= SMALL]
        few = (big or list(range(len(s["tensors"]))))[:5] + ([len(s["tensors"]) - 1] if len(s["tensors"]) > 5 else [])
        return [adamw(s["tensors"][i], s["step"], i, case["zero"]) for i in few]
    x, W = s["x"].double(), s["W"].double()
    if op == "linear_fwd":
        pre = torch.einsum("mk,nk->mn", x, W)
        if s["bias"] is not None:
            pre = pre + s["bias"].double()
        y = {"none": lambda t: t, "relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t),
             "gelu": lambda t: t * 0.5 * torch.erfc(-t / math.sqrt(2))}[case["act"]](pre)
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return [y, pre if case["pre"] else None]
    t = s["g"].double()
    if s["pre"] is not None:
        a = s["pre"].double()
        t = t * {"relu": lambda: (a > 0).double(), "silu": lambda: torch.sigmoid(a) * (1 + a * torch.sigmoid(-a)),
                 "gelu": lambda: 0.5 * torch.erfc(-a / math.sqrt(2)) + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)}[case["act"]]()
    return [torch.einsum("mn,nk->mk", t, W), torch.einsum("mn,mk->nk", t, x), t.sum(0) if case["bias"] else None]
