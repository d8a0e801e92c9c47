"""Cases that time the operators of the expert block's training step: grouped
matrix products with ragged groups (forward, input gradient, weight gradient),
the experts' SwiGLU with its 8-bit checkpoint, and the norms' passes.

``run`` computes an operator in elementary fp32 torch operations, or, with
``own`` set, calls the framework's entry point on the same state.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 32            # columns of gate_up that share one checkpoint scale
EPS = 1e-6


def listed():
    return [
        # gate_up of one decoded token: 6 of 64 experts, one row each (latency, weights streamed)
        dict(name="forward-one-token", op="matmul", form="forward", rows=6, E=64, n=2048, k=2048,
             dtype="bf16", out="bf16", skew="spread", pad=0.0),
        # gate_up of a training step of the 64-expert layer (T=4096, top 6)
        dict(name="forward-train", op="matmul", form="forward", rows=24576, E=64, n=2048, k=2048,
             dtype="bf16", out="bf16", skew="even", pad=0.0),
        # down product of the 256-expert layer (T=16384, top 8) under skewed routing with padded
        # tokens; fp32 rows, as moe_combine takes them
        dict(name="forward-skewed-f32", op="matmul", form="forward", rows=131072, E=256, n=6144,
             k=1024, dtype="bf16", out="f32", skew="zipf", pad=0.02),
        # gradient of gate_up's input in the 128-expert layer (T=8192, top 8): the largest product;
        # fp32 rows, summed per token by moe_combine
        dict(name="dgrad-large", op="matmul", form="dgrad", rows=65536, E=128, n=4096, k=6144,
             dtype="bf16", out="f32", skew="even", pad=0.0),
        # a small fp16 batch with sizes off every tile boundary
        dict(name="dgrad-odd-f16", op="matmul", form="dgrad", rows=777, E=16, n=1416, k=2040,
             dtype="f16", out="f16", skew="zipf", pad=0.1),
        # gate_up's weight gradient in the 64-expert training step
        dict(name="wgrad-train", op="matmul", form="wgrad", rows=24576, E=64, n=2048, k=2048,
             dtype="bf16", out="bf16", skew="even", pad=0.0),
        # a micro-batch added to the fp32 weight gradient of 24 wide experts (T=2048, top 3)
        dict(name="wgrad-accumulate", op="matmul", form="wgrad", rows=6144, E=24, n=4096, k=6144,
             dtype="bf16", out="f32", skew="zipf", pad=0.0),
        # activation and checkpoint of the 128-expert layer (T=8192, top 8)
        dict(name="swiglu-save", op="swiglu", form="forward", rows=65536, I=2048, dtype="bf16",
             pad=0.01),
        # its backward pass from the checkpoint
        dict(name="swiglu-backward", op="swiglu", form="backward", rows=65536, I=2048,
             dtype="bf16", pad=0.01),
        # layer norm of a small decoding batch (latency)
        dict(name="layer-norm-few-rows", op="norm", form="forward", kind="layer", T=32, H=6144,
             dtype="bf16", residual=False),
        # layer norm's gradients in the 64-expert training step
        dict(name="layer-norm-backward", op="norm", form="backward", kind="layer", T=4096, H=2048,
             dtype="bf16", residual=False),
        # the block norm's gradients in the 128-expert layer, the residual's gradient added
        dict(name="rms-norm-backward", op="norm", form="backward", kind="rms", T=8192, H=6144,
             dtype="bf16", residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "swiglu", "norm"])
    if op == "matmul":
        form = rng.choice(["forward", "dgrad", "wgrad"])
        E = _log(rng, 1, 256)
        n, k = 8 * _log(rng, 8, 768), 8 * _log(rng, 8, 768)
        while E * n * k > 2 ** 30:
            E = max(1, E // 2)
        rows = _log(rng, 1, 65536)
        while rows * n * k > 2 ** 40:
            rows //= 2
        dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
        if dtype == "f32":
            rows = min(rows, 2048)     # fp32 products run on the CUDA cores: small layers
            n, k = min(n, 1024), min(k, 1024)
        return dict(op=op, form=form, rows=rows, E=E, n=n, k=k, dtype=dtype,
                    out=rng.choice([dtype, "f32"]), skew=rng.choice(["even", "zipf", "spread", "one"]),
                    pad=rng.choice([0.0, 0.0, rng.uniform(0, 0.3)]))
    if op == "swiglu":
        I = 16 * _log(rng, 2, 512)
        return dict(op=op, form=rng.choice(["forward", "backward"]), I=I,
                    rows=_log(rng, 1, min(131072, 2 ** 27 // I)), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    pad=rng.choice([0.0, rng.uniform(0, 0.3)]))
    H = _log(rng, 32, 8192)
    if rng.random() < 0.75:
        H = (H + 7) // 8 * 8
    kind = rng.choice(["layer", "layer", "rms"])
    form = "backward" if kind == "rms" else rng.choice(["forward", "backward"])
    return dict(op=op, form=form, kind=kind, T=_log(rng, 1, min(65536, 48 * 2 ** 20 // H)), H=H,
                dtype=rng.choice(["bf16", "bf16", "f32"]),
                residual=form == "backward" and rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _sizes(case, rs):
    """Rows of each expert: `live` rows dealt to E experts."""
    E, live = case["E"], case["rows"] - int(case["rows"] * case["pad"])
    if case["skew"] == "one":              # every row to one expert
        sizes = np.zeros(E, dtype=np.int64)
        sizes[rs.randint(E)] = live
    elif case["skew"] == "spread":         # as far apart as can be: a token's top-k
        sizes = np.full(E, live // E, dtype=np.int64)
        sizes[rs.permutation(E)[: live % E]] += 1
    else:
        p = np.ones(E) if case["skew"] == "even" else rs.permutation(1.0 / np.arange(1, E + 1))
        sizes = rs.multinomial(live, p / p.sum())
    return [int(v) for v in sizes]


def _randn(shape, dtype, gen, scale=1.0):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen).mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rs = np.random.RandomState(seed % (2 ** 31))
    t = DT[case["dtype"]]
    s = {"case": dict(case)}
    if case["op"] == "matmul":
        E, n, k, R = case["E"], case["n"], case["k"], case["rows"]
        o = DT[case["out"]]
        s["sizes"] = _sizes(case, rs)
        s["offsets"] = torch.tensor([0] + list(np.cumsum(s["sizes"])), dtype=torch.int32, device="cuda")
        if case["form"] == "forward":
            s["a"], s["w"] = _randn((R, k), t, gen), _randn((E, n, k), t, gen, 0.02)
            s["out"] = torch.zeros((R, n), dtype=o, device="cuda")
        elif case["form"] == "dgrad":
            s["dout"], s["w"] = _randn((R, n), t, gen, 0.1), _randn((E, n, k), t, gen, 0.02)
            s["out"] = torch.zeros((R, k), dtype=o, device="cuda")
        else:
            s["dout"], s["a"] = _randn((R, n), t, gen, 0.1), _randn((R, k), t, gen)
            # fp32 weight gradients are accumulated over micro-batches
            s["accumulate"] = case["out"] == "f32"
            s["out"] = _randn((E, n, k), o, gen) if s["accumulate"] else torch.zeros((E, n, k), dtype=o, device="cuda")
        if own:
            import mixture_experts_feed_b200 as moe
            s["G"] = moe.GroupedMatmul(R, E, n, k, t, o)
            s["ws"] = moe.new_grouped_workspace(s["G"])
    elif case["op"] == "swiglu":
        R, I = case["rows"], case["I"]
        live = R - int(R * case["pad"])
        s["live"] = live
        s["offsets"] = torch.tensor([0, live // 3, live], dtype=torch.int32, device="cuda")
        s["perm_slot"] = torch.randperm(R, generator=gen, device="cuda").to(torch.int32)
        s["topk_w"] = torch.rand(R, generator=gen, device="cuda") * 2.0
        gu = _randn((R, 2 * I), t, gen)
        # channels of unlike scale, as trained projections have them
        gu.mul_(torch.exp(torch.randn(2 * I, generator=gen, device="cuda")).to(t))
        if case["form"] == "forward":
            s["gu"] = gu
            s["h"] = torch.zeros((R, I), dtype=t, device="cuda")
            s["q"] = torch.zeros((R, 2 * I), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            s["scale"] = torch.zeros((R, 2 * I // BLOCK), dtype=torch.uint8, device="cuda")
        else:
            s["q"], s["scale"] = _quantise(gu)
            s["dh"] = _randn((R, I), t, gen, 0.1)
            s["dgu"] = torch.zeros((R, 2 * I), dtype=t, device="cuda")
            s["h"] = torch.zeros((R, I), dtype=t, device="cuda")
            s["dw"] = torch.zeros(R, device="cuda")
        if own:
            import mixture_experts_feed_b200 as moe
            s["ws"] = moe.new_status_workspace()
    else:
        T, H = case["T"], case["H"]
        s["x"] = _randn((T, H), t, gen).add_(0.25)
        s["weight"] = _randn((H,), t, gen, 0.1).add_(1.0)
        s["bias"] = _randn((H,), t, gen, 0.1) if case["kind"] == "layer" else None
        s["out"] = torch.zeros((T, H), dtype=t, device="cuda")
        if case["form"] == "backward":
            s["dout"] = _randn((T, H), t, gen, 0.1)
            s["dres"] = _randn((T, H), t, gen, 0.1) if case["residual"] else None
            s["dweight"] = torch.zeros(H, device="cuda")
            s["dbias"] = torch.zeros(H, device="cuda") if case["kind"] == "layer" else None
            if own:
                import mixture_experts_feed_b200 as moe
                s["ws"] = moe.new_norm_workspace(T, H)
    return s


# ------------------------------------------------------- the operators' calls
def _run_own(s):
    import mixture_experts_feed_b200 as moe
    case = s["case"]
    op, form = case["op"], case["form"]
    if op == "matmul":
        if form == "forward":
            moe.moe_grouped_matmul(s["G"], s["a"], s["w"], s["offsets"], s["out"], s["ws"])
        elif form == "dgrad":
            moe.moe_grouped_matmul_dgrad(s["G"], s["dout"], s["w"], s["offsets"], s["out"], s["ws"])
        else:
            moe.moe_grouped_matmul_wgrad(s["G"], s["dout"], s["a"], s["offsets"], s["out"], s["ws"],
                                         accumulate=s["accumulate"])
        return s["out"]
    if op == "swiglu":
        if form == "forward":
            moe.moe_swiglu_checkpoint(s["gu"], s["offsets"], s["perm_slot"], s["topk_w"], s["h"],
                                      s["q"], s["scale"], s["ws"])
            return {"h": s["h"], "q": s["q"], "scale": s["scale"]}
        moe.moe_swiglu_backward(s["q"], s["scale"], s["dh"], s["offsets"], s["perm_slot"], s["topk_w"],
                                s["dgu"], s["dw"], s["h"], s["ws"])
        return {"dgu": s["dgu"], "dw": s["dw"], "h": s["h"]}
    if form == "forward":
        moe.moe_layer_norm(s["x"], s["weight"], s["bias"], s["out"], EPS)
        return s["out"]
    if case["kind"] == "layer":
        moe.moe_layer_norm_backward(s["x"], s["weight"], s["dout"], s["out"], s["dweight"], s["dbias"],
                                    s["ws"], EPS, dres=s["dres"])
        return {"dx": s["out"], "dweight": s["dweight"], "dbias": s["dbias"]}
    moe.moe_rmsnorm_backward(s["x"], s["weight"], s["dout"], s["out"], s["dweight"], s["ws"], EPS,
                             dres=s["dres"])
    return {"dx": s["out"], "dweight": s["dweight"]}


# ------------------------------------------------------------- plain forms
def _quantise(x):
    """e4m3 values and exponent bytes (2^(b - 127)) of blocks of 32 columns."""
    R, C = x.shape
    v = x.float().view(R, C // BLOCK, BLOCK)
    fine = torch.isfinite(v)
    amax = torch.where(fine, v, 0.0).abs().amax(-1)
    m, e = torch.frexp(amax)                        # amax = m 2^e, m in [0.5, 1)
    # the least exponent with amax / 2^b <= 448 = 0.875 * 2^9
    b = torch.where(m <= 0.875, e - 9, e - 8)
    b = torch.where(amax > 0, b, -127).clamp(-127, 127).to(torch.int32)
    q = torch.where(fine, torch.ldexp(v, -b[..., None]), float("nan"))
    return q.view(R, C).to(torch.float8_e4m3fn), (b + 127).to(torch.uint8)


def _dequantise(q, scale, t):
    R, C = q.shape
    e = scale.to(torch.int32) - 127
    return torch.ldexp(q.to(t).view(R, C // BLOCK, BLOCK), e[..., None]).view(R, C)


def _plain_matmul(s):
    case, at, out = s["case"], 0, s["out"]
    for e, m in enumerate(s["sizes"]):
        rows = slice(at, at + m)
        at += m
        if case["form"] == "wgrad":
            if m == 0 and s["accumulate"]:
                continue
            d = s["dout"][rows].float().t() @ s["a"][rows].float()
            out[e] = (d + out[e]) if s["accumulate"] else d
        elif m > 0:
            w = s["w"][e].float()
            out[rows] = (s["a"][rows].float() @ w.t()) if case["form"] == "forward" else (s["dout"][rows].float() @ w)
    return out


def _plain_swiglu(s):
    live, t = s["live"], DT[s["case"]["dtype"]]
    slot = s["perm_slot"][:live].long()
    w = s["topk_w"][slot][:, None]
    if s["case"]["form"] == "forward":
        gu = s["gu"][:live]
        g, u = gu[:, ::2].float(), gu[:, 1::2].float()
        s["h"][:live] = (w * (g / (1 + torch.exp(-g))) * u).to(t)
        s["q"][:live], s["scale"][:live] = _quantise(gu)
        return {"h": s["h"], "q": s["q"], "scale": s["scale"]}
    gu = _dequantise(s["q"][:live], s["scale"][:live], torch.float32)
    g, u, dh = gu[:, ::2], gu[:, 1::2], s["dh"][:live].float()
    sg = 1 / (1 + torch.exp(-g))
    a = g * sg
    s["dgu"][:live, ::2] = (w * dh * u * sg * (1 + g * (1 - sg))).to(t)
    s["dgu"][:live, 1::2] = (w * dh * a).to(t)
    s["h"][:live] = (w * a * u).to(t)
    s["dw"].zero_()
    s["dw"][slot] = (dh * a * u).sum(1)
    return {"dgu": s["dgu"], "dw": s["dw"], "h": s["h"]}


def _norm(x, kind):
    xc = x - x.mean(1, keepdim=True) if kind == "layer" else x
    r = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    return xc * r, r


def _plain_norm(s):
    case, t = s["case"], DT[s["case"]["dtype"]]
    w = s["weight"].float()
    xh, r = _norm(s["x"].float(), case["kind"])
    if case["form"] == "forward":
        s["out"].copy_((xh * w + s["bias"].float()).to(t))
        return s["out"]
    dout = s["dout"].float()
    gy = dout * w
    dx = gy - xh * (gy * xh).mean(1, keepdim=True)
    if case["kind"] == "layer":
        dx = dx - gy.mean(1, keepdim=True)
        s["dbias"].copy_(dout.sum(0))
    dx = dx * r
    if case["residual"]:
        dx = dx + s["dres"].float()
    s["out"].copy_(dx.to(t))
    s["dweight"].copy_((dout * xh).sum(0))
    r = {"dx": s["out"], "dweight": s["dweight"]}
    return dict(r, dbias=s["dbias"]) if case["kind"] == "layer" else r


def run(state):
    if own:
        return _run_own(state)
    return {"matmul": _plain_matmul, "swiglu": _plain_swiglu, "norm": _plain_norm}[state["case"]["op"]](state)


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    el = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] == "matmul":
        b, o = el[case["dtype"]], el[case["out"]]
        E, n, k = case["E"], case["n"], case["k"]
        live = case["rows"] - int(case["rows"] * case["pad"])
        # experts that can have rows: their weights have to be read
        used = 1 if case["skew"] == "one" else min(E, live)
        if case["form"] == "wgrad":
            byts = b * live * (n + k) + o * (2 * used if case["out"] == "f32" else E) * n * k
        else:
            byts = b * live * (k if case["form"] == "forward" else n) + b * used * n * k + \
                o * live * (n if case["form"] == "forward" else k)
        return {"bytes": byts + 4 * (E + 1), "flops": 2 * live * n * k}
    b = el[case["dtype"]]
    if case["op"] == "swiglu":
        I = case["I"]
        live = case["rows"] - int(case["rows"] * case["pad"])
        ckpt = 2 * I + 2 * I // BLOCK
        if case["form"] == "forward":
            return {"bytes": live * (2 * I * b + I * b + ckpt + 8), "flops": 12 * live * I}
        return {"bytes": live * (ckpt + I * b + 2 * I * b + I * b + 12), "flops": 24 * live * I}
    T, H = case["T"], case["H"]
    if case["form"] == "forward":
        return {"bytes": b * (2 * T * H + 2 * H), "flops": 8 * T * H}
    grads = 2 if case["kind"] == "layer" else 1
    return {"bytes": b * ((4 if case["residual"] else 3) * T * H + H) + 4 * grads * H, "flops": 16 * T * H}


# --------------------------------------------------- the definitions in fp64
def _exact_matmul(case, s):
    off = s["offsets"].tolist()
    res = s["out"].double()
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if case["form"] == "forward":
            res[lo:hi] = torch.einsum("rk,nk->rn", s["a"][lo:hi].double(), s["w"][e].double())
        elif case["form"] == "dgrad":
            res[lo:hi] = torch.einsum("rn,nk->rk", s["dout"][lo:hi].double(), s["w"][e].double())
        else:
            d = torch.einsum("rn,rk->nk", s["dout"][lo:hi].double(), s["a"][lo:hi].double())
            res[e] = res[e] + d if s["accumulate"] else d
    return res


def _exact_swiglu(case, s):
    R, I, live = case["rows"], case["I"], s["live"]
    w = s["topk_w"].double()[s["perm_slot"].long()]
    w[live:] = 0
    if case["form"] == "forward":
        x = s["gu"].double().reshape(R, I, 2)
        h = w[:, None] * x[..., 0] * torch.sigmoid(x[..., 0]) * x[..., 1]
        h[live:] = 0
        # the exponent of a block by search over its candidates, not by its bits
        blocks = s["gu"].double().reshape(R, 2 * I // BLOCK, BLOCK)
        top = blocks.abs().amax(-1)
        e = torch.where(top > 0, torch.ceil(torch.log2(top / 448.0)), -127.0).clamp(-127, 127)
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
        e = torch.where((top <= 448.0 * torch.exp2(e - 1)) & (e > -127), e - 1, e)
        y = blocks / torch.exp2(e)[..., None]
        # e4m3: 3 fraction bits down to 2^-6, then steps of 2^-9
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        q = (torch.round(y / step) * step).reshape(R, 2 * I)
        q[live:] = 0
        return {"h": h, "q": q, "scale": None}
    gu = s["q"].double().reshape(R, -1, BLOCK) * torch.exp2(s["scale"].double() - 127)[..., None]
    gu = gu.reshape(R, I, 2).detach().requires_grad_(True)
    wv = w.clone().requires_grad_(True)
    dh = s["dh"].double()
    with torch.enable_grad():
        h = wv[:, None] * gu[..., 0] * torch.sigmoid(gu[..., 0]) * gu[..., 1]
    dgu, dwr = torch.autograd.grad(h, (gu, wv), dh)
    h, dgu = h.detach(), dgu.reshape(R, 2 * I)
    dgu[live:] = 0
    dw = torch.zeros_like(dwr)
    dw[s["perm_slot"][:live].long()] = dwr[:live]
    return {"dgu": dgu, "dw": dw, "h": h}


def _exact_norm(case, s):
    x = s["x"].double().requires_grad_(True)
    w = s["weight"].double().requires_grad_(True)
    b = s["bias"].double().requires_grad_(True) if case["kind"] == "layer" else None
    with torch.enable_grad():
        if b is not None:
            var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
            y = (x - mean) * torch.rsqrt(var + EPS) * w + b
        else:
            y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w
    if case["form"] == "forward":
        return y.detach()
    got = torch.autograd.grad(y, [x, w] + ([b] if b is not None else []), s["dout"].double())
    dx = got[0] + s["dres"].double() if s["dres"] is not None else got[0]
    r = {"dx": dx, "dweight": got[1]}
    return dict(r, dbias=got[2]) if b is not None else r


def exact(case, seed):
    s = prepare(case, seed)
    return {"matmul": _exact_matmul, "swiglu": _exact_swiglu, "norm": _exact_norm}[case["op"]](case, s)
