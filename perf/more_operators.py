"""Measured cases of the operators of a pre-norm gated feed-forward block.

Five operators: the root-mean-square norm with the residual's addition
(``norm``; optionally as E4M3 codes with scales), its gradient
(``norm_backward``), the gated feed-forward block (``ffn``), its gradient
(``ffn_backward``), and clipping by the global norm of many gradients
(``clip``). With ``own`` false, ``run`` computes them with elementary torch
operations in 32 bits; with ``own`` true it calls the library.

Definitions (T tokens of width d; w the norm's weight):

    s = x + residual                      (returned in the residual's type)
    rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
    scale = max|y| / 448 over a token or a block of 128 channels (1 for
    zeros),  code = E4M3(y (1 / scale))
    backward, from the s that was returned: a = dy w, n = s rstd,
    dx = d_sum + rstd (a - n mean(a n)),  dw = sum_t dy n

    gate = x Wg^T,  up = x Wu^T,  h = silu(gate) up,  y = h Wd^T
    backward, from the gate and up that were returned: dh = dy Wd,
    dg = dh up silu'(gate),  du = dh silu(gate),  dx = dg Wg + du Wu,
    dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h

    norm = sqrt(sum over all tensors of g^2)
    out = g min(1, max_norm / (norm + 1e-6))
"""
import math

import torch

own = False

EPS = 1e-6
CLIP_EPS = 1e-6
E4M3_MAX = 448.0
BLOCK = 128

# The largest listed case of each kind bounds the drawn ones.
MOST_NORM = 16384 * 6656
MOST_FFN = 4.4e12
MOST_CLIP = 340_000_000


def listed():
    return [
        # one token of a decode step on a 32-bit residual stream: nothing but latency
        dict(name="norm_token", op="norm", T=1, d=8704, x="bfloat16", residual="float32", codes=""),
        # the layer's full batch in front of an 8-bit product: a scale for each 128 channels
        dict(name="norm_blocks", op="norm", T=16384, d=6656, x="bfloat16", residual="bfloat16", codes="block"),
        # the mid layer's batch in training, the stream in bf16
        dict(name="norm_backward_mid", op="norm_backward", T=4096, d=2048, dy="bfloat16", stream="bfloat16", d_sum=True),
        # the full batch, the stream and its gradient in 32 bits
        dict(name="norm_backward_wide", op="norm_backward", T=8192, d=6656, dy="bfloat16", stream="float32", d_sum=True),
        # one token through the shared expert: all of its weights for one row
        dict(name="ffn_token", op="ffn", T=1, d=8704, F=10240, save=False),
        # a small batch of decoding sequences, not a power of two
        dict(name="ffn_batch", op="ffn", T=27, d=8704, F=10240, save=False),
        # the mid layer's widths in training: gate and up are kept for the backward pass
        dict(name="ffn_mid", op="ffn", T=4096, d=2048, F=2048, save=True),
        # the shared expert over a whole batch of the widest layer
        dict(name="ffn_shared", op="ffn", T=8192, d=8704, F=10240, save=True),
        # a ragged batch and widths that no tile divides
        dict(name="ffn_backward_odd", op="ffn_backward", T=777, d=1336, F=2040),
        # the shared expert's backward pass
        dict(name="ffn_backward_shared", op="ffn_backward", T=4096, d=8704, F=10240),
        # the tiny layer's gradients, 32 bits and odd ones among them: latency
        dict(name="clip_tiny", op="clip", tensors=14, n=600_000, types="mixed", over=2.0),
        # the mid layer's gradients: a few very large tensors and some small ones
        dict(name="clip_layer", op="clip", tensors=8, n=330_000_000, types="bfloat16", over=3.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "ffn", "ffn_backward", "clip"])
    if op in ("norm", "norm_backward"):
        d = _log_int(rng, 100, 10240)
        if rng.random() < 0.7:
            d = max(128, d // 128 * 128)
        T = max(1, min(_log_int(rng, 1, 65536), MOST_NORM // (2 * d)))
        if op == "norm":
            x = rng.choice(["bfloat16", "bfloat16", "float32"])
            r = rng.choice(["", "float32"] if x == "float32" else ["", "bfloat16", "float32"])
            return dict(op=op, T=T, d=d, x=x, residual=r, codes=rng.choice(["", "", "token", "block"]))
        return dict(op=op, T=T, d=d, dy=rng.choice(["bfloat16", "float32"]), stream=rng.choice(["bfloat16", "float32"]),
                    d_sum=rng.random() < 0.7)
    if op in ("ffn", "ffn_backward"):
        per = 6.0 if op == "ffn" else 12.0
        d, F = 8 * _log_int(rng, 16, 1088), 8 * _log_int(rng, 16, 1280)
        T = max(1, min(_log_int(rng, 1, 16384), int(MOST_FFN / (per * d * F))))
        return dict(op=op, T=T, d=d, F=F, save=rng.random() < 0.5) if op == "ffn" else dict(op=op, T=T, d=d, F=F)
    return dict(op=op, tensors=rng.randint(1, 40), n=_log_int(rng, 1000, MOST_CLIP), types=rng.choice(["mixed", "bfloat16", "float32"]),
                over=rng.choice([0.5, 1.5, 30.0]))


_SIZE = {"bfloat16": 2, "float32": 4, "": 0}


def work(case):
    op = case["op"]
    if op == "norm":
        n, res = case["T"] * case["d"], _SIZE[case["residual"]]
        out = 1 if case["codes"] else _SIZE[case["x"]]
        scales = 0 if not case["codes"] else 4 * case["T"] * (1 if case["codes"] == "token" else -(-case["d"] // BLOCK))
        return {"bytes": n * (_SIZE[case["x"]] + 2 * res + out) + scales + 4 * case["T"] + 2 * case["d"], "flops": 5.0 * n}
    if op == "norm_backward":
        n, st = case["T"] * case["d"], _SIZE[case["stream"]]
        return {"bytes": n * (_SIZE[case["dy"]] + st * (3 if case["d_sum"] else 2)) + 4 * case["T"] + 6 * case["d"], "flops": 9.0 * n}
    if op == "clip":
        b = sum(n * _SIZE[t] for n, t in _clip_shapes(case))
        return {"bytes": 2 * b + 4, "flops": 3.0 * case["n"]}
    T, d, F = case["T"], case["d"], case["F"]
    if op == "ffn":
        return {"bytes": 2 * (3 * d * F + 2 * T * d + (2 * T * F if case["save"] else 0)), "flops": 6.0 * T * d * F}
    return {"bytes": 2 * (6 * d * F + 3 * T * d + 2 * T * F), "flops": 12.0 * T * d * F}


def _clip_shapes(case):
    """Sizes and types of the gradients: each about half of what is left, as a model has a few large tensors and many small ones."""
    left, got, many = case["n"], [], case["tensors"]
    for i in range(many):
        n = left if i == many - 1 else max(1, left // 2 + (i % 3))
        n = min(n, left)
        t = case["types"] if case["types"] != "mixed" else ("bfloat16", "float32")[i % 2]
        got.append((n, t))
        left -= n
        if left <= 0:
            break
    return got


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6007 + 29)
    return g


def _randn(shape, gen, dtype, scale=1.0):
    t = torch.randn(shape, generator=gen, device="cuda")
    return t.mul_(scale).to(dtype) if scale != 1.0 else t.to(dtype)


def prepare(case, seed):
    gen = _generator(seed)
    st = dict(case)
    op, bf16 = case["op"], torch.bfloat16
    if op in ("norm", "norm_backward"):
        T, d = case["T"], case["d"]
        # a trained norm's weights lie around 1
        st["weight"] = (1.0 + 0.2 * torch.randn((d,), generator=gen, device="cuda")).to(bf16)
        # some channels of a residual stream are far stronger than the others
        strong = torch.exp(0.7 * torch.randn((d,), generator=gen, device="cuda"))
        if op == "norm":
            st["xs"] = _randn((T, d), gen, getattr(torch, case["x"]))
            st["res"] = (_randn((T, d), gen, torch.float32) * strong).to(getattr(torch, case["residual"])) if case["residual"] else None
            return st
        stream = getattr(torch, case["stream"])
        st["s"] = (_randn((T, d), gen, torch.float32) * strong).to(stream)
        st["rstd"] = torch.rsqrt(st["s"].float().square().mean(1) + EPS)  # what the forward pass left behind
        st["dys"] = _randn((T, d), gen, getattr(torch, case["dy"]), 1e-3)
        st["ds"] = _randn((T, d), gen, stream, 1e-3) if case["d_sum"] else None
        return st
    if op == "clip":
        st["grads"] = [_randn((n,), gen, getattr(torch, t), 1e-3) for n, t in _clip_shapes(case)]
        st["out"] = [torch.empty_like(g) for g in st["grads"]]
        # `over`: how far the norm is above the largest one allowed
        st["max_norm"] = 1e-3 * math.sqrt(case["n"]) / case["over"]
        return st
    T, d, F = case["T"], case["d"], case["F"]
    st["x"] = _randn((T, d), gen, bf16)
    st["w_g"] = _randn((F, d), gen, bf16, 1.0 / math.sqrt(d))
    st["w_u"] = _randn((F, d), gen, bf16, 1.0 / math.sqrt(d))
    st["w_d"] = _randn((d, F), gen, bf16, 1.0 / math.sqrt(F))
    if op == "ffn_backward":
        # what the forward pass left behind, and the gradient that arrives
        st["gate"] = _randn((T, F), gen, bf16)
        st["up"] = _randn((T, F), gen, bf16)
        st["dy"] = _randn((T, d), gen, bf16, 1e-3)
    if own:
        from mixture_experts_layer_router_gb300 import capi

        st["ffn"] = capi.GatedFFN(d, F, max_tokens=T, training=op == "ffn_backward")
    return st


def _plain_norm(st):
    s = st["xs"].to(torch.float32)
    if st["res"] is not None:
        s = s + st["res"].to(torch.float32)
    rstd = 1.0 / torch.sqrt((s * s).mean(1) + EPS)
    y = s * rstd[:, None] * st["weight"].to(torch.float32)
    out = {"rstd": rstd}
    if st["res"] is not None:
        out["sum"] = s.to(st["res"].dtype)
    if not st["codes"]:
        out["y"] = y.to(st["xs"].dtype)
        return out
    T, d = y.shape
    block = d if st["codes"] == "token" else BLOCK
    n = -(-d // block)
    if n * block != d:
        y = torch.cat([y, torch.zeros((T, n * block - d), device=y.device)], 1)
    y = y.view(T, n, block)
    top = y.abs().amax(2)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    q = (y * (1.0 / scale)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(T, n * block)[:, :d]
    out["codes"] = q.contiguous().to(torch.float8_e4m3fn)
    out["scales"] = scale
    return out


def _plain_norm_backward(st):
    w, r = st["weight"].to(torch.float32), st["rstd"][:, None]
    n = st["s"].to(torch.float32) * r
    dy = st["dys"].to(torch.float32)
    a = dy * w
    dx = (a - n * (a * n).mean(1, keepdim=True)) * r
    if st["ds"] is not None:
        dx = dx + st["ds"].to(torch.float32)
    return {"dx": dx.to(st["s"].dtype), "dw": (dy * n).sum(0)}


def _plain_ffn(st):
    x = st["x"].to(torch.float32)
    gate = torch.matmul(x, st["w_g"].to(torch.float32).t())
    up = torch.matmul(x, st["w_u"].to(torch.float32).t())
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.matmul(h, st["w_d"].to(torch.float32).t()).to(torch.bfloat16)
    if not st["save"]:
        return {"y": y}
    return {"y": y, "gate": gate.to(torch.bfloat16), "up": up.to(torch.bfloat16)}


def _plain_ffn_backward(st):
    f32, b16 = torch.float32, torch.bfloat16
    x, dy = st["x"].to(f32), st["dy"].to(f32)
    gate, up = st["gate"].to(f32), st["up"].to(f32)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    act = gate * sig
    dh = torch.matmul(dy, st["w_d"].to(f32))
    dg = dh * up * (sig * (1.0 + gate * (1.0 - sig)))
    du = dh * act
    dx = torch.matmul(dg, st["w_g"].to(f32)) + torch.matmul(du, st["w_u"].to(f32))
    return {"dx": dx.to(b16), "dw_g": torch.matmul(dg.t(), x).to(b16), "dw_u": torch.matmul(du.t(), x).to(b16),
            "dw_d": torch.matmul(dy.t(), act * up).to(b16)}


def _plain_clip(st):
    total = torch.stack([g.to(torch.float32).square().sum() for g in st["grads"]]).sum()
    norm = torch.sqrt(total)
    coef = torch.clamp(st["max_norm"] / (norm + CLIP_EPS), max=1.0)
    for o, g in zip(st["out"], st["grads"]):
        o.copy_(g.to(torch.float32) * coef)
    return {"norm": norm.view(1), "out": st["out"]}


def run(state):
    op = state["op"]
    if own:
        from mixture_experts_layer_router_gb300 import capi

        if op == "norm":
            got = capi.rms_norm(state["xs"], state["weight"], eps=EPS, residual=state["res"], quantize=state["codes"] or None)
            if state["codes"]:
                got["codes"] = got["codes"].view(torch.float8_e4m3fn)
            return got
        if op == "norm_backward":
            return capi.rms_norm_backward(state["dys"], state["s"], state["weight"], state["rstd"], d_sum=state["ds"])
        if op == "ffn":
            got = state["ffn"].forward(state["x"], state["w_g"], state["w_u"], state["w_d"], save=state["save"])
            return dict(zip(("y", "gate", "up"), got)) if state["save"] else {"y": got}
        if op == "ffn_backward":
            return state["ffn"].backward(state["dy"], state["x"], state["gate"], state["up"], state["w_g"], state["w_u"], state["w_d"])
        norm = capi.clip_gradients(state["grads"], state["max_norm"], eps=CLIP_EPS, out=state["out"])
        return {"norm": norm, "out": state["out"]}
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_backward":
        return _plain_norm_backward(state)
    if op == "ffn":
        return _plain_ffn(state)
    if op == "ffn_backward":
        return _plain_ffn_backward(state)
    return _plain_clip(state)


def _nearest_e4m3(v):
    """The E4M3 number nearest to each of the 64-bit values, ties to the even one."""
    m = v.abs()
    e = torch.floor(torch.log2(torch.where(m > 0, m, torch.ones_like(m)))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.copysign((torch.round(m / step) * step).clamp(max=E4M3_MAX), v)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        s = st["xs"].double() + (0 if st["res"] is None else st["res"].double())
        rstd = (s.pow(2).sum(1) / case["d"] + EPS).pow(-0.5)
        y = torch.einsum("td,t,d->td", s, rstd, st["weight"].double())
        out = {"rstd": rstd}
        if st["res"] is not None:
            out["sum"] = s
        if not case["codes"]:
            return {**out, "y": y}
        width = case["d"] if case["codes"] == "token" else BLOCK
        parts = y.split(width, 1)
        scales = torch.stack([p.abs().max(1).values for p in parts], 1) / E4M3_MAX
        scales[scales == 0] = 1.0
        codes = torch.cat([_nearest_e4m3(p / scales[:, i, None]) for i, p in enumerate(parts)], 1)
        return {**out, "codes": codes, "scales": scales}
    if op == "norm_backward":
        s, w, dy, r = st["s"].double(), st["weight"].double(), st["dys"].double(), st["rstd"].double()
        # with rstd a function of s: d rstd / d s = -rstd^3 s / d
        inner = torch.einsum("td,d,td->t", dy, w, s)
        dx = dy * w * r[:, None] - s * (inner * r ** 3 / case["d"])[:, None]
        if st["ds"] is not None:
            dx += st["ds"].double()
        return {"dx": dx, "dw": torch.einsum("td,td,t->d", dy, s, r)}
    if op == "clip":
        norm = math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in st["grads"]))
        coef = min(1.0, st["max_norm"] / (norm + CLIP_EPS))
        return {"norm": torch.tensor([norm], dtype=torch.float64), "out": [g.double() * coef for g in st["grads"]]}
    x, wg, wu, wd = (st[k].double() for k in ("x", "w_g", "w_u", "w_d"))
    if op == "ffn":
        gate, up = x @ wg.T, x @ wu.T
        y = (gate * torch.sigmoid(gate) * up) @ wd.T
        return {"y": y, "gate": gate, "up": up} if case["save"] else {"y": y}
    dy, gate, up = st["dy"].double(), st["gate"].double(), st["up"].double()
    sig = torch.sigmoid(gate)
    dh = dy @ wd
    dw_d = dy.T @ (sig * gate * up)
    dg = dh * up * (sig + gate * sig * (1.0 - sig))
    du = dh * (gate * sig)
    return {"dx": dg @ wg + du @ wu, "dw_g": dg.T @ x, "dw_u": du.T @ x, "dw_d": dw_d}
