"""Measured cases of the operators that train the layer's router and matrices.

Four operators: the router's balance loss with per-expert counts
(``balance_loss``), the gradient of that loss and of the gates with respect to
the router logits (``router_backward``), the Newton-Schulz orthogonalisation of
a matrix (``orthogonalize``), and the optimiser step around it (``muon_step``).
With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true it calls the library.

Definitions (S sequences of L tokens; N_s valid tokens of sequence s; p =
softmax of a token's logits, lse its log-sum-exp; k experts per token):

    counts[s, e]   slots of valid tokens that chose expert e
    prob_sum[s, e] sum of p_e over the valid tokens;  z_sum[s] sum of lse^2
    balance = mean_s E / (k N_s^2) sum_e counts[s, e] prob_sum[s, e]
    z       = mean_s z_sum[s] / N_s
    loss    = (balance_coef balance + z_coef z, balance, z)

    X_0 = U / (|U|_F + 1e-7);  X <- a X + (b A + c A^2) X with A = X X^T
    (A = X^T X and the products on the right for tall matrices), five times
    step: m <- mu m + g, U = g + mu m, W <- (1 - lr wd) W - lr scale X
"""
import math

import torch

own = False

COEFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
BALANCE_COEF, Z_COEF = 1e-2, 1e-3
LR, MU, WD = 2e-4, 0.95, 0.1

# The largest listed case of each kind bounds the drawn ones.
MOST_LOGITS = 65536 * 256
MOST_FLOPS = 3.4e12  # of the plain products


def listed():
    return [
        # one small micro-batch of the tiny layer: nothing but latency
        dict(name="loss_tiny", op="loss", S=1, L=128, E=16, k=2, pad=False),
        # the mid layer's batch with padded rows
        dict(name="loss_mid", op="loss", S=1, L=4096, E=64, k=4, pad=True),
        # 512 experts, top-8, a whole batch as one group (global-batch loss)
        dict(name="loss_wide", op="loss", S=1, L=16384, E=512, k=8, pad=False),
        # 16 padded sequences of 4096 tokens, the loss per sequence, 256 experts, top-7
        dict(name="loss_sequences", op="loss", S=16, L=4096, E=256, k=7, pad=True),
        # the backward of the mid layer's batch, renormalised gates
        dict(name="backward_mid", op="backward", S=1, L=4096, E=64, k=4, pad=True, renorm=True),
        # 512 experts, top-8, plain softmax gates
        dict(name="backward_wide", op="backward", S=1, L=16384, E=512, k=8, pad=False, renorm=False),
        # 16 padded sequences, renormalised gates
        dict(name="backward_sequences", op="backward", S=16, L=4096, E=256, k=7, pad=True, renorm=True),
        # the mid layer's router matrix: one short wide matrix, latency
        dict(name="orthogonalize_router", op="orthogonalize", batch=1, rows=64, cols=2048, grad="bfloat16"),
        # the mid layer's 64 gate matrices in one call
        dict(name="orthogonalize_experts", op="orthogonalize", batch=64, rows=2048, cols=1024, grad="bfloat16"),
        # odd sizes that no tile divides, a 32-bit gradient
        dict(name="orthogonalize_odd", op="orthogonalize", batch=3, rows=777, cols=1333, grad="float32"),
        # a 4096 x 8704 latent projection: 32-bit master weights and momentum
        dict(name="step_projection", op="step", batch=1, rows=4096, cols=8704, grad="bfloat16", weight="float32"),
        # eight expert down matrices, weights kept in bf16
        dict(name="step_experts", op="step", batch=8, rows=1024, cols=2048, grad="bfloat16", weight="bfloat16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "backward", "orthogonalize", "step"])
    if op in ("loss", "backward"):
        E = _log_int(rng, 7, 512)
        k = rng.randint(1, min(16, E))
        S = rng.choice([1, 1, _log_int(rng, 2, 64)])
        T = _log_int(rng, 100, 65536)
        if T * E > MOST_LOGITS:
            T = MOST_LOGITS // E
        case = dict(op=op, S=S, L=max(1, T // S), E=E, k=k, pad=rng.random() < 0.5)
        if op == "backward":
            case["renorm"] = rng.random() < 0.5
        return case
    rows, cols = _log_int(rng, 33, 8704), _log_int(rng, 33, 8704)
    while _plain_flops(1, rows, cols) > MOST_FLOPS:
        rows, cols = _log_int(rng, 33, 8704), _log_int(rng, 33, 8704)
    most = max(1, min(64, int(MOST_FLOPS / _plain_flops(1, rows, cols)), 2 ** 27 // (rows * cols)))
    case = dict(op=op, batch=_log_int(rng, 1, most), rows=rows, cols=cols, grad=rng.choice(["bfloat16", "float32"]))
    if op == "step":
        case["weight"] = rng.choice(["bfloat16", "float32"])
    return case


def _plain_flops(batch, rows, cols):
    m, n = min(rows, cols), max(rows, cols)
    return batch * STEPS * (4.0 * m * m * n + 2.0 * m ** 3)


def work(case):
    if case["op"] in ("loss", "backward"):
        T = case["S"] * case["L"]
        E, k = case["E"], case["k"]
        pad = T if case["pad"] else 0
        if case["op"] == "loss":
            return {"bytes": T * E * 4 + T * k * 4 + pad + case["S"] * E * 8, "flops": 5.0 * T * E}
        return {"bytes": 2 * T * E * 4 + T * k * 8 + pad + case["S"] * E * 4, "flops": 8.0 * T * E}
    # X X^T and A^2 are symmetric: half of their products
    b, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    flops = b * STEPS * (m * m * n + m ** 3 + 2.0 * m * m * n)
    g = 2 if case["grad"] == "bfloat16" else 4
    if case["op"] == "orthogonalize":
        return {"bytes": b * m * n * (g + 2), "flops": flops}
    w = 2 if case["weight"] == "bfloat16" else 4
    return {"bytes": b * m * n * (g + 2 * 4 + 2 * w), "flops": flops}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _router_inputs(case, gen):
    S, L, E, k = case["S"], case["L"], case["E"], case["k"]
    T = S * L
    # hidden states of unit scale against router rows give logits of about unit
    # scale; a few experts are more in demand than the others
    bias = 0.5 * torch.randn((E,), generator=gen, device="cuda")
    logits = torch.randn((T, E), generator=gen, device="cuda") + bias
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    valid = None
    if case["pad"]:  # the tail of every sequence is padding
        length = (L * (0.5 + 0.5 * torch.rand((S, 1), generator=gen, device="cuda"))).ceil()
        valid = (torch.arange(L, device="cuda")[None, :] < length).reshape(T).to(torch.uint8)
    return logits.contiguous(), idx.contiguous(), valid


def _gradient(shape, gen):
    """What a micro-batch leaves behind: a sum over tokens of outer products,
    with channels of unequal strength, and some noise."""
    b, r, c = shape
    t = 256
    out = torch.empty(shape, device="cuda")
    for i in range(b):
        delta = torch.randn((t, r), generator=gen, device="cuda")
        delta *= (1.0 + 9.0 * torch.rand((r,), generator=gen, device="cuda")) / 10.0
        x = torch.randn((t, c), generator=gen, device="cuda")
        x *= (1.0 + 9.0 * torch.rand((c,), generator=gen, device="cuda")) / 10.0
        out[i] = (delta.T @ x) / t
        out[i] += 0.02 * torch.randn((r, c), generator=gen, device="cuda")
    return out * 1e-3


def prepare(case, seed):
    gen = _generator(seed)
    state = dict(case)
    if case["op"] in ("loss", "backward"):
        logits, idx, valid = _router_inputs(case, gen)
        state.update(logits=logits, idx=idx, valid=valid)
        if case["op"] == "backward":
            T = case["S"] * case["L"]
            state["d_gates"] = torch.randn((T, case["k"]), generator=gen, device="cuda") / T
            state["d_loss"] = torch.ones((1,), device="cuda")
            # what the forward pass left behind: per-expert counts and valid tokens
            ok = torch.ones((T,), device="cuda", dtype=torch.int32) if valid is None else valid.to(torch.int32)
            state["counts"] = _counts(idx, ok, case["S"], case["L"], case["E"])
            state["tokens"] = ok.view(case["S"], case["L"]).sum(1).to(torch.int32)
        if own:
            from mixture_experts_layer_router_gb300 import capi

            # the layer's handle; its widths do not enter the router's loss
            state["layer"] = capi.LatentMoE(128, 128, case["E"], case["k"], 128, max_tokens=case["S"] * case["L"],
                                            renorm=bool(case.get("renorm", False)))
        return state
    shape = (case["batch"], case["rows"], case["cols"])
    state["g"] = _gradient(shape, gen).to(getattr(torch, case["grad"])).contiguous()
    if case["op"] == "step":
        # a momentum that has run for a while and weights of ordinary scale
        state["m"] = _gradient(shape, gen).mul_(4.0).contiguous()
        state["w"] = (0.02 * torch.randn(shape, generator=gen, device="cuda")).to(getattr(torch, case["weight"]))
        state["scale"] = 0.2 * math.sqrt(max(case["rows"], case["cols"]))
    if own:
        from mixture_experts_layer_router_gb300 import capi

        state["muon"] = capi.Muon(case["rows"], case["cols"], batch=case["batch"], steps=STEPS, coefs=COEFS, eps=EPS)
    return state


def _counts(idx, ok, S, L, E):
    T, k = idx.shape
    seq = torch.arange(T, device=idx.device) // L
    flat = (seq[:, None] * E + idx).reshape(-1)
    out = torch.zeros((S * E,), dtype=torch.int32, device=idx.device)
    out.index_add_(0, flat, ok[:, None].expand(T, k).reshape(-1).to(torch.int32))
    return out.view(S, E)


def _softmax(x):
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    s = e.sum(1, keepdim=True)
    return e / s, (m + torch.log(s))[:, 0]


def _plain_loss(st):
    S, L, E, k = st["S"], st["L"], st["E"], st["k"]
    p, lse = _softmax(st["logits"])
    T = S * L
    ok = torch.ones((T,), dtype=torch.int32, device=p.device) if st["valid"] is None else (st["valid"] != 0).to(torch.int32)
    f = ok.to(torch.float32)
    counts = _counts(st["idx"], ok, S, L, E)
    tokens = ok.view(S, L).sum(1).to(torch.int32)
    prob_sum = (p * f[:, None]).view(S, L, E).sum(1)
    z_sum = (lse * lse * f).view(S, L).sum(1)
    n = tokens.to(torch.float32)
    inv = torch.where(n > 0, 1.0 / n, torch.zeros_like(n))
    balance = ((counts.to(torch.float32) * prob_sum).sum(1) * inv * inv * (E / k)).sum() / S
    z = (z_sum * inv).sum() / S
    loss = torch.stack([BALANCE_COEF * balance + Z_COEF * z, balance, z])
    return {"loss": loss, "counts": counts, "prob_sum": prob_sum, "z_sum": z_sum, "tokens": tokens}


def _plain_backward(st):
    S, L, E, k = st["S"], st["L"], st["E"], st["k"]
    T = S * L
    p, lse = _softmax(st["logits"])
    f = torch.ones((T,), device=p.device) if st["valid"] is None else (st["valid"] != 0).to(torch.float32)
    n = st["tokens"].to(torch.float32)
    inv = torch.where(n > 0, 1.0 / n, torch.zeros_like(n))
    w = st["counts"].to(torch.float32) * (inv * inv)[:, None] * (BALANCE_COEF * E / (S * k)) * st["d_loss"]
    w = w[:, None, :].expand(S, L, E).reshape(T, E)
    q = (2.0 * Z_COEF / S) * inv * st["d_loss"]
    q = q[:, None].expand(S, L).reshape(T) * lse
    d = p * (w - (p * w).sum(1, keepdim=True) + q[:, None]) * f[:, None]
    ids = st["idx"].long()
    g = torch.gather(p, 1, ids)
    if st["renorm"]:
        g = g / g.sum(1, keepdim=True)
    dot = (g * st["d_gates"]).sum(1, keepdim=True)
    if st["renorm"]:
        return d.scatter_add(1, ids, g * (st["d_gates"] - dot))
    return (d - p * dot).scatter_add(1, ids, g * st["d_gates"])


def _plain_newton_schulz(u):
    a, b, c = COEFS
    x = u.to(torch.float32)
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return x.transpose(1, 2) if tall else x


def run(state):
    op = state["op"]
    if op == "loss":
        if own:
            return state["layer"].balance_loss(state["logits"], state["idx"], valid=state["valid"], seq_len=state["L"],
                                               balance_coef=BALANCE_COEF, z_coef=Z_COEF)
        return _plain_loss(state)
    if op == "backward":
        if own:
            return state["layer"].router_backward(state["logits"], state["idx"], state["counts"], state["tokens"],
                                                  d_gates=state["d_gates"], valid=state["valid"], seq_len=state["L"],
                                                  balance_coef=BALANCE_COEF, z_coef=Z_COEF, d_loss=state["d_loss"])
        return _plain_backward(state)
    if op == "orthogonalize":
        if own:
            return state["muon"].orthogonalize(state["g"])
        return _plain_newton_schulz(state["g"]).to(torch.bfloat16).contiguous()
    g, m, w = state["g"], state["m"], state["w"]
    if own:
        state["muon"].step(w, g, m, lr=LR, momentum_coef=MU, weight_decay=WD, scale=state["scale"], nesterov=True)
    else:
        m.mul_(MU).add_(g.to(torch.float32))
        x = _plain_newton_schulz(g.to(torch.float32) + MU * m)
        w.copy_(w.to(torch.float32) * (1.0 - LR * WD) - (LR * state["scale"]) * x)
    return {"w": w, "m": m}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("loss", "backward"):
        return _exact_router(st)
    g = st["g"].double()
    if case["op"] == "orthogonalize":
        return torch.stack([_exact_polar(g[i]) for i in range(case["batch"])])
    m = MU * st["m"].double() + g
    u = g + MU * m
    x = torch.stack([_exact_polar(u[i]) for i in range(case["batch"])])
    return {"w": st["w"].double() * (1.0 - LR * WD) - LR * st["scale"] * x, "m": m}


def _exact_polar(u):
    """The iteration on one matrix in 64 bits, always on its short side."""
    short = u if u.shape[0] <= u.shape[1] else u.t()
    x = short / (torch.linalg.vector_norm(short) + EPS)
    eye = torch.eye(x.shape[0], dtype=x.dtype, device=x.device)
    for _ in range(STEPS):
        gram = x @ x.t()
        x = (COEFS[0] * eye + gram @ (COEFS[1] * eye + COEFS[2] * gram)) @ x
    return x if u.shape[0] <= u.shape[1] else x.t()


def _exact_router(st):
    S, L, E, k = st["S"], st["L"], st["E"], st["k"]
    logits = st["logits"].double().view(S, L, E)
    ids = st["idx"].long().view(S, L, k)
    ok = torch.ones((S, L), dtype=torch.bool, device=logits.device) if st["valid"] is None else st["valid"].view(S, L) != 0
    lse = torch.logsumexp(logits, 2)
    p = torch.exp(logits - lse[..., None])
    chosen = torch.zeros((S, L, E), dtype=torch.int32, device=logits.device)
    chosen.scatter_(2, ids, 1)  # the experts of one token differ
    counts = (chosen * ok[..., None]).sum(1)
    n = ok.sum(1)
    inv = torch.where(n > 0, 1.0 / n.double(), torch.zeros_like(n, dtype=torch.float64))
    if st["op"] == "loss":
        prob = torch.einsum("sle,sl->se", p, ok.double())
        z_sum = (lse ** 2 * ok).sum(1)
        balance = (E / k) * ((counts * inv[:, None]) * (prob * inv[:, None])).sum() / S
        z = (z_sum * inv).mean()
        return {"loss": torch.stack([BALANCE_COEF * balance + Z_COEF * z, balance, z]), "counts": counts.to(torch.int32),
                "prob_sum": prob, "z_sum": z_sum, "tokens": n.to(torch.int32)}
    # the gradient with respect to the probabilities, through the softmax's Jacobian
    dp = (BALANCE_COEF * E / (S * k)) * counts * (inv ** 2)[:, None]
    dp = dp[:, None, :] * ok[..., None]
    dlse = (2.0 * Z_COEF / S) * inv[:, None] * lse * ok
    gates = torch.gather(p, 2, ids)
    dg = st["d_gates"].double().view(S, L, k)
    if st["renorm"]:
        total = gates.sum(2, keepdim=True)
        dg = (dg - (dg * gates / total).sum(2, keepdim=True)) / total
    dp = dp.scatter_add(2, ids, dg)
    d = p * (dp - (p * dp).sum(2, keepdim=True) + dlse[..., None])
    return d.view(S * L, E)
