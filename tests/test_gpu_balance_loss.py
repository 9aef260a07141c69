"""The router's balance loss and the router backward against their definition
in float64 (gradients by automatic differentiation of that definition, and by
differences of it).

Tolerances. An fp32 softmax probability: the difference x - max is exact to
2^-24 of itself, the exponential multiplies that by up to |x - max| and adds
2 ulp, the row sum of up to 512 terms in lanes adds about 16 roundings: for
|x - max| <= 32 at most (32 + 2 + 16 + 2) 2^-24 = 3.1e-6 of p. A column sum
adds a chain of at most 300 rows a lane here, 300 * 2^-24 = 1.8e-5 at the very
worst, all roundings in one direction: P_TOL = 2.2e-5. The loss sums products
of those: L_TOL = 5e-5. A gradient entry is a sum of terms, each exact to
about 1e-5 of itself (two probabilities and a sum over E): its error is
compared with G_TOL = 1e-5 times the sum of the terms' absolute values.
"""
import pytest
import torch

from mixture_experts_layer_router_gb300 import capi
import gpu_helpers as gh

pytestmark = pytest.mark.gpu

P_TOL, L_TOL, G_TOL = 2.2e-5, 5e-5, 1e-5
BC, ZC = 0.03, 0.002


def layer(E, k, T, renorm=False):
    gh.lib()
    return capi.LatentMoE(128, 128, E, k, 128, max_tokens=T, renorm=renorm)


def inputs(T, E, k, seed, scale=1.0, pad=False):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn((T, E), generator=g) * scale).cuda()
    idx = torch.topk(logits + torch.randn((T, E), generator=g).cuda(), k, dim=1).indices
    valid = (torch.rand((T,), generator=g) < 0.7).to(torch.uint8).cuda() if pad else None
    dg = torch.randn((T, k), generator=g).cuda()
    return logits, idx.to(torch.int32).contiguous(), valid, dg


def counts_mask(logits, valid):
    ok = ~(logits == float("-inf")).all(1)
    return ok if valid is None else ok & (valid != 0)


def definition(x, idx, valid, S, bc=BC, zc=ZC):
    """float64 stats and loss; x [T, E] may require gradients."""
    T, E = x.shape
    k = idx.shape[1]
    ok = counts_mask(x.detach(), valid)
    safe = torch.where(ok[:, None], x, torch.zeros_like(x))
    lse = torch.logsumexp(safe, 1)
    p = torch.exp(safe - lse[:, None]) * ok[:, None]
    hot = torch.zeros((T, E + 1), dtype=torch.float64, device=x.device)
    id64 = idx.long()
    id64 = torch.where((id64 >= 0) & (id64 < E), id64, torch.full_like(id64, E))
    hot.scatter_add_(1, id64, torch.ones_like(id64, dtype=torch.float64))
    counts = (hot[:, :E] * ok[:, None]).view(S, T // S, E).sum(1)
    n = ok.view(S, T // S).sum(1)
    inv = torch.where(n > 0, 1.0 / n.clamp(min=1).double(), torch.zeros_like(n, dtype=torch.float64))
    prob = p.view(S, T // S, E).sum(1)
    zsum = (lse.square() * ok).view(S, T // S).sum(1)
    balance = ((counts * inv[:, None]) * (prob * inv[:, None])).sum() * E / (k * S)
    z = (zsum * inv).sum() / S
    return {"loss": torch.stack([bc * balance + zc * z, balance, z]), "counts": counts,
            "prob_sum": prob, "z_sum": zsum, "tokens": n, "p": p, "lse": lse, "inv": inv, "ok": ok}


def gates_of(x, idx, renorm):
    E = x.shape[1]
    inside = (idx >= 0) & (idx < E)
    ids = torch.where(inside, idx, torch.zeros_like(idx)).long()
    if renorm:
        sel = torch.where(inside, torch.gather(x, 1, ids), torch.full_like(ids, 0).double() - float("inf"))
        dead = (sel == float("-inf")).all(1, keepdim=True)
        return torch.softmax(torch.where(dead, torch.zeros_like(sel), sel), 1) * ~dead * inside
    dead = (x == float("-inf")).all(1, keepdim=True)
    p = torch.softmax(torch.where(dead, torch.zeros_like(x), x), 1) * ~dead
    return torch.gather(p, 1, ids) * inside


def rel(a, b):
    return float((a.double() - b).norm() / b.norm().clamp(min=1e-300))


def check_loss(L, logits, idx, valid, seq_len, T):
    S = T // (seq_len or T)
    got = L.balance_loss(logits, idx, valid=valid, seq_len=seq_len, balance_coef=BC, z_coef=ZC)
    again = L.balance_loss(logits, idx, valid=valid, seq_len=seq_len, balance_coef=BC, z_coef=ZC)
    want = definition(logits.double(), idx, valid, S)
    assert torch.equal(got["counts"].double(), want["counts"])
    assert torch.equal(got["tokens"].long(), want["tokens"])
    assert rel(got["prob_sum"], want["prob_sum"]) <= P_TOL
    assert rel(got["z_sum"], want["z_sum"]) <= P_TOL
    assert rel(got["loss"], want["loss"]) <= L_TOL
    for key in got:
        assert torch.equal(got[key], again[key]), key
    return got


def check_backward(L, logits, idx, valid, seq_len, dg, got, renorm, d_loss=None):
    T, E = logits.shape
    S = T // (seq_len or T)
    out = L.router_backward(logits, idx, got["counts"], got["tokens"], d_gates=dg, valid=valid,
                            seq_len=seq_len, balance_coef=BC, z_coef=ZC, d_loss=d_loss)
    up = 1.0 if d_loss is None else float(d_loss)
    x = logits.double().requires_grad_(True)
    ref = definition(x, idx, valid, S)
    total = up * ref["loss"][0]
    gates = None
    if dg is not None:
        gates = gates_of(x, idx, renorm)
        total = total + (gates * dg.double()).sum()
    total.backward()
    want = torch.where(torch.isnan(x.grad), torch.zeros_like(x.grad), x.grad)
    # sum of the absolute terms of every entry
    with torch.no_grad():
        seq = torch.arange(T, device=x.device) // (T // S)
        w = (up * BC * E / (idx.shape[1] * S) * ref["counts"] * ref["inv"][:, None] ** 2)[seq]
        q = (up * 2 * ZC / S * ref["inv"])[seq] * ref["lse"].abs()
        p = ref["p"]
        size = p * (w.abs() + (p * w.abs()).sum(1, keepdim=True) + q[:, None])
        if dg is not None:
            g = gates
            inside = (idx >= 0) & (idx < E)
            ids = torch.where(inside, idx, torch.zeros_like(idx)).long()
            d = (g * dg.double()).abs()
            full = torch.softmax(torch.where(torch.isinf(x).all(1, keepdim=True), torch.zeros_like(x), x), 1)
            size = size + full * d.sum(1, keepdim=True)
            size = size.scatter_add(1, ids, (d + g * d.sum(1, keepdim=True)) * inside)
    err = (out.double() - want).abs()
    bad = err > G_TOL * size + 1e-30
    assert not bool(bad.any()), (int(bad.sum()), float((err / (size + 1e-300)).max()))
    return out


CASES = [(1, 1, 1), (1, 8, 2), (1, 512, 16), (2, 3, 3), (5, 7, 3), (31, 13, 4), (33, 16, 2),
         (100, 17, 5), (128, 16, 2), (257, 60, 6), (512, 64, 4), (300, 100, 8), (640, 128, 8),
         (333, 255, 7), (1024, 256, 7), (97, 300, 9), (200, 384, 8), (777, 511, 8), (4096, 64, 4),
         (5000, 512, 8), (20000, 10, 3)]


@pytest.mark.parametrize("pad", [False, True])
@pytest.mark.parametrize("T,E,k", CASES)
def test_loss_and_backward(T, E, k, pad):
    for renorm in (False, True):
        L = layer(E, k, T, renorm)
        logits, idx, valid, dg = inputs(T, E, k, T * 7 + E, pad=pad)
        got = check_loss(L, logits, idx, valid, 0, T)
        check_backward(L, logits, idx, valid, 0, dg, got, renorm)
        check_backward(L, logits, idx, valid, 0, None, got, renorm,
                       d_loss=torch.tensor([2.5], device="cuda"))
        assert L.status() == 0
