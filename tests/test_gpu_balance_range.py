"""The router's balance loss and backward at logits of any magnitude, against
their definition in float64 (probabilities from differences to the row's maximum,
so that the reference itself does not lose them).

Tolerances as derived in test_gpu_balance_loss: P_TOL of a probability, and
G_TOL of the sum of the absolute values of a gradient entry's terms.
"""
import pytest
import torch

from mixture_experts_layer_router_gb300 import capi

from test_gpu_balance_loss import BC, G_TOL, P_TOL, ZC, inputs, layer, rel

pytestmark = pytest.mark.gpu

MAGNITUDES = [9.9e5, 1.01e6, 1e7, 1e8, 1e9, 1e10, 1e12, 1e15, 1e20, 1e30, 9e36, 1.1e37]


def large_rows(E, k, seed, most=1e38):
    """For every magnitude and sign: a row of equal logits, one with a maximum one
    step above the rest, one half at it and half ordinary; ordinary rows between."""
    values = [s * v for v in MAGNITUDES if v <= most for s in (1.0, -1.0)]
    T = 4 * len(values)
    logits, idx, _, dg = inputs(T, E, k, seed)
    for i, v in enumerate(values):
        v = torch.tensor(v, device="cuda")
        logits[4 * i] = v
        logits[4 * i + 1] = v
        logits[4 * i + 1, (3 * i) % E] = torch.nextafter(v, v.new_tensor(float("inf")))
        logits[4 * i + 2, : E // 2] = v
    return T, logits, idx, dg


def check_gradient(got, want, size):
    bad = (got.double() - want).abs() > G_TOL * size + 1e-30
    assert not bool(bad.any()), bad.any(1).nonzero().flatten().tolist()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(16, 2), (64, 4), (61, 4), (13, 3), (256, 7), (509, 8)])
def test_large_logits(E, k, renorm):
    T, logits, idx, dg = large_rows(E, k, 5)
    h = layer(E, k, T, renorm)
    x = logits.double()
    p = torch.softmax(x, 1)
    # a sequence a token: prob_sum is p itself
    each = h.balance_loss(logits, idx, seq_len=1, balance_coef=BC)
    assert bool((each["tokens"] == 1).all())
    assert bool((each["counts"].sum(1) == k).all())
    assert bool(((each["prob_sum"].double() - p).abs() <= P_TOL * p + 1e-37).all())
    whole = h.balance_loss(logits, idx, balance_coef=BC)
    assert int(whole["tokens"]) == T
    assert rel(whole["prob_sum"][0], p.sum(0)) <= P_TOL
    counts = torch.zeros((E,), dtype=torch.float64, device="cuda").index_add_(
        0, idx.flatten().long(), torch.ones(T * k, dtype=torch.float64, device="cuda"))
    assert torch.equal(whole["counts"][0].double(), counts)
    assert rel(whole["loss"][1:2], (counts * p.sum(0)).sum()[None] * E / (k * T * T)) <= 2 * P_TOL
    # the gradient, the loss's part and the gates' part
    out = h.router_backward(logits, idx, whole["counts"], whole["tokens"], d_gates=dg,
                            balance_coef=BC)
    w = BC * E / (k * T * T) * counts
    loss_part = p * (w - (p * w).sum(1, keepdim=True))
    g = torch.gather(p, 1, idx.long())
    if renorm:
        g = torch.softmax(torch.gather(x, 1, idx.long()), 1)
    d = g * dg.double()
    D = d.sum(1, keepdim=True)
    dense = torch.zeros_like(p) if renorm else p * D
    sparse = (d - g * D) if renorm else d
    want = (loss_part - dense).scatter_add(1, idx.long(), sparse)
    size = p * (w + (p * w).sum(1, keepdim=True) + d.abs().sum(1, keepdim=True))
    size = size.scatter_add(1, idx.long(), d.abs() + g * d.abs().sum(1, keepdim=True))
    check_gradient(out, want, size)
    assert h.status() == 0


@pytest.mark.parametrize("E,k", [(64, 4), (61, 4)])
def test_large_logits_with_the_z_term(E, k):
    """Up to 1e15, where the squares of lse are still finite."""
    T, logits, idx, _ = large_rows(E, k, 6, most=1e15)
    h = layer(E, k, T)
    x = logits.double()
    p, lse = torch.softmax(x, 1), torch.logsumexp(x, 1)
    each = h.balance_loss(logits, idx, seq_len=1, balance_coef=BC, z_coef=ZC)
    assert bool(((each["z_sum"].double() - lse ** 2).abs() <= P_TOL * lse ** 2).all())
    whole = h.balance_loss(logits, idx, balance_coef=BC, z_coef=ZC)
    assert rel(whole["z_sum"], (lse ** 2).sum()[None]) <= P_TOL
    out = h.router_backward(logits, idx, whole["counts"], whole["tokens"], balance_coef=BC,
                            z_coef=ZC)
    w = BC * E / (k * T * T) * whole["counts"][0].double()
    q = 2 * ZC / T * lse[:, None]
    dot = (p * w).sum(1, keepdim=True)
    check_gradient(out, p * (w - dot + q), p * (w + dot + q.abs()))


@pytest.mark.parametrize("E,k", [(64, 4), (13, 3)])
def test_no_z_term_without_its_coefficient(E, k):
    """A row whose lse squared overflows: z is infinite, and with z_coef = 0 it is no
    part of the loss."""
    T = 32
    h = layer(E, k, T)
    logits, idx, _, _ = inputs(T, E, k, 7)
    logits[3] = torch.finfo(torch.float32).min
    for seq_len in (0, 8):
        got = h.balance_loss(logits, idx, seq_len=seq_len, balance_coef=0.5, z_coef=0.0)
        assert bool(torch.isinf(got["z_sum"]).any()) and bool(torch.isinf(got["loss"][2]))
        assert bool(torch.isfinite(got["loss"][1]))
        assert torch.equal(got["loss"][0], 0.5 * got["loss"][1])
        again = h.balance_loss_from_stats(got, balance_coef=0.5, z_coef=0.0)
        assert bool(torch.isinf(again[2]))
        assert torch.equal(again[0], 0.5 * again[1])
        on = h.balance_loss(logits, idx, seq_len=seq_len, balance_coef=0.5, z_coef=1e-3)
        assert bool(torch.isinf(on["loss"][0]))
    # NaN stays NaN with either coefficient at zero
    logits[5, 1] = float("nan")
    for bc, zc in ((0.5, 0.0), (0.0, 0.5), (0.0, 0.0)):
        assert bool(torch.isnan(h.balance_loss(logits, idx, balance_coef=bc, z_coef=zc)["loss"][0]))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(16, 2), (64, 4), (61, 4), (13, 3), (256, 7), (512, 16), (8, 1)])
def test_padding_may_hold_anything_beside_gates(E, k, renorm):
    """Padded tokens whose gates carry no gradient get zeros whatever their logits
    hold, and leave the other tokens' gradients as they are, bit for bit."""
    T = 90
    h = layer(E, k, T, renorm)
    logits, idx, _, dg = inputs(T, E, k, 13)
    pad = torch.arange(T, device="cuda") % 3 == 1
    valid = (~pad).to(torch.uint8)
    dg[pad] = 0.0
    st = h.balance_loss(logits, idx, valid=valid, balance_coef=BC, z_coef=ZC)
    args = dict(d_gates=dg, valid=valid, balance_coef=BC, z_coef=ZC)
    clean = h.router_backward(logits, idx, st["counts"], st["tokens"], **args)
    assert not bool(clean[pad].any()) and bool(clean[~pad].any())
    inf, nan = float("inf"), float("nan")
    dirty = logits.clone()
    rows = pad.nonzero().flatten().tolist()
    fills = [nan, inf, -inf, torch.finfo(torch.float32).max, torch.finfo(torch.float32).min]
    for i, r in enumerate(rows):
        if i % 3 == 0:
            dirty[r] = fills[i // 3 % len(fills)]            # the whole row
        elif i % 3 == 1:
            dirty[r, idx[r, 0].long()] = fills[i // 3 % 2]   # a chosen expert
        else:
            dirty[r, (idx[r, 0].long() + 1) % E] = fills[i // 3 % 2]
    again = h.balance_loss(dirty, idx, valid=valid, balance_coef=BC, z_coef=ZC)
    for key in st:
        assert torch.equal(st[key], again[key]), key
    got = h.router_backward(dirty, idx, st["counts"], st["tokens"], **args)
    assert torch.equal(got, clean)


@pytest.mark.parametrize("E,k", [(64, 4), (13, 3), (512, 8)])
def test_gates_of_padding_with_nan_elsewhere(E, k):
    """Renormalised gates depend on the chosen logits alone: a NaN beside them in a
    padded token does not reach their gradient. Plain gates hold every logit, and the
    NaN is not hidden."""
    T = 40
    logits, idx, _, dg = inputs(T, E, k, 19)
    valid = torch.ones(T, dtype=torch.uint8, device="cuda")
    valid[::2] = 0
    other = torch.ones((T, E), dtype=torch.bool, device="cuda").scatter_(1, idx.long(), False)
    spot = other.to(torch.int32).argmax(1)  # the first expert that was not chosen
    dirty = logits.clone()
    dirty[::2] = dirty[::2].scatter(1, spot[::2, None], float("nan"))
    for renorm in (True, False):
        h = layer(E, k, T, renorm)
        st = h.balance_loss(logits, idx, valid=valid)
        clean = h.router_backward(logits, idx, st["counts"], st["tokens"], d_gates=dg, valid=valid)
        got = h.router_backward(dirty, idx, st["counts"], st["tokens"], d_gates=dg, valid=valid)
        if renorm:
            assert torch.equal(got, clean)
        else:
            assert torch.equal(got[1::2], clean[1::2])
            assert bool(torch.isnan(got[::2]).any(1).all())


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(16, 2), (61, 4), (512, 16)])
def test_gradients_of_dropped_slots_are_not_read(E, k, renorm):
    """A slot whose id is outside [0, E) contributes nothing, whatever its d_gates hold."""
    T = 33
    h = layer(E, k, T, renorm)
    logits, idx, _, dg = inputs(T, E, k, 29)
    idx[::3, 0] = -1
    idx[1::3, k - 1] = E
    st = h.balance_loss(logits, idx, balance_coef=BC)
    assert h.status() == capi.STATUS_BAD_EXPERT
    dropped = (idx < 0) | (idx >= E)
    args = dict(balance_coef=BC)
    want = h.router_backward(logits, idx, st["counts"], st["tokens"],
                             d_gates=dg.masked_fill(dropped, 0.0), **args)
    assert bool(torch.isfinite(want).all())
    for v in (5.0, float("inf"), float("nan")):
        got = h.router_backward(logits, idx, st["counts"], st["tokens"],
                                d_gates=dg.masked_fill(dropped, v), **args)
        assert torch.equal(got, want), v
