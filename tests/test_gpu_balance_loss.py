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


@pytest.mark.parametrize("S,L,E,k", [(2, 1, 5, 2), (3, 5, 16, 2), (16, 64, 64, 4), (200, 7, 60, 6),
                                     (2, 5000, 32, 4), (9, 33, 512, 8), (40, 700, 256, 7),
                                     (152, 3, 8, 8), (1, 6001, 13, 1)])
def test_sequences(S, L, E, k):
    T = S * L
    for renorm in (False, True):
        h = layer(E, k, T, renorm)
        logits, idx, valid, dg = inputs(T, E, k, T + E, scale=2.0, pad=True)
        valid.view(S, L)[0] = 0  # a sequence of padding alone
        got = check_loss(h, logits, idx, valid, L, T)
        assert int(got["tokens"][0]) == 0 and not bool(got["counts"][0].any())
        check_backward(h, logits, idx, valid, L, dg, got, renorm,
                       d_loss=torch.tensor([0.5], device="cuda"))
        assert h.status() == 0


def test_nothing_counts():
    h = layer(16, 2, 64)
    logits, idx, _, dg = inputs(64, 16, 2, 5)
    valid = torch.zeros(64, dtype=torch.uint8, device="cuda")
    logits[3] = float("nan")  # padding may hold anything
    got = h.balance_loss(logits, idx, valid=valid, balance_coef=BC, z_coef=ZC)
    for key in got:
        assert not bool(got[key].any()), key
    out = h.router_backward(logits, idx, got["counts"], got["tokens"], valid=valid,
                            balance_coef=BC, z_coef=ZC)
    assert torch.equal(out, torch.zeros_like(out))


@pytest.mark.parametrize("E,k", [(8, 2), (60, 6), (64, 4), (512, 8)])
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_logits(E, k, renorm):
    """Masks of -inf and of the type's lowest value: some experts, whole rows."""
    T = 96
    h = layer(E, k, T, renorm)
    logits, idx, _, dg = inputs(T, E, k, 11)
    low = torch.finfo(torch.float32).min
    logits[0] = float("-inf")           # nothing left: the row does not count
    logits[1] = low                     # equal lowest values: uniform
    logits[2, : E // 2] = float("-inf")
    logits[3, : E // 2] = low
    logits[4, 1:] = float("-inf")       # one expert left
    logits[5] = 3.0e38                  # the other end
    logits[6] *= 1e4
    logits[7] = logits[7] * 1e-30 + 80.0
    # row 1's and 5's z terms overflow by definition; they are checked apart
    z_rows = torch.ones(T, dtype=torch.uint8, device="cuda")
    z_rows[1] = z_rows[5] = 0
    got = check_loss(h, logits, idx, z_rows, 0, T)
    assert int(got["tokens"]) == T - 3
    check_backward(h, logits, idx, z_rows, 0, dg, got, renorm)
    one = h.balance_loss(logits, idx, balance_coef=1.0, z_coef=0.0)
    p = torch.softmax(logits.double(), 1)
    p[0] = 0
    assert int(one["tokens"]) == T - 1
    assert rel(one["prob_sum"][0], p.sum(0)) <= P_TOL
    assert torch.isinf(one["z_sum"]).all()


def test_nan_is_not_hidden():
    h = layer(32, 4, 50)
    logits, idx, _, dg = inputs(50, 32, 4, 3)
    logits[7, 5] = float("nan")
    got = h.balance_loss(logits, idx, balance_coef=BC, z_coef=ZC)
    assert torch.isnan(got["loss"]).all() and int(got["tokens"]) == 50
    out = h.router_backward(logits, idx, got["counts"], got["tokens"], d_gates=dg,
                            balance_coef=BC, z_coef=ZC)
    bad = torch.isnan(out).any(1)
    assert bool(bad[7]) and int(bad.sum()) == 1


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(8, 4), (64, 4), (13, 6), (256, 16)])
def test_given_choices(E, k, renorm):
    """Replayed choices: repeated ids add up, ids outside [0, E) drop out, ids of
    vanishing probability keep their renormalised gates."""
    T = 70
    h = layer(E, k, T, renorm)
    logits, idx, _, dg = inputs(T, E, k, 17)
    idx[0] = idx[0, 0]
    idx[1, 1] = idx[1, 0]
    idx[2, 0] = -1
    idx[3, k - 1] = E
    idx[4] = 1 << 30
    idx[5, 0] = -(1 << 31)
    logits[6] += 200.0 * (torch.arange(E, device="cuda") == E - 1)
    idx[6] = torch.arange(k, device="cuda") % (E - 1)
    got = check_loss(h, logits, idx, None, 0, T)
    assert h.status() == capi.STATUS_BAD_EXPERT
    assert h.status() == 0
    check_backward(h, logits, idx, None, 0, dg, got, renorm)
    a = h.router_backward(logits, idx, got["counts"], got["tokens"], d_gates=dg)
    for _ in range(3):
        assert torch.equal(a, h.router_backward(logits, idx, got["counts"], got["tokens"],
                                                d_gates=dg))


@pytest.mark.parametrize("E,ld,ldd", [(64, 80, 64), (64, 67, 72), (60, 61, 60), (512, 516, 520)])
def test_row_strides_and_in_place(E, ld, ldd):
    T, k = 130, 4
    h = layer(E, k, T)
    logits, idx, _, dg = inputs(T, E, k, 23)
    wide = torch.full((T, ld), 1e9, device="cuda")
    wide[:, :E] = logits
    view = wide[:, :E]
    got = h.balance_loss(view, idx, balance_coef=BC, z_coef=ZC)
    plain = h.balance_loss(logits, idx, balance_coef=BC, z_coef=ZC)
    assert torch.equal(got["counts"], plain["counts"])
    assert rel(got["loss"], plain["loss"].double()) <= L_TOL
    out = torch.full((T, ldd), 7.0, device="cuda")
    args = dict(d_gates=dg, balance_coef=BC, z_coef=ZC)
    h.router_backward(view, idx, got["counts"], got["tokens"], out=out[:, :E], **args)
    assert torch.all(out[:, E:] == 7.0) and torch.all(wide[:, E:] == 1e9)
    want = h.router_backward(logits, idx, got["counts"], got["tokens"], **args)
    torch.testing.assert_close(out[:, :E], want, rtol=1e-5, atol=1e-9)
    same = logits.clone()
    h.router_backward(same, idx, got["counts"], got["tokens"], out=same, **args)
    assert torch.equal(same, want)


def test_sums_of_micro_batches():
    """The stats of two halves add up to the whole batch's; the loss of the sums
    and the gradient with the sums are the whole batch's."""
    T, E, k = 1000, 64, 4
    h = layer(E, k, T)
    logits, idx, valid, dg = inputs(T, E, k, 31, pad=True)
    whole = h.balance_loss(logits, idx, valid=valid, balance_coef=BC, z_coef=ZC)
    cut = 360
    halves = [h.balance_loss(logits[a:b], idx[a:b], valid=valid[a:b]) for a, b in
              ((0, cut), (cut, T))]
    total = {n: halves[0][n] + halves[1][n] for n in ("counts", "prob_sum", "z_sum", "tokens")}
    assert torch.equal(total["counts"], whole["counts"])
    loss = h.balance_loss_from_stats(total, balance_coef=BC, z_coef=ZC)
    assert rel(loss, whole["loss"].double()) <= L_TOL
    d = h.router_backward(logits, idx, whole["counts"], whole["tokens"], d_gates=dg, valid=valid,
                          balance_coef=BC, z_coef=ZC)
    parts = [h.router_backward(logits[a:b], idx[a:b], total["counts"], total["tokens"],
                               d_gates=dg[a:b], valid=valid[a:b], balance_coef=BC, z_coef=ZC)
             for a, b in ((0, cut), (cut, T))]
    assert torch.equal(d, torch.cat(parts))
    seqs = h.balance_loss(logits, idx, valid=valid, seq_len=100, balance_coef=BC, z_coef=ZC)
    again = h.balance_loss_from_stats(seqs, balance_coef=BC, z_coef=ZC)
    assert rel(again, seqs["loss"].double()) <= L_TOL


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_by_differences(renorm):
    """<gradient, v> against central differences of the float64 definition along
    v. The definition is smooth: a step of 1e-4 leaves an error of order 1e-8;
    the gradient's own is 1e-5 of the sum of its absolute terms."""
    T, E, k, S = 24, 20, 3, 2
    h = layer(E, k, T, renorm)
    logits, idx, valid, dg = inputs(T, E, k, 41, pad=True)
    got = h.balance_loss(logits, idx, valid=valid, seq_len=T // S, balance_coef=BC, z_coef=ZC)
    d = h.router_backward(logits, idx, got["counts"], got["tokens"], d_gates=dg, valid=valid,
                          seq_len=T // S, balance_coef=BC, z_coef=ZC).double()

    def f(x):
        return definition(x, idx, valid, S)["loss"][0] + (gates_of(x, idx, renorm) *
                                                          dg.double()).sum()

    for seed in range(5):
        v = torch.randn((T, E), generator=torch.Generator().manual_seed(seed),
                        dtype=torch.float64).cuda()
        e = 1e-4
        diff = (f(logits.double() + e * v) - f(logits.double() - e * v)) / (2 * e)
        assert abs(float((d * v).sum() - diff)) <= 1e-5 * float((d * v).abs().sum()) + 1e-6


def test_other_stream_and_graph():
    T, E, k = 4096, 64, 4
    h = layer(E, k, T)
    logits, idx, _, dg = inputs(T, E, k, 47)
    want = h.balance_loss(logits, idx, balance_coef=BC, z_coef=ZC)
    d = h.router_backward(logits, idx, want["counts"], want["tokens"], d_gates=dg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = h.balance_loss(logits, idx, balance_coef=BC, z_coef=ZC)
        e = h.router_backward(logits, idx, got["counts"], got["tokens"], d_gates=dg)
    side.synchronize()
    for key in want:
        assert torch.equal(want[key], got[key]), key
    assert torch.equal(d, e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = h.balance_loss(logits, idx, balance_coef=BC, z_coef=ZC)
        e = h.router_backward(logits, idx, got["counts"], got["tokens"], d_gates=dg)
    before = h.launch_count()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert h.launch_count() == before
    for key in want:
        assert torch.equal(want[key], got[key]), key
    assert torch.equal(d, e)


def test_matches_the_forwards_statistics():
    """On the routing of a forward: the statistics of latentmoe_lbl_stats."""
    from mixture_experts_layer_router_gb300 import synth
    cfg = synth.CONFIGS["tiny"]
    w = synth.make_weights(cfg, 2, "cuda")
    h = gh.make_layer(cfg, w)
    h.forward(synth.make_x(cfg, 2, "cuda"))
    r = h.get_routing(cfg.T, "cuda")
    prob, counts = h.lbl_stats("cuda")
    got = h.balance_loss(r["logits"], r["idx"])
    assert torch.equal(got["counts"][0], counts)
    assert rel(got["prob_sum"][0], prob.double()) <= 2 * P_TOL
    assert int(got["tokens"]) == cfg.T


def test_refusals():
    T, E, k = 64, 16, 2
    h = layer(E, k, T)
    logits, idx, _, dg = inputs(T, E, k, 1)
    got = h.balance_loss(logits, idx)
    lib, hd = capi.load(), h.handle
    st = capi.latentmoe_balance_stats(*(got[n].data_ptr() for n in
                                        ("counts", "prob_sum", "z_sum", "tokens")))
    loss = torch.empty(3, device="cuda")
    import ctypes

    def fwd(T_=T, ld=E, seq=0, p=logits.data_ptr(), bc=1.0, i=idx.data_ptr(), o=loss.data_ptr()):
        return lib.latentmoe_balance_loss(hd, p, ld, i, None, T_, seq, bc, 0.0, ctypes.byref(st),
                                          o, None)

    assert fwd() == capi.OK
    assert fwd(T_=0) == fwd(T_=-1) == fwd(T_=T + 1) == capi.ERR_INVALID_ARG
    assert fwd(seq=7) == fwd(seq=-1) == capi.ERR_INVALID_ARG
    assert fwd(ld=E - 1) == capi.ERR_INVALID_ARG
    assert fwd(p=None) == fwd(i=None) == fwd(o=None) == capi.ERR_INVALID_ARG
    assert fwd(bc=float("nan")) == capi.ERR_INVALID_ARG
    assert fwd(p=logits.data_ptr() + 4, T_=1) == capi.ERR_UNSUPPORTED
    out = torch.empty_like(logits)

    def bwd(c=got["counts"].data_ptr(), n=got["tokens"].data_ptr(), i=idx.data_ptr(),
            g=dg.data_ptr(), o=out.data_ptr(), ldd=E, seq=0):
        return lib.latentmoe_router_backward(hd, logits.data_ptr(), E, i, g, None, c, n, T, seq,
                                             1.0, 0.0, None, o, ldd, None)

    assert bwd() == bwd(g=None, i=None) == capi.OK
    assert bwd(c=None) == bwd(n=None) == bwd(o=None) == bwd(i=None) == capi.ERR_INVALID_ARG
    assert bwd(ldd=E - 1) == bwd(seq=5) == capi.ERR_INVALID_ARG
    assert bwd(o=out.data_ptr() + 4) == capi.ERR_UNSUPPORTED
    assert lib.latentmoe_balance_loss_from_stats(hd, ctypes.byref(st), 0, 1.0, 0.0,
                                                 loss.data_ptr(), None) == capi.ERR_INVALID_ARG
    st.counts = None
    assert fwd() == capi.ERR_INVALID_ARG
    torch.cuda.synchronize()
    # the binding's own checks
    for bad in (dict(logits=logits.double()), dict(logits=logits[:, :8]), dict(idx=idx.long()),
                dict(idx=idx[:10]), dict(seq_len=7), dict(valid=torch.ones(T, device="cuda")),
                dict(logits=logits.t().contiguous().t()), dict(logits=logits.cpu())):
        args = dict(logits=logits, idx=idx)
        args.update(bad)
        with pytest.raises(ValueError):
            h.balance_loss(**args)
    for bad in (dict(counts=got["counts"].long()), dict(tokens=got["tokens"][:0]),
                dict(d_gates=dg.half()), dict(d_loss=torch.ones(2, device="cuda"))):
        args = dict(logits=logits, idx=idx, counts=got["counts"], tokens=got["tokens"])
        args.update(bad)
        with pytest.raises(ValueError):
            h.router_backward(**args)


def test_offsets_beyond_32_bits():
    """More than 2^31 logits: uniform rows but for the last three, whose part of the
    sums and gradients is known by itself."""
    T, E, k = 2 ** 22 + 3, 512, 1
    h = layer(E, k, T)
    logits = torch.zeros((T, E), device="cuda")
    tail, _, _, _ = inputs(3, E, k, 3, scale=2.0)
    logits[-3:] = tail
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    idx[-3:, 0] = torch.tensor([E - 1, 5, E - 1], device="cuda")
    got = h.balance_loss(logits, idx, balance_coef=1.0, z_coef=0.5)
    assert int(got["tokens"]) == T
    assert got["counts"][0, [0, 5, E - 1]].tolist() == [T - 3, 1, 2]
    p = torch.softmax(tail.double(), 1)
    want = torch.full((E,), (T - 3) / E, dtype=torch.float64, device="cuda") + p.sum(0)
    # a lane adds up to 2000 equal terms here: 2000 roundings
    assert rel(got["prob_sum"][0], want) <= 2000 * 2.0 ** -24
    d = h.router_backward(logits, idx, got["counts"], got["tokens"], balance_coef=1.0, z_coef=0.5)
    w = got["counts"][0].double() * E / (k * float(T) ** 2)
    lse = torch.logsumexp(tail.double(), 1, keepdim=True)
    q = 2 * 0.5 / T
    dot = (p * w).sum(1, keepdim=True)
    ref = p * (w - dot + q * lse)
    size = p * (w + dot + q * lse.abs())
    assert bool(((d[-3:].double() - ref).abs() <= G_TOL * size + 1e-30).all())


def test_outputs_of_another_stream_do_not_take_memory_in_use():
    """Memory freed on the current stream, where a kernel has still to write it, is
    not handed to the outputs of a call on another stream."""
    T, E, k = 512, 64, 4
    L = layer(E, k, T)
    logits, idx, _, dg = inputs(T, E, k, 5)
    want = L.balance_loss(logits, idx, balance_coef=BC, z_coef=ZC)
    grad = L.router_backward(logits, idx, want["counts"], want["tokens"], d_gates=dg)
    torch.empty(3, device="cuda").fill_(7.0)  # loads the fill kernel
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # 10 ms at 2 GHz
    for shape in ((T, E), (1, E), (3,), (1,)):
        late = [torch.empty(shape, device="cuda").fill_(7.0) for _ in range(4)]
        del late
    got = L.balance_loss(logits, idx, balance_coef=BC, z_coef=ZC, stream=side)
    loss = L.balance_loss_from_stats(got, balance_coef=BC, z_coef=ZC, stream=side)
    d = L.router_backward(logits, idx, got["counts"], got["tokens"], d_gates=dg, stream=side)
    torch.cuda.synchronize()
    for key in want:
        assert torch.equal(got[key], want[key]), key
    assert torch.equal(d, grad) and rel(loss, want["loss"].double()) <= L_TOL


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(300, 16, 2), (4096, 64, 4), (1000, 255, 7), (512, 512, 16)])
def test_gradient_over_the_logits(T, E, k, renorm):
    h = layer(E, k, T, renorm)
    logits, idx, valid, dg = inputs(T, E, k, T + E, pad=True)
    st = h.balance_loss(logits, idx, valid=valid, balance_coef=BC, z_coef=ZC)
    args = dict(d_gates=dg, valid=valid, balance_coef=BC, z_coef=ZC)
    want = h.router_backward(logits, idx, st["counts"], st["tokens"], **args)
    h.router_backward(logits, idx, st["counts"], st["tokens"], out=logits, **args)
    assert torch.equal(logits, want)
