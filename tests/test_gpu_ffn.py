"""Gated feed-forward block and its gradient against the formulas in float64.

Tolerances. Operands are bf16 and their products exact in fp32; a sum of K products
is off by at most (K + 4) 2^-24 of the sum of their magnitudes. h, dg and du are
rounded to bf16 before the next product: half a step, R = 2^-8, of an entry (with
the activation's own error, a few 2^-22, far below it). So for D = A B^T with A so
rounded, entry by entry,
    |D - exact| <= R |exact| + ((1 + R) R + 2^-16 + (K + 4) 2^-24) (|A| |B|^T),
the first term being the result's own rounding (0 in fp32). dh is such a sum itself,
without a rounding: it is off by E = (d + 4) 2^-24 |dy| |Wd|, however small it comes out
where its terms cancel, and dg and du by |up SiLU'| E and |SiLU| E, which |B| then passes
on (one token's dW has nothing to average that out). That worst case grows
with K where the roundings in fact cancel; so results of 1000 entries or more are
also held to it in the mean square: two independent roundings of at most R / sqrt(3)
each, 3.2e-3 of the result's norm, TOL = 4e-3 (fp32 results: one, 2.3e-3, the same
TOL).
"""
import ctypes

import pytest
import torch

from mixture_experts_layer_router_gb300 import capi
import gpu_helpers as gh

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
R = 2.0 ** -8
TOL = 4e-3


def rand(shape, seed, scale=1.0, dtype=BF16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def block(T, d, F, seed=0):
    w = {"w_g": rand((F, d), seed + 1, d ** -0.5), "w_u": rand((F, d), seed + 2, d ** -0.5),
         "w_d": rand((d, F), seed + 3, F ** -0.5)}
    return rand((T, d), seed), w


def formula(x, w):
    g, u = x.double() @ w["w_g"].double().T, x.double() @ w["w_u"].double().T
    h = g * torch.sigmoid(g) * u
    return g, u, h, h @ w["w_d"].double().T


def gradients(dy, x, gate, up, w):
    """name -> (exact, magnitudes |A| |B|^T, K, what dh is off by, passed on)."""
    dy, x, g, u = (t.double() for t in (dy, x, gate, up))
    wg, wu, wd = (w[n].double() for n in ("w_g", "w_u", "w_d"))
    T, F = g.shape
    s = torch.sigmoid(g)
    dh, off = dy @ wd, (dy.shape[1] + 4) * 2.0 ** -24 * (dy.abs() @ wd.abs())
    slope, act = u * (s + g * s * (1 - s)), g * s
    dg, du, h = dh * slope, dh * act, act * u
    og, ou = off * slope.abs(), off * act.abs()
    zero = torch.zeros((), device="cuda", dtype=torch.float64)
    return {"dx": (dg @ wg + du @ wu, dg.abs() @ wg.abs() + du.abs() @ wu.abs(), 2 * F,
                   og @ wg.abs() + ou @ wu.abs()),
            "dw_g": (dg.T @ x, dg.abs().T @ x.abs(), T, og.T @ x.abs()),
            "dw_u": (du.T @ x, du.abs().T @ x.abs(), T, ou.T @ x.abs()),
            "dw_d": (dy.T @ h, dy.abs().T @ h.abs(), T, zero)}


def check(got, exact, size, K, passed=0.0, out=BF16):
    slack = (1 + R) * R + 2.0 ** -16 + (K + 4) * 2.0 ** -24
    own = R if out == BF16 else 2.0 ** -24
    d = (got.double() - exact).abs()
    assert bool((d <= own * exact.abs() + slack * size + (1 + R) ** 2 * passed + 1e-30).all()), float((d / (slack * size + 1e-30)).max())
    if got.numel() >= 1000:
        assert float(d.norm()) <= TOL * float(exact.norm())


# one row, fewer rows and columns than a tile has, borders of the tiles (64, 128, 256)
# and their neighbours, several tiles in every direction
# (and 7 and 8 rows: the border of the padded operands)
SIZES = [(1, 8, 8), (1, 256, 512), (7, 200, 136), (8, 136, 200), (3, 16, 24), (17, 1024, 640), (64, 64, 64), (65, 72, 200), (128, 256, 256),
         (129, 136, 1032), (255, 264, 520), (256, 512, 128), (257, 1032, 136), (777, 1336, 2040),
         (1000, 128, 1024), (2048, 256, 384)]


# the kernel for few tokens: borders of its token tiles and of its tiles of weights
FEW = [(2, 128, 64), (15, 72, 72), (16, 128, 128), (17, 64, 8), (32, 1544, 136), (33, 8, 1000), (64, 2048, 2048),
       (65, 520, 3000), (127, 136, 264), (128, 4096, 1024), (128, 40, 56), (8, 8704, 512), (1, 8704, 10240)]


@pytest.mark.parametrize("mode", [0, 1, 2, 3])
@pytest.mark.parametrize("T,d,F", SIZES + FEW)
def test_forward(T, d, F, mode):
    gh.lib()
    x, w = block(T, d, F, seed=T + d + F)
    g, u, h, y = formula(x, w)
    m = capi.GatedFFN(d, F, max_tokens=T)
    m.set_sm_pairs(mode)
    got = m.forward(x, **w, save=True)
    assert m.status() == 0
    for t, want, n in ((got[1], g, "w_g"), (got[2], u, "w_u")):
        size = x.double().abs() @ w[n].double().abs().T
        assert bool(((t.double() - want).abs() <= R * want.abs() + (d + 4) * 2.0 ** -24 * size).all())
    check(got[0], y, h.abs() @ w["w_d"].double().abs().T, F)
    assert torch.equal(m.forward(x, **w), got[0])
    assert torch.equal(m.forward(x, **w, save=True)[1], got[1])
    assert m.status() == 0


@pytest.mark.parametrize("mode", [0, 1, 2, 3])
@pytest.mark.parametrize("T,d,F", SIZES + FEW)
def test_backward(T, d, F, mode):
    gh.lib()
    x, w = block(T, d, F, seed=T + d + F)
    gate, up, dy = rand((T, F), 1), rand((T, F), 2), rand((T, d), 3, 1e-2)
    m = capi.GatedFFN(d, F, max_tokens=T, training=True)
    m.set_sm_pairs(mode)
    got = m.backward(dy, x, gate, up, **w)
    assert m.status() == 0
    want = gradients(dy, x, gate, up, w)
    for n in want:
        check(got[n], *want[n])
    again = m.backward(dy, x, gate, up, **w)
    assert all(torch.equal(again[n], got[n]) for n in got)
    f32 = m.backward(dy, x, gate, up, **w, dw_dtype=F32)
    for n in ("dw_g", "dw_u", "dw_d"):
        assert f32[n].dtype == F32
        check(f32[n], *want[n], out=F32)
        assert torch.equal(f32[n].to(BF16), got[n])
    total = {n: f32[n].clone() for n in ("dw_g", "dw_u", "dw_d")}
    twice = m.backward(dy, x, gate, up, **w, out=total, accumulate=True)
    for n in total:
        assert twice[n] is total[n] and torch.equal(total[n], f32[n] + f32[n])
    assert torch.equal(twice["dx"], got["dx"])
    for need in (("dx",), ("dw_d",), ("dw_g", "dw_u"), ("dw_u",)):
        some = m.backward(dy, x, gate, up, **w, need=need)
        assert set(some) == set(need) and all(torch.equal(some[n], got[n]) for n in need)
    assert m.status() == 0


def test_extreme_gates():
    """Gates far out on both sides: SiLU and its derivative go to g and 1, and to 0."""
    gh.lib()
    T, d, F = 40, 64, 512
    _, w = block(T, d, F)
    x, dy, up = rand((T, d), 5), rand((T, d), 6), rand((T, F), 7)
    gate = rand((T, F), 8, 40.0)
    gate[0] = 300.0
    gate[1] = -300.0
    gate[2] = 0.0
    m = capi.GatedFFN(d, F, max_tokens=T, training=True)
    got = m.backward(dy, x, gate, up, **w)
    for n, want in gradients(dy, x, gate, up, w).items():
        check(got[n], *want)
    x = x * 100
    g, u, h, y = formula(x, w)
    check(m.forward(x, **w), y, h.abs() @ w["w_d"].double().abs().T, F)


def test_rows_of_wider_tensors_and_fewer_than_the_most():
    """Strided rows in and out; T below max_tokens; what lies beside and behind the rows
    is NaN and neither read nor written."""
    gh.lib()
    T, d, F = 150, 264, 328
    x, w = block(T, d, F)
    dy, gate, up = rand((T, d), 3, 1e-2), rand((T, F), 4), rand((T, F), 5)
    m = capi.GatedFFN(d, F, max_tokens=400, training=True)
    first = capi.GatedFFN(d, F, max_tokens=T, training=True)
    y = first.forward(x, **w)
    grads = first.backward(dy, x, gate, up, **w)
    # fill the workspace beyond T with something else
    m.forward(rand((400, d), 9, 1e4), **w)
    m.backward(rand((400, d), 9, 1e4), rand((400, d), 9), rand((400, F), 9), rand((400, F), 9), **w)

    def wide(t):
        big = torch.full((T + 50, t.shape[1] + 24), float("nan"), device="cuda", dtype=BF16)
        big[:T, 8:8 + t.shape[1]] = t
        return big, big[:T, 8:8 + t.shape[1]]

    bx, vx = wide(x)
    bdy, vdy = wide(dy)
    by, vy = wide(torch.zeros((T, d)))
    bdx, vdx = wide(torch.zeros((T, d)))
    for mode in (0, 1, 2, 3):
        m.set_sm_pairs(mode)
        first.set_sm_pairs(mode)
        m.forward(vx, **w, out=vy)
        assert torch.equal(vy, first.forward(x, **w))
        got = m.backward(vdy, vx, gate, up, **w, out={"dx": vdx})
        assert all(torch.equal(got[n], v) for n, v in first.backward(dy, x, gate, up, **w).items())
        for b in (by, bdx):
            assert int(b.isnan().sum()) == b.numel() - T * d
    assert m.status() == 0 and y.isfinite().all() and all(v.isfinite().all() for v in grads.values())


@pytest.mark.parametrize("T", [5, 200])
def test_bad_rows_stay_their_own(T):
    gh.lib()
    d, F = 136, 264
    x, w = block(T, d, F)
    dy, gate, up = rand((T, d), 3, 1e-2), rand((T, F), 4), rand((T, F), 5)
    m = capi.GatedFFN(d, F, max_tokens=T, training=True)
    y, dx = m.forward(x, **w), m.backward(dy, x, gate, up, **w)["dx"]
    keep = [i for i in range(T) if i != 3]
    for bad in (float("nan"), float("inf")):
        x2, dy2 = x.clone(), dy.clone()
        x2[3, 7] = bad
        dy2[3, 100] = bad
        y2 = m.forward(x2, **w)
        assert torch.equal(y2[keep], y[keep]) and bool(y2[3].isnan().any())
        dx2 = m.backward(dy2, x, gate, up, **w)["dx"]
        assert torch.equal(dx2[keep], dx[keep]) and bool(dx2[3].isnan().any())


def test_stream_and_graph():
    gh.lib()
    T, d, F = 200, 256, 512
    x, w = block(T, d, F)
    dy = rand((T, d), 3, 1e-2)
    m = capi.GatedFFN(d, F, max_tokens=T, training=True)
    y, gate, up = m.forward(x, **w, save=True)
    grads = m.backward(dy, x, gate, up, **w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, gate2, up2 = m.forward(x, **w, save=True, stream=side)
    grads2 = m.backward(dy, x, gate2, up2, **w, stream=side)
    side.synchronize()
    assert torch.equal(y2, y) and all(torch.equal(grads2[n], grads[n]) for n in grads)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hy, hgate, hup = m.forward(x, **w, save=True)
        held = m.backward(dy, x, hgate, hup, **w)
    for seed in (5, 6):
        x.copy_(rand((T, d), seed))
        w["w_u"].copy_(rand((F, d), seed + 1, d ** -0.5))
        g.replay()
        held_now = {n: v.clone() for n, v in held.items()}
        y, gate, up = m.forward(x, **w, save=True)
        assert torch.equal(hy, y) and torch.equal(hgate, gate) and torch.equal(hup, up)
        now = m.backward(dy, x, gate, up, **w)
        assert all(torch.equal(held_now[n], now[n]) for n in now)
    assert m.status() == 0


def test_two_handles_at_once():
    """Handles share nothing: calls of every kernel on two streams at the same time."""
    gh.lib()
    d, F = 264, 520
    sets = []
    for i, T in enumerate((5, 16, 100, 700)):
        x, w = block(T, d, F, seed=10 * i)
        dy, gate, up = rand((T, d), i + 1, 1e-2), rand((T, F), i + 2), rand((T, F), i + 3)
        two = [capi.GatedFFN(d, F, max_tokens=T, training=True) for _ in range(2)]
        want = (two[0].forward(x, **w), two[0].backward(dy, x, gate, up, **w))
        sets.append((x, w, dy, gate, up, two, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for x, w, dy, gate, up, two, want in sets:
            for m, st in zip(two, streams):
                got.append((m.forward(x, **w, stream=st), m.backward(dy, x, gate, up, **w, stream=st), want))
    torch.cuda.synchronize()
    for y, g, want in got:
        assert torch.equal(y, want[0]) and all(torch.equal(g[n], want[1][n]) for n in g)
    assert all(m.status() == 0 for s in sets for m in s[5])


def test_against_differences():
    """sum(dy y) in float64 along the gradient's own direction, for x and each weight:
    central differences are exact to 1e-6 here (h 1e-4); the gradient's own roundings
    (TOL) and those of the gate and up that the forward stored (R of each, which move
    dg, du and h by at most 3 R) leave 2e-2 of its norm."""
    gh.lib()
    T, d, F = 24, 64, 96
    x, w = block(T, d, F)
    dy = rand((T, d), 3)
    m = capi.GatedFFN(d, F, max_tokens=T, training=True)
    y, gate, up = m.forward(x, **w, save=True)
    got = m.backward(dy, x, gate, up, **w)
    at = {"x": x.double(), **{n: v.double() for n, v in w.items()}}

    def loss(p):
        return float((dy.double() * formula(p["x"], p)[3]).sum())

    for n in ("x", "w_g", "w_u", "w_d"):
        grad = got["dx" if n == "x" else "d" + n].double()
        v = grad / grad.norm()
        h = 1e-4
        diff = (loss({**at, n: at[n] + h * v}) - loss({**at, n: at[n] - h * v})) / (2 * h)
        assert abs(diff - float(grad.norm())) <= 2e-2 * float(grad.norm())


def test_refusals():
    lib = gh.lib()
    T, d, F = 16, 64, 128
    x, w = block(T, d, F)
    dy, gate, up = rand((T, d), 3), rand((T, F), 4), rand((T, F), 5)
    m = capi.GatedFFN(d, F, max_tokens=T)
    with pytest.raises(capi.LatentMoEError) as e:
        m.backward(dy, x, gate, up, **w)
    assert e.value.code == capi.ERR_INVALID_ARG  # not made for training
    m = capi.GatedFFN(d, F, max_tokens=T, training=True)
    with pytest.raises(capi.LatentMoEError):
        m.forward(rand((T + 1, d), 1), **w)  # past max_tokens
    with pytest.raises(capi.LatentMoEError):
        m.forward(x[:0], **w)
    for bad in (dict(x=x.float()), dict(x=x[:, :32]), dict(x=x.T), dict(x=x[:1].expand(T, d)),
                dict(w_g=w["w_d"]), dict(w_d=w["w_d"].float()), dict(w_u=w["w_u"].T.contiguous().T),
                dict(x=x.cpu())):
        with pytest.raises(ValueError):
            m.forward(**{"x": x, **w, **bad})
    odd = torch.zeros(T * d + 1, device="cuda", dtype=BF16)[1:].view(T, d)
    with pytest.raises(capi.LatentMoEError) as e:
        m.forward(odd, **w)
    assert e.value.code == capi.ERR_UNSUPPORTED
    with pytest.raises(capi.LatentMoEError) as e:
        m.forward(rand((T, d + 4), 1)[:, :d], **w)
    assert e.value.code == capi.ERR_UNSUPPORTED
    out = {"dw_g": torch.zeros((F, d), device="cuda", dtype=BF16), "dw_u": torch.zeros((F, d), device="cuda", dtype=BF16),
           "dw_d": torch.zeros((d, F), device="cuda", dtype=BF16)}
    with pytest.raises(capi.LatentMoEError) as e:
        m.backward(dy, x, gate, up, **w, out=out, accumulate=True)
    assert e.value.code == capi.ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        m.backward(dy, x, gate, up, **w, accumulate=True)
    with pytest.raises(ValueError):
        m.backward(dy, x, gate[:, :64], up, **w)
    with pytest.raises(capi.LatentMoEError):
        m.backward(dy, x, gate, up, **w, need=())
    # the C entries with something missing
    cw = capi.latentmoe_ffn_weights(*(w[n].data_ptr() for n in ("w_g", "w_u", "w_d")))
    some = capi.latentmoe_ffn_weights(w["w_g"].data_ptr(), None, w["w_d"].data_ptr())
    y = torch.empty_like(x)
    call = lambda cw, gate, up, T: lib.latentmoe_ffn_forward(  # noqa: E731
        m.handle, ctypes.byref(cw), x.data_ptr(), 0, y.data_ptr(), 0, gate, up, T, None)
    assert call(some, None, None, T) == capi.ERR_INVALID_ARG
    assert call(cw, gate.data_ptr(), None, T) == capi.ERR_INVALID_ARG
    assert call(cw, None, None, 0) == capi.ERR_INVALID_ARG
    assert m.status() == 0
