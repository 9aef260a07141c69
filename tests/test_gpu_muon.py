"""Newton-Schulz orthogonalisation and the optimiser step around it, against
the iteration in float64.

Tolerance of the result (2-norm, relative): the output's rounding to bf16, at
most 2^-8 of an entry and 2^-8 / sqrt(3) in the mean square, and the fp16
operands, each entry of X, A' and P' off by at most 2^-11 of itself. A step
passes an error of relative size e in one of its three operands on with a factor
of order one (|p'| <= 3.4, and below one where the singular values gather), so
five steps add up to at most 5 * 3 * 2^-11 / sqrt(3) = 4.2e-3: TOL = 6.5e-3.
Matrices of low rank plus noise are held to the same: their small directions are
the sharpest test of the kept 32-bit X. The updated weights are off by lr * scale
times that, plus their own rounding; the momentum is two fp32 roundings, exactly
those of torch.
"""
import ctypes

import pytest
import torch

from mixture_experts_layer_router_gb300 import capi
import gpu_helpers as gh

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.7750, 2.0315)
TOL = 6.5e-3


def newton_schulz(u, coefs=(COEF,) * 5, eps=1e-7):
    """float64 iteration on a stack [..., rows, cols]."""
    x = u.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    for a, b, c in coefs:
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.mT if tall else x


def rand(shape, seed, kind="normal"):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=gen, device="cuda")
    if kind == "lowrank":
        r = 8
        x = 0.1 * x + torch.randn(shape[:-1] + (r,), generator=gen, device="cuda") @ \
            torch.randn(shape[:-2] + (r, shape[-1]), generator=gen, device="cuda")
    return x


def rel(x, y):
    return float((x.double() - y).norm() / y.norm())


# short sides of 128 and 129, long sides of 4096 and 4097: the border of the
# one-launch kernel; 256 / 257 columns: one and two of its CTAs
SIZES = [(1, 1, 1), (1, 1, 200), (1, 200, 1), (2, 7, 5), (1, 64, 64), (1, 128, 128), (3, 129, 130),
         (1, 130, 129), (2, 100, 700), (2, 700, 100), (1, 64, 2048), (1, 513, 1025),
         (1, 1025, 513), (4, 256, 384), (1, 777, 1333),
         (3, 128, 257), (2, 16, 4096), (1, 4097, 33), (5, 100, 256), (2, 31, 2049),
         (1, 256, 256), (1, 130, 4100)]


@pytest.mark.parametrize("pairs", [0, 1, 2, 3])
@pytest.mark.parametrize("batch,rows,cols", SIZES)
def test_orthogonalize(batch, rows, cols, pairs):
    gh.lib()
    m = capi.Muon(rows, cols, batch=batch)
    m.set_sm_pairs(pairs)
    for dt in (torch.bfloat16, torch.float32):
        g = rand((batch, rows, cols), rows * 31 + cols).mul_(1e-3).to(dt)
        o = m.orthogonalize(g)
        assert m.status() == 0
        assert o.shape == g.shape and o.dtype == torch.bfloat16
        assert rel(o, newton_schulz(g)) <= TOL
        assert torch.equal(o, m.orthogonalize(g))


@pytest.mark.parametrize("batch,rows,cols", [(2, 96, 640), (2, 640, 96), (1, 512, 768),
                                             (1, 768, 512), (1, 1024, 1024)])
def test_low_rank_and_rank_deficient(batch, rows, cols):
    gh.lib()
    m = capi.Muon(rows, cols, batch=batch)
    for kind, seed in (("lowrank", 3), ("lowrank", 4)):
        g = rand((batch, rows, cols), seed, kind)
        assert rel(m.orthogonalize(g), newton_schulz(g)) <= TOL
    # an exact outer product: one direction, the rest exactly zero
    g = torch.zeros((batch, rows, cols), device="cuda")
    g[:, 3, 5] = 2.0
    o = m.orthogonalize(g)
    assert rel(o, newton_schulz(g)) <= TOL
    assert int((o != 0).sum()) == batch


@pytest.mark.parametrize("rows,cols", [(64, 300), (300, 64), (200, 300), (300, 200)])
def test_zeros_nan_and_infinity_stay_in_their_matrix(rows, cols):
    gh.lib()
    m = capi.Muon(rows, cols, batch=5)
    g = rand((5, rows, cols), 9)
    clean = m.orthogonalize(g)
    g2 = g.clone()
    g2[1] = 0
    g2[2, rows - 1, 0] = float("nan")
    g2[3, 0, cols - 1] = float("inf")
    o = m.orthogonalize(g2)
    assert torch.equal(o[0], clean[0]) and torch.equal(o[4], clean[4])
    assert torch.equal(o[1], torch.zeros_like(o[1]))
    assert torch.isnan(o[2]).all()
    assert torch.isnan(o[3]).any()
    # and nothing of it is left behind
    assert torch.equal(m.orthogonalize(g), clean)
    assert m.status() == 0


# few tiles and a long side: the first product of a step is split over its k
@pytest.mark.parametrize("pairs", [0, 2, 3])
@pytest.mark.parametrize("batch,rows,cols", [(1, 256, 7168), (1, 7168, 256), (2, 33, 4200),
                                             (1, 200, 2000), (3, 150, 1025), (1, 8704, 64),
                                             (1, 1, 20000), (7, 260, 1600)])
def test_long_sides(batch, rows, cols, pairs):
    gh.lib()
    m = capi.Muon(rows, cols, batch=batch)
    m.set_sm_pairs(pairs)
    g = rand((batch, rows, cols), rows + cols).to(torch.bfloat16)
    o = m.orthogonalize(g)
    assert m.status() == 0
    assert rel(o, newton_schulz(g)) <= TOL
    for _ in range(3):  # the sum does not depend on which part comes last
        assert torch.equal(o, m.orthogonalize(g))
    bad = g.clone()
    bad[batch - 1, rows - 1, cols - 1] = float("nan")
    x = m.orthogonalize(bad)
    assert torch.equal(x[:-1], o[:-1]) and torch.isnan(x[-1]).all()


@pytest.mark.parametrize("rows,cols", [(100, 300), (300, 200)])
@pytest.mark.parametrize("scale", [1e-15, 1e-6, 1.0, 1e12])
def test_scale_of_the_update(rows, cols, scale):
    """Scale drops out while the norm is far above eps, and the small norms below
    eps shrink X as the definition says."""
    gh.lib()
    m = capi.Muon(rows, cols)
    g = rand((1, rows, cols), 21) * scale
    assert rel(m.orthogonalize(g), newton_schulz(g)) <= TOL


@pytest.mark.parametrize("rows,cols", [(64, 200), (260, 200)])
@pytest.mark.parametrize("coefs", [
    [COEF], [COEF] * 2, [COEF] * 9, [(1.5, -0.5, 0.0)] * 8, [(15 / 8, -10 / 8, 3 / 8)] * 7,
    [(1.0, 0.0, 0.0)] * 3,
    [(4.0, -6.0, 2.5), (3.0, -4.0, 1.5), (1.875, -1.25, 0.375)]])
def test_coefficients_and_steps(rows, cols, coefs):
    """Few and many steps, classical and mixed coefficients; nine steps let the
    errors of nine add up: 9/5 of the tolerance's part."""
    gh.lib()
    m = capi.Muon(rows, cols, steps=len(coefs), coefs=coefs)
    g = rand((1, rows, cols), 33)
    assert rel(m.orthogonalize(g), newton_schulz(g, coefs)) <= TOL * max(1.0, len(coefs) / 5)


def test_default_coefficients():
    gh.lib()
    g = rand((1, 100, 120), 2)
    a = capi.Muon(100, 120).orthogonalize(g)
    b = capi.Muon(100, 120, steps=5, coefs=COEF).orthogonalize(g)
    assert torch.equal(a, b)


@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (3, 64, 300), (2, 300, 64), (1, 333, 257),
                                             (2, 256, 512), (1, 514, 130)])
@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
def test_step(batch, rows, cols, gdt, wdt):
    gh.lib()
    h = capi.Muon(rows, cols, batch=batch)
    lr, mu, wd, scale = 0.05, 0.9, 0.1, 0.7
    w = rand((batch, rows, cols), 1).mul_(0.1).to(wdt)
    m = rand((batch, rows, cols), 2).mul_(1e-3)
    for it, nesterov in enumerate((True, False, True)):
        g = rand((batch, rows, cols), 3 + it).mul_(1e-3).to(gdt)
        w0, m0 = w.double(), m.clone()
        h.step(w, g, m, lr=lr, momentum_coef=mu, weight_decay=wd, scale=scale, nesterov=nesterov)
        want_m = m0.mul(mu).add(g.float())
        assert torch.equal(m, want_m)
        u = g.double() + mu * want_m.double() if nesterov else want_m.double()
        x = newton_schulz(u)
        want = w0 * (1 - lr * wd) - lr * scale * x
        err = (w.double() - want).norm()
        half_step = 2.0 ** -8 if wdt == torch.bfloat16 else 2.0 ** -23
        assert float(err) <= float(lr * scale * 4.2e-3 * x.norm() + half_step * want.norm())
    assert h.status() == 0


def test_in_place_and_no_batch_dimension():
    gh.lib()
    for rows, cols in ((64, 200), (200, 300)):
        m = capi.Muon(rows, cols)
        g = rand((rows, cols), 8).to(torch.bfloat16)
        want = m.orthogonalize(g)
        assert want.shape == (rows, cols)
        assert m.orthogonalize(g, out=g) is g
        assert torch.equal(g, want)


def test_launch_counts():
    gh.lib()
    g = rand((1, 128, 256), 1)
    m = capi.Muon(128, 256)
    m.orthogonalize(g)
    assert m.launch_count() == 1
    m.set_sm_pairs(0)
    m.orthogonalize(g)
    assert m.launch_count() == 4
    m = capi.Muon(129, 256)
    m.orthogonalize(rand((1, 129, 256), 1))
    assert m.launch_count() == 3


@pytest.mark.parametrize("batch,rows,cols", [(1, 64, 2048), (3, 300, 500), (40, 256, 256)])
def test_streams_and_graphs(batch, rows, cols):
    gh.lib()
    m = capi.Muon(rows, cols, batch=batch)
    g = rand((batch, rows, cols), 5).to(torch.bfloat16)
    want = m.orthogonalize(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = m.orthogonalize(g)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.orthogonalize(g)
    for seed in (6, 7):
        g.copy_(rand((batch, rows, cols), seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, m.orthogonalize(g))
    assert m.status() == 0


def test_back_to_back_calls_and_two_handles():
    """Calls that nothing waits between, and two handles on two streams."""
    gh.lib()
    a, b = capi.Muon(300, 500, batch=2), capi.Muon(64, 700)
    ga = [rand((2, 300, 500), i) for i in range(4)]
    gb = [rand((1, 64, 700), 10 + i) for i in range(4)]
    wa = [a.orthogonalize(g) for g in ga]
    wb = [b.orthogonalize(g) for g in gb]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    oa = [a.orthogonalize(g, stream=s1) for g in ga]
    ob = [b.orthogonalize(g, stream=s2) for g in gb]
    torch.cuda.synchronize()
    for x, y in zip(wa + wb, oa + ob):
        assert torch.equal(x, y)
    assert a.status() == 0 and b.status() == 0


def test_refusals():
    lib = gh.lib()
    m = capi.Muon(32, 48, batch=2)
    g = rand((2, 32, 48), 1)
    o = torch.empty((2, 32, 48), dtype=torch.bfloat16, device="cuda")
    hd, p, q = m.handle, g.data_ptr(), o.data_ptr()
    f = lib.latentmoe_muon_orthogonalize
    assert f(hd, None, 1, q, None) == f(hd, p, 1, None, None) == capi.ERR_INVALID_ARG
    assert f(hd, p, 2, q, None) == f(hd, p, -1, q, None) == capi.ERR_INVALID_ARG
    assert f(hd, p + 4, 1, q, None) == f(hd, p, 1, q + 2, None) == capi.ERR_UNSUPPORTED
    w, mo = torch.zeros_like(g), torch.zeros_like(g)
    base = dict(g=p, momentum=mo.data_ptr(), w=w.data_ptr(), g_dtype=1, w_dtype=1, nesterov=1,
                lr=0.1, momentum_coef=0.9, weight_decay=0.0, scale=1.0)

    def step(**kw):
        return lib.latentmoe_muon_step(hd, ctypes.byref(capi.latentmoe_muon_update(
            **{**base, **kw})), None)

    assert step() == capi.OK
    for bad in (dict(g=None), dict(momentum=None), dict(w=None), dict(g_dtype=3),
                dict(w_dtype=-1), dict(lr=float("nan")), dict(scale=float("inf")),
                dict(momentum_coef=float("nan")), dict(weight_decay=float("inf"))):
        assert step(**bad) == capi.ERR_INVALID_ARG, bad
    assert step(w=w.data_ptr() + 4) == step(momentum=mo.data_ptr() + 8) == capi.ERR_UNSUPPORTED
    assert lib.latentmoe_muon_step(hd, None, None) == capi.ERR_INVALID_ARG
    for mode in (-1, 4):
        assert lib.latentmoe_muon_set_sm_pairs(hd, mode) == capi.ERR_INVALID_ARG
    torch.cuda.synchronize()
    for bad in (g[0], g.half(), g.cpu(), g.mT, g[:, :, :40]):
        with pytest.raises(ValueError):
            m.orthogonalize(bad)
    with pytest.raises(ValueError):
        m.orthogonalize(g, out=torch.empty_like(g))
    with pytest.raises(ValueError):
        m.step(w, g, mo.bfloat16(), lr=0.1)
    assert m.status() == 0


def test_offsets_beyond_32_bits():
    """A stack of more than 2^31 elements: its first and last matrices are right,
    the zeros between stay zero."""
    gh.lib()
    batch, side = 1100, 1400
    assert batch * side * side > 2 ** 31
    m = capi.Muon(side, side, batch=batch)
    g = torch.zeros((batch, side, side), dtype=torch.bfloat16, device="cuda")
    for b in (0, batch - 1):
        g[b] = rand((side, side), 50 + b).to(torch.bfloat16)
    o = m.orthogonalize(g)
    assert m.status() == 0
    for b in (0, batch - 1):
        assert rel(o[b], newton_schulz(g[b])) <= TOL
    assert not bool(o[1:batch - 1].any())


def test_output_of_another_stream_does_not_take_memory_in_use():
    m = capi.Muon(300, 200)
    g = rand((300, 200), 3)
    want = m.orthogonalize(g)
    torch.empty_like(want).fill_(7.0)  # loads the fill kernel
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # 10 ms at 2 GHz
    late = [torch.empty_like(want).fill_(7.0) for _ in range(4)]
    del late
    o = m.orthogonalize(g, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, want)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,rows,cols", [(1, 100, 304), (2, 300, 104), (2, 128, 512), (1, 33, 131),
                                             (2, 304, 200), (1, 200, 333), (1, 333, 201)])
def test_small_updates_with_a_small_eps(batch, rows, cols, dt):
    """The smallest eps that is taken, and updates whose squares are no fp32 numbers."""
    gh.lib()
    m = capi.Muon(rows, cols, batch=batch, eps=1e-30)
    x = rand((batch, rows, cols), 37)
    few = torch.zeros_like(x)
    few[:, ::7, ::5] = 1e13  # some entries far above the others
    for g in (x * 1e-18, x * 1e-20, x * 1e-22, x * 1e-24, x * 1e-28, x * 1e-31, x * 1e-34,
              x * 1e-24 + few * x * 1e-24, x):
        g = g.to(dt)
        assert rel(m.orthogonalize(g), newton_schulz(g, eps=1e-30)) <= TOL
    w, mo = torch.zeros_like(x), torch.zeros_like(x)
    g = (x * 1e-24).to(dt)
    m.step(w, g, mo, lr=1.0, momentum_coef=0.5, nesterov=True)
    want = -newton_schulz(g.double() * 1.5, eps=1e-30)
    assert rel(w, want) <= TOL
    zero = torch.zeros_like(g)
    assert torch.equal(m.orthogonalize(zero), torch.zeros_like(x, dtype=torch.bfloat16))
    assert m.status() == 0
