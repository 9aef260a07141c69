"""Global gradient norm and clipping against float64.

Tolerances. u = 2^-24. A thread adds at most 64 squares of a tile in fp32 (one rounding
each; eight sums of eight, so no number goes through more than 16 additions), then
compensated fp32 and 64-bit sums: below 38 u of the sum, 19 u of the norm, and its own
rounding. NORM = 24 u. The factor is as
exact, and a product is rounded once: half a step of the type.
"""
import ctypes

import pytest
import torch

from mixture_experts_layer_router_gb300 import capi
import gpu_helpers as gh

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NORM = 24 * U
BF16, F32 = torch.bfloat16, torch.float32


def rand(n, seed, dtype, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=gen, device="cuda") * scale).to(dtype)


def true_norm(grads):
    return sum(float(g.double().square().sum()) for g in grads) ** 0.5


def check(grads, over, eps=1e-6):
    norm = true_norm(grads)
    max_norm = norm / over
    before = [g.clone() for g in grads]
    got = capi.gradient_norm(grads)
    assert got.shape == (1,) and got.dtype == F32
    assert abs(float(got) - norm) <= NORM * norm
    out = [torch.full_like(g, 7.0) for g in grads]
    n = capi.clip_gradients(grads, max_norm, eps=eps, out=out)
    assert torch.equal(n, got)
    for g, b in zip(grads, before):
        assert torch.equal(g, b)
    c = min(1.0, max_norm / (norm + eps)) if norm > 0 else 1.0
    for g, o in zip(grads, out):
        want = g.double() * c
        tol = torch.finfo(g.dtype).eps / 2 + 2 * NORM
        assert bool(((o.double() - want).abs() <= tol * want.abs() + 1e-40).all())
    n = capi.clip_gradients(grads, max_norm, eps=eps)
    assert torch.equal(n, got)
    for g, o in zip(grads, out):
        assert torch.equal(g, o)


@pytest.mark.parametrize("sizes", [
    [1], [2], [7], [8], [9], [16385], [32768], [32769], [100000, 3, 0, 1], [0, 5, 0], [5_000_001],
    [300_000] * 31, [17] * 30, [17] * 31, [1, 2, 3, 4, 5, 6, 7, 8, 9] * 20])
@pytest.mark.parametrize("types", ["bf16", "f32", "mixed"])
def test_norm_and_clip(sizes, types):
    gh.lib()
    kinds = {"bf16": [BF16], "f32": [F32], "mixed": [BF16, F32]}[types]
    grads = [rand(n, 11 * i + n, kinds[i % len(kinds)], 1e-2) for i, n in enumerate(sizes)]
    check(grads, 3.0)


def test_not_clipped_below_the_limit():
    gh.lib()
    grads = [rand(n, n, t) for n, t in ((1000, BF16), (33, F32), (70_000, F32))]
    before = [g.clone() for g in grads]
    norm = true_norm(grads)
    out = [torch.empty_like(g) for g in grads]
    capi.clip_gradients(grads, 1.01 * norm, out=out)
    capi.clip_gradients(grads, 1.01 * norm)
    capi.clip_gradients(grads, float("inf"))
    for g, b, o in zip(grads, before, out):
        assert torch.equal(g, b) and torch.equal(o, b)
    capi.clip_gradients(grads, 0.0)
    assert all(bool((g == 0).all()) for g in grads)


def test_more_tensors_than_a_launch_takes():
    gh.lib()
    for count in (1000, 1001, 2345):
        grads = [rand(1 + i % 300, i, BF16 if i % 3 else F32) for i in range(count)]
        check(grads, 2.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_views_of_one_buffer(dtype):
    """Tensors that begin and end inside a 16-byte piece, next to one another: each is
    scaled once, and what is in no tensor stays; out aligned otherwise than g."""
    gh.lib()
    flat = rand(100_000, 1, dtype)
    cuts = [(0, 1), (1, 4), (5, 8), (13, 3), (17, 40_000), (40_018, 59_000)]
    grads = [flat[a:a + n] for a, n in cuts]
    want, norm = flat.double().clone(), true_norm(grads)
    c = 0.5 * norm / (norm + 1e-6)
    keep = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
    for a, n in cuts:
        want[a:a + n] *= c
        keep[a:a + n] = False
    before = flat.clone()
    other = torch.zeros(flat.numel() + 3, dtype=dtype, device="cuda")
    outs = [other[a + 3:a + 3 + n] for a, n in cuts]
    capi.clip_gradients(grads, 0.5 * norm, out=outs)
    capi.clip_gradients(grads, 0.5 * norm)
    tol = torch.finfo(dtype).eps / 2 + 2 * NORM
    assert bool(((flat.double() - want).abs() <= tol * want.abs())[~keep].all())
    assert torch.equal(flat[keep], before[keep])
    assert torch.equal(other[3:][~keep], flat[~keep])
    assert bool((other[:3] == 0).all()) and bool((other[3:][keep] == 0).all())


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-22, 1e-13, 1e12, 1e18, 1e24, 1e34])
def test_magnitudes(scale):
    """Numbers whose squares fp32 cannot hold, alone and among ordinary ones."""
    gh.lib()
    x = rand(50_000, 2, F32) * scale
    # 1e-38: subnormal entries, exact in fp32 and in the 64-bit sum
    norm = true_norm([x])
    assert abs(float(capi.gradient_norm([x])) - norm) <= NORM * norm + 1e-44
    y = rand(30_000, 3, BF16)
    both = true_norm([x, y])
    assert abs(float(capi.gradient_norm([x, y])) - both) <= NORM * both
    b = x.to(BF16)
    assert abs(float(capi.gradient_norm([b])) - true_norm([b])) <= NORM * true_norm([b]) + 1e-44


def test_zeros():
    gh.lib()
    grads = [torch.zeros(40_000, device="cuda"), torch.zeros(3, device="cuda", dtype=BF16)]
    assert float(capi.clip_gradients(grads, 1.0)) == 0.0
    assert float(capi.gradient_norm([torch.zeros(0, device="cuda")])) == 0.0
    assert float(capi.clip_gradients([torch.zeros(0, device="cuda")], 1.0)) == 0.0
    assert all(bool((g == 0).all()) for g in grads)


def test_not_finite():
    gh.lib()
    a, b = rand(5000, 1, BF16), rand(70_000, 2, F32)
    b[69_999] = float("nan")
    assert bool(capi.clip_gradients([a, b], 1.0).isnan())
    assert bool(a.isnan().all()) and bool(b.isnan().all())
    a, b = rand(5000, 1, BF16), rand(70_000, 2, F32)
    a[77] = float("-inf")
    assert float(capi.clip_gradients([a, b], 1.0)) == float("inf")
    assert bool(a[77].isnan()) and bool((b == 0).all())
    a[77] = 0
    assert bool((a == 0).all())


def test_stream_and_graph():
    gh.lib()
    grads = [rand(n, n, t) for n, t in ((1000, BF16), (33, F32), (700_000, F32))]
    norm = true_norm(grads)
    out = [torch.empty_like(g) for g in grads]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = capi.clip_gradients(grads, norm / 2, out=out, stream=side)
    side.synchronize()
    assert abs(float(n) - norm) <= NORM * norm
    g = torch.cuda.CUDAGraph()
    held = [torch.empty_like(x) for x in grads]
    with torch.cuda.graph(g):
        held_norm = capi.clip_gradients(grads, norm / 2, out=held)
    for k in (1.0, 0.25, 8.0):
        for x in grads:
            x.mul_(k)
        g.replay()
        n = capi.clip_gradients(grads, norm / 2, out=out)
        assert torch.equal(n, held_norm)
        assert all(torch.equal(a, b) for a, b in zip(out, held))


def test_two_streams_at_once():
    """Calls share nothing: many on two streams, with different tensors, each right."""
    gh.lib()
    sets = [[rand(200_000, i, F32), rand(70_001, i + 9, BF16)] for i in range(2)]
    norms = [true_norm(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            got[i].append(capi.gradient_norm(sets[i], stream=st))
    torch.cuda.synchronize()
    for g, n in zip(got, norms):
        assert all(abs(float(v) - n) <= NORM * n and float(v) == float(g[0]) for v in g)


def test_overlaps_are_refused():
    gh.lib()
    x = rand(1000, 1, F32)
    free = torch.empty(2000, device="cuda")
    before = x.clone()
    bad = [([x, x], None), ([x[:600], x[500:]], None), ([x[:500], x[500:]], [free[:500], free[499:999]]),
           ([x[:500]], [x[1:501]]), ([x[:300], x[300:600]], [x[300:600], x[:300]]),
           ([x[:300], x[300:600]], [free[:300], x[:300]])]
    for grads, out in bad:
        with pytest.raises(capi.LatentMoEError) as e:
            capi.clip_gradients(grads, 1.0, out=out)
        assert e.value.code == capi.ERR_INVALID_ARG
    assert torch.equal(x, before)
    # a norm may count a tensor twice, and empty tensors lie anywhere
    n = true_norm([x, x])
    assert abs(float(capi.gradient_norm([x, x])) - n) <= NORM * n
    capi.clip_gradients([x[:500], x[500:], x[400:400]], 1e9)
    assert torch.equal(x, before)
