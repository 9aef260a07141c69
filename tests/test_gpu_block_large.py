"""Offsets past 32 bits: tensors of more than 2^31 elements, checked by their first, middle
and last rows against the same call on those rows alone (norm, gated block: a row's result
depends on its own row) and against float64 (clipping)."""
import pytest
import torch

from mixture_experts_layer_router_gb300 import capi
import gpu_helpers as gh

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def rows_of(T):
    return torch.tensor([0, 1, T // 2 - 1, T // 2, T - 2, T - 1], device="cuda")


def fill(T, d, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty((T, d), device="cuda", dtype=BF16)
    for part in x.split(1 << 14):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * scale)
    return x


def test_norm_and_backward():
    gh.lib()
    T, d = 140_000, 16_384
    x, w = fill(T, d, 1), torch.rand(d, device="cuda") + 0.5
    r = rows_of(T)
    got = capi.rms_norm(x, w, quantize="block", keep_y=True)
    few = capi.rms_norm(x[r], w, quantize="block", keep_y=True)
    for n in few:
        assert torch.equal(got[n][r], few[n])
    rstd = got["rstd"]
    del got
    b = capi.rms_norm_backward(x, x, w, rstd, d_sum=x)
    few = capi.rms_norm_backward(x[r], x[r], w, rstd[r], d_sum=x[r], dw=False)
    assert torch.equal(b["dx"][r], few["dx"])
    # dw = sum of x^2 rstd over the rows: each term is within 2 u of itself, at most 1100 in
    # a row with one another, all positive
    want = torch.zeros(d, device="cuda", dtype=torch.float64)
    for a, s in zip(x.split(1 << 13), rstd.split(1 << 13)):
        want += (a.double().square() * s.double()[:, None]).sum(0)
    assert bool(((b["dw"].double() - want).abs() <= 1200 * 2.0 ** -24 * want).all())


def test_clip():
    gh.lib()
    n = (1 << 31) + 12_345
    g = fill(1 << 17, 1 << 14, 2, 1e-3).view(-1)
    g = torch.cat([g, g[:12_345]])
    assert g.numel() == n
    total = sum(float(p.double().square().sum()) for p in g.split(1 << 28)) ** 0.5
    head, tail = g[:1000].clone(), g[-1000:].clone()
    norm = capi.clip_gradients([g], total / 4)
    assert abs(float(norm) - total) <= 24 * 2.0 ** -24 * total
    for a, b in ((g[:1000], head), (g[-1000:], tail)):
        want = b.double() * (total / 4 / (total + 1e-6))
        assert bool(((a.double() - want).abs() <= (2.0 ** -8 + 1e-5) * want.abs()).all())


def test_gated_block():
    gh.lib()
    T, d, F = 270_000, 64, 8192
    x, dy = fill(T, d, 3), fill(T, d, 4, 1e-2)
    w = {"w_g": fill(F, d, 5, d ** -0.5), "w_u": fill(F, d, 6, d ** -0.5), "w_d": fill(d, F, 7, F ** -0.5)}
    m = capi.GatedFFN(d, F, max_tokens=T, training=True)
    m.set_sm_pairs(1)
    r = rows_of(T)
    y, gate, up = m.forward(x, **w, save=True)
    dx = m.backward(dy, x, gate, up, **w, need=("dx",))["dx"]
    # the same k order whatever the number of rows: equal bits (8 rows: operands unpadded)
    r8 = torch.cat([r, r[:2]])
    few = capi.GatedFFN(d, F, max_tokens=8, training=True)
    few.set_sm_pairs(1)
    y8, gate8, up8 = few.forward(x[r8], **w, save=True)
    assert torch.equal(y[r8], y8) and torch.equal(gate[r8], gate8) and torch.equal(up[r8], up8)
    assert torch.equal(dx[r8], few.backward(dy[r8], x[r8], gate8, up8, **w, need=("dx",))["dx"])
    assert m.status() == 0 and few.status() == 0
