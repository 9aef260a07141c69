"""Newton-Schulz orthogonalisation and the optimiser step around it, against
the iteration in float64.

Tolerance of the result (2-norm, relative). The output's rounding to bf16 adds
at most 2^-8 of an entry. Operands are fp16: every entry of X, A and P is off
by at most 2^-11 of itself, as an independent error of at most 2^-11 / sqrt(3)
in the mean square. To first order a step's result moves by the rounding of A
(entering through b A + 2 c A^2), of P and of X, each weighted by at most
|b| s^3 + 2 |c| s^5 <= 9 at s = 1.2 for errors spread over all directions, but
an error of relative size e in a symmetric m x m factor of norm about sqrt(m)
has a 2-norm per direction of e only; the iteration's derivative at its
attracting interval is below 1 in the mean, so five steps add up to at most
5 * 3 * 2^-11 / sqrt(3) = 4.2e-3. Together 4.2e-3 + 2^-8 / sqrt(3) = 6.5e-3.
"""
import numpy as np
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


SIZES = [(1, 1, 1), (1, 1, 200), (1, 200, 1), (2, 7, 5), (1, 64, 64), (1, 128, 128), (3, 129, 130),
         (1, 130, 129), (2, 100, 700), (2, 700, 100), (1, 64, 2048), (1, 513, 1025),
         (1, 1025, 513), (4, 256, 384), (1, 777, 1333)]


@pytest.mark.parametrize("pairs", [0, 1, 2])
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
