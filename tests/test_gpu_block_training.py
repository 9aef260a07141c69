"""The block-training example: the norm, the gated block, their gradients, clipping and
Muon as a training program runs them, and the chain's gradients against torch's autograd
in float64.

Tolerance of the gradients (2-norm, relative). Along the chain these are rounded to bf16,
each by at most 2^-8 of an entry, 2^-8 / sqrt(3) = 2.3e-3 in the mean square: y, gate, up,
h, dg, du, d_out (and dx of the block for the norm's weight and x). A weight's gradient
meets at most seven of them, each with a factor of order one: sqrt(7) 2.3e-3 = 6e-3, of
order one meaning up to 2: TOL = 1.2e-2. The gradient of s holds d_out in fp32, so it is
closer.
"""
import os
import sys

import pytest
import torch

from mixture_experts_layer_router_gb300 import capi
import gpu_helpers as gh

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
TOL = 1.2e-2


def exact(weights, norm, batches):
    """Gradients of the mean loss over the batches, and of every batch's x, in float64."""
    p = {k: v.double().requires_grad_() for k, v in {**weights, "norm": norm}.items()}
    xs, loss = [], 0.0
    for x, stream, target in batches:
        x = x.double().requires_grad_()
        xs.append(x)
        s = x + stream.double()
        y = s * (s.square().mean(1, keepdim=True) + 1e-6).rsqrt() * p["norm"]
        gate = y @ p["w_g"].T
        out = (gate * torch.sigmoid(gate) * (y @ p["w_u"].T)) @ p["w_d"].T
        loss = loss + (s + out - target.double()).square().mean() / len(batches)
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in p.items()}, [x.grad for x in xs]


@pytest.mark.parametrize("T,d,F", [(96, 256, 512), (1, 64, 128), (5, 136, 72), (300, 200, 264)])
def test_gradients_of_the_chain(T, d, F):
    gh.lib()
    import block_training as ex
    master = ex.make(d, F, seed=3)
    master["norm"] = master["norm"] + 0.1 * torch.randn(d, device="cuda",
                                                        generator=torch.Generator("cuda").manual_seed(9))
    weights = {k: master[k].to(torch.bfloat16) for k in ex.NAMES}
    grads = {k: torch.zeros_like(v) for k, v in master.items()}
    block = capi.GatedFFN(d, F, max_tokens=T, training=True)
    batches = [ex.batch(T, d, i) for i in range(2)]
    loss, dxs = 0.0, []
    for b in batches:
        part, dx = ex.micro_batch(block, weights, master["norm"], *b, grads, 0.5)
        loss += 0.5 * float(part)
        dxs.append(dx)
    assert block.status() == 0
    want_loss, want, want_dx = exact(weights, master["norm"], batches)
    assert abs(loss - want_loss) <= TOL * want_loss
    for k in grads:
        assert float((grads[k].double() - want[k]).norm()) <= TOL * float(want[k].norm()), k
    for a, b in zip(dxs, want_dx):
        assert float((a.double() - b).norm()) <= TOL * float(b.norm())
    # clipped to half the norm
    total = sum(float(g.double().square().sum()) for g in grads.values()) ** 0.5
    before = {k: g.clone() for k, g in grads.items()}
    n = capi.clip_gradients(list(grads.values()), 0.5 * total)
    assert abs(float(n) - total) <= 1e-5 * total
    for k in grads:
        assert torch.allclose(grads[k], before[k] * (0.5 * total / (total + 1e-6)), rtol=1e-5, atol=0)


def test_example_runs():
    gh.lib()
    import block_training as ex
    history = ex.train(steps=4, verbose=False)
    assert len(history) == 4 and all(torch.isfinite(torch.tensor(h)).all() for h in history)
    # the same steps again give the same numbers, bit for bit
    assert ex.train(steps=3, verbose=False) == history[:3]


def test_micro_batch_in_a_graph():
    """The whole chain captured and replayed with new inputs."""
    gh.lib()
    import block_training as ex
    T, d, F = 64, 128, 256
    master = ex.make(d, F)
    weights = {k: master[k].to(torch.bfloat16) for k in ex.NAMES}
    block = capi.GatedFFN(d, F, max_tokens=T, training=True)
    x, stream, target = ex.batch(T, d, 0)

    def run(grads):
        for g in grads.values():
            g.zero_()
        loss, dx = ex.micro_batch(block, weights, master["norm"], x, stream, target, grads, 1.0)
        n = capi.clip_gradients(list(grads.values()), 0.1)
        return loss, dx, n

    held, now = ({k: torch.zeros_like(v) for k, v in master.items()} for _ in range(2))
    run(now)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(held)
    for seed in (4, 5):
        for t, v in zip((x, stream, target), ex.batch(T, d, seed)):
            t.copy_(v)
        g.replay()
        got = [t.clone() for t in out]
        want = run(now)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(held[k], now[k]) for k in held)
    assert block.status() == 0
