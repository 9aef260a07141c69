"""Training a pre-norm gated feed-forward block, the shared expert's, on 32-bit master
weights: two micro-batches a step, gradients added up in fp32.

A micro-batch goes through
  rms_norm           s = x + stream in fp32, y = norm(s) in bf16
  GatedFFN.forward   out = block(y); gate and up are kept
and back through
  GatedFFN.backward  the weights' gradients (added to those of the micro-batches before)
                     and that of y
  rms_norm_backward  the gradient of s, and that of the norm's weight
and a step ends with
  clip_gradients     all gradients to one global norm
  Muon.step          the three matrices (the norm's weight takes a plain step)
The loss is the mean squared distance of s + out from a target.

    python examples/block_training.py [--steps 30]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from mixture_experts_layer_router_gb300 import capi  # noqa: E402

NAMES = ("w_g", "w_u", "w_d")


def make(d: int, F: int, seed: int = 0):
    """Master weights of the block and its norm, fp32."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(rows, cols, fan_in):
        return torch.randn((rows, cols), generator=gen, device="cuda") / fan_in ** 0.5

    return {"w_g": rand(F, d, d), "w_u": rand(F, d, d), "w_d": rand(d, F, F),
            "norm": torch.ones(d, device="cuda")}


def batch(T: int, d: int, seed: int):
    """x (bf16), the residual stream and the target (fp32), [T, d] each."""
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    x, stream, target = (torch.randn((T, d), generator=gen, device="cuda") for _ in range(3))
    return x.to(torch.bfloat16), stream, target


def micro_batch(block, weights, norm, x, stream, target, grads, scale: float):
    """Adds the gradients of scale * loss to grads; returns (loss, gradient of x)."""
    n = capi.rms_norm(x, norm, residual=stream)
    s, y = n["sum"], n["y"]
    out, gate, up = block.forward(y, **weights, save=True)
    off = s + out.float() - target
    d_out = (2.0 * scale / off.numel()) * off
    g = block.backward(d_out.to(torch.bfloat16), y, gate, up, **weights, accumulate=True,
                       out={"d" + k: grads[k] for k in NAMES})
    b = capi.rms_norm_backward(g["dx"], s, norm, n["rstd"], d_sum=d_out)
    grads["norm"] += b["dw"]
    return off.square().mean(), b["dx"]


def train(steps: int = 30, T: int = 96, d: int = 256, F: int = 512, micro: int = 2,
          lr: float = 0.01, max_norm: float = 0.5, seed: int = 0, verbose: bool = True):
    """Runs the steps and returns each step's (loss, norm of the gradients)."""
    master = make(d, F, seed)
    momentum = {k: torch.zeros_like(master[k]) for k in NAMES}
    muon = {k: capi.Muon(*master[k].shape) for k in NAMES}
    grads = {k: torch.zeros_like(v) for k, v in master.items()}
    block = capi.GatedFFN(d, F, max_tokens=T, training=True)
    history = []
    for step in range(steps):
        for g in grads.values():
            g.zero_()
        weights = {k: master[k].to(torch.bfloat16) for k in NAMES}
        loss = 0.0
        for i in range(micro):
            x, stream, target = batch(T, d, i)
            part, _ = micro_batch(block, weights, master["norm"], x, stream, target, grads,
                                  1.0 / micro)
            loss = loss + part / micro
        norm = capi.clip_gradients(list(grads.values()), max_norm)
        for k in NAMES:
            muon[k].step(master[k], grads[k], momentum[k], lr=lr, weight_decay=0.01)
        master["norm"] -= lr * grads["norm"]
        history.append((float(loss), float(norm)))
        if verbose and (step % 5 == 0 or step + 1 == steps):
            print(f"step {step:3d}  loss {history[-1][0]:.4f}  gradient norm {history[-1][1]:.4f}")
    for h in (block, *muon.values()):
        if h.status() != 0:
            raise RuntimeError("device status %d" % h.status())
    return history


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=30)
    train(p.parse_args().steps)
