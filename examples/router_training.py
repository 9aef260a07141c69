"""Training a LatentMoE layer's router and expert matrices, one step after another.

A step runs the layer's forward, takes the routing it chose, and from there
  balance_loss      load-balancing loss and per-expert counts of the choices
  router_backward   its gradient, and that of the gates, with respect to the logits
  Muon.step         orthogonalised update of the router matrix, and of the
                    experts' gate matrices as one stack
on 32-bit master weights, which are loaded back into the layer as bf16. The
gradients that a training program gets from its own backward pass (of the gates,
and of the expert matrices) are stand-ins here: the program passes them as
tensors.

    python examples/router_training.py [--steps 30]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from mixture_experts_layer_router_gb300 import capi, synth  # noqa: E402


def train(steps: int = 30, lr: float = 0.02, balance_coef: float = 1.0, z_coef: float = 1e-3,
          seq_len: int = 32, seed: int = 0, verbose: bool = True):
    """Runs the steps on the tiny layer and returns each step's (balance, z,
    largest share of the slots that one expert got)."""
    cfg = synth.CONFIGS["tiny"]
    dev = "cuda"
    w = synth.make_weights(cfg, seed, dev)
    x = synth.make_x(cfg, seed, dev)
    # a router that starts out lopsided: a few rows point along the mean token
    x = (x.float() + 1.0).to(torch.bfloat16)
    w["w_r"][: cfg.E // 4] += (0.5 / cfg.d) * torch.ones_like(w["w_r"][: cfg.E // 4])
    layer = capi.LatentMoE(cfg.d, cfg.l, cfg.E, cfg.k, cfg.F, cfg.Fs, max_tokens=cfg.T, renorm=True)

    router = w["w_r"].float().contiguous()      # [E, d] master weights
    router_m = torch.zeros_like(router)
    gates_w = w["w_g"].float().contiguous()     # [E, F, l], one matrix an expert
    gates_m = torch.zeros_like(gates_w)
    muon_router = capi.Muon(cfg.E, cfg.d)
    muon_gates = capi.Muon(cfg.F, cfg.l, batch=cfg.E)
    gen = torch.Generator(device=dev).manual_seed(seed)
    d_gates = 1e-4 * torch.randn((cfg.T, cfg.k), generator=gen, device=dev) / cfg.T
    valid = torch.ones(cfg.T, dtype=torch.uint8, device=dev)
    valid.view(-1, seq_len)[:, -2:] = 0         # two tokens of padding a sequence

    history = []
    for step in range(steps):
        w["w_r"] = router.to(torch.bfloat16)
        w["w_g"] = gates_w.to(torch.bfloat16)
        layer.load_weights(w)
        layer.forward(x)
        r = layer.get_routing(cfg.T, dev)
        s = layer.balance_loss(r["logits"], r["idx"], valid=valid, seq_len=seq_len,
                               balance_coef=balance_coef, z_coef=z_coef)
        d_logits = layer.router_backward(r["logits"], r["idx"], s["counts"], s["tokens"],
                                         d_gates=d_gates, valid=valid, seq_len=seq_len,
                                         balance_coef=balance_coef, z_coef=z_coef)
        # the router is linear in x; its matrix's gradient is the program's own
        d_router = d_logits.t().matmul(x.float())
        muon_router.step(router, d_router, router_m, lr=lr, weight_decay=0.0)
        d_experts = 1e-3 * torch.randn(gates_w.shape, generator=gen, device=dev)
        muon_gates.step(gates_w, d_experts.to(torch.bfloat16), gates_m, lr=1e-4, weight_decay=0.1)

        counts = s["counts"].sum(0)
        _, balance, z = s["loss"].tolist()
        share = float(counts.max()) / float(counts.sum())
        history.append((balance, z, share))
        if verbose and (step % 5 == 0 or step + 1 == steps):
            print(f"step {step:3d}  balance {balance:.4f}  z {z:.3f}  largest share {share:.3f}")
    for h in (layer, muon_router, muon_gates):
        if h.status() != 0:
            raise RuntimeError("device status %d" % h.status())
    return history


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=30)
    train(p.parse_args().steps)
