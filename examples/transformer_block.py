"""A transformer block's dense MLP and expert MLP, forward, backward and an SGD step, on the library's
operators alone (torch holds the memory and sorts the rows by expert):

  shards --tgather--> x --norm--> h --linear + gelu--> a --linear--> y
  r, h2 = block_norm(y, residual x, gate)      the norms around the block boundary in one pass
  h2 --sort by expert--> linear + silu --> linear --unsort, weigh--> y2;  out = r + y2

    python examples/transformer_block.py [--steps 20] [--tokens 1000] [--width 512]

trains the block to map its input to a fixed random target and prints the loss of each step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tile_gather_comm_gb300 as tgc  # noqa: E402

BF = torch.bfloat16


def make_params(D, hidden, experts, gates, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)

    def n(*shape, sigma):
        return (torch.randn(*shape, generator=g, device=device) * sigma).to(BF)

    return {"norm_w": torch.ones(D, device=device, dtype=BF),
            "w1": n(hidden, D, sigma=D ** -0.5), "b1": torch.zeros(hidden, device=device, dtype=BF),
            "w2": n(D, hidden, sigma=hidden ** -0.5), "b2": torch.zeros(D, device=device, dtype=BF),
            "gate": n(gates, D, sigma=0.1) + 1, "post_w": torch.ones(D, device=device, dtype=BF),
            "pre_w": torch.ones(D, device=device, dtype=BF),
            "e1": n(experts, hidden, D, sigma=D ** -0.5), "e2": n(experts, D, hidden, sigma=hidden ** -0.5)}


def route(tokens, experts, device, seed=1):
    """A fixed routing: each token's expert and weight, the sorted order and the experts' offsets."""
    g = torch.Generator(device=device).manual_seed(seed)
    expert = torch.randint(0, experts, (tokens,), generator=g, device=device)
    weight = (torch.rand(tokens, 1, generator=g, device=device) * 0.5 + 0.5).to(BF)
    order = torch.argsort(expert, stable=True)
    offsets = torch.zeros(experts + 1, device=device, dtype=torch.int32)
    offsets[1:] = torch.cumsum(torch.bincount(expert, minlength=experts), 0)
    return order, offsets, weight


def forward(p, shards, routing):
    """The block's output and what its backward pass needs."""
    order, offsets, weight = routing
    D, M = shards[0].shape[1], sum(s.shape[0] for s in shards)
    new = lambda cols: torch.empty(M, cols, device=weight.device, dtype=BF)  # noqa: E731
    k = {}
    k["x"] = new(D)
    tgc.tgc_tgather(k["x"].view(1, 1, 1, M, D), [s.view(1, 1, 1, *s.shape) for s in shards])
    hidden = p["w1"].shape[0]
    k["h"], k["z1"], k["a1"], k["y"], k["r"], k["h2"] = new(D), new(hidden), new(hidden), new(D), new(D), new(D)
    tgc.tgc_block_norm(k["x"], None, k["h"], pre="rms", pre_weight=p["norm_w"])
    tgc.tgc_linear(k["h"], p["w1"], k["a1"], bias=p["b1"], act="gelu", z=k["z1"])
    tgc.tgc_linear(k["a1"], p["w2"], k["y"], bias=p["b2"])
    tgc.tgc_block_norm(k["y"], k["r"], k["h2"], x=k["x"], gate=p["gate"], post="rms", post_weight=p["post_w"],
                       pre="rms", pre_weight=p["pre_w"])
    k["he"], k["ze"], k["ae"], k["ye"] = k["h2"][order], new(hidden), new(hidden), new(D)
    tgc.tgc_linear(k["he"], p["e1"], k["ae"], act="silu", z=k["ze"], offsets=offsets)
    tgc.tgc_linear(k["ae"], p["e2"], k["ye"], offsets=offsets)
    y2 = torch.empty_like(k["ye"])
    y2[order] = k["ye"] * weight[order]
    out = new(D)
    tgc.tgc_block_norm(y2, out, x=k["r"], pre="none")
    return out, k


def backward(p, k, routing, dout):
    """The parameters' gradients from the output's."""
    order, offsets, weight = routing
    g = {name: torch.empty_like(v) for name, v in p.items()}
    like = torch.empty_like
    dye = dout[order] * weight[order]
    dae, dhe, dh2 = like(k["ae"]), like(k["he"]), like(k["h2"])
    tgc.tgc_linear_bwd(dye, k["ae"], p["e2"], dx=dae, dw=g["e2"], offsets=offsets)
    tgc.tgc_linear_bwd(dae, k["he"], p["e1"], z=k["ze"], act="silu", dx=dhe, dw=g["e1"], offsets=offsets)
    dh2[order] = dhe
    dy, da1, dh = like(k["y"]), like(k["a1"]), like(k["h"])
    tgc.tgc_block_norm_bwd(k["y"], k["r"], dout, dh2, gate=p["gate"], post="rms", post_weight=p["post_w"], pre="rms",
                           pre_weight=p["pre_w"], dy=dy, dgate=g["gate"], dpost_weight=g["post_w"],
                           dpre_weight=g["pre_w"])
    tgc.tgc_linear_bwd(dy, k["a1"], p["w2"], dx=da1, dw=g["w2"], dbias=g["b2"])
    tgc.tgc_linear_bwd(da1, k["h"], p["w1"], z=k["z1"], act="gelu", dx=dh, dw=g["w1"], dbias=g["b1"])
    tgc.tgc_block_norm_bwd(None, k["x"], None, dh, pre="rms", pre_weight=p["norm_w"], dpre_weight=g["norm_w"])
    return g


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--experts", type=int, default=6)
    ap.add_argument("--lr", type=float, default=2.0)
    a = ap.parse_args(argv)
    dev = torch.device("cuda")
    ranks, gates = 4, 2
    M = a.tokens // (ranks * gates) * (ranks * gates)
    gen = torch.Generator(device=dev).manual_seed(7)
    shards = [torch.randn(M // ranks, a.width, generator=gen, device=dev).to(BF) for _ in range(ranks)]
    target = torch.randn(M, a.width, generator=gen, device=dev)
    p = make_params(a.width, 4 * a.width, a.experts, gates, dev)
    routing = route(M, a.experts, dev)
    losses = []
    for step in range(a.steps):
        out, kept = forward(p, shards, routing)
        diff = out.float() - target
        losses.append(float((diff * diff).mean()))
        grads = backward(p, kept, routing, (diff * (2.0 / M)).to(BF))
        for name, v in p.items():
            v.sub_((a.lr * 0.01 * grads[name].float()).to(BF))
        print(f"step {step:3d}  loss {losses[-1]:.4f}")
    tgc.tgc_async_status()
    return losses


if __name__ == "__main__":
    main()
