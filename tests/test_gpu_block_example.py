"""The transformer-block example: its gradients against autograd in 64 bits, and its training loop."""
import importlib.util
import os

import pytest
import torch

from tests.helpers import requires_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    requires_gpu()
    spec = importlib.util.spec_from_file_location("transformer_block", os.path.join(ROOT, "examples", "transformer_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(p, shards, routing):
    order, offsets, weight = routing
    off = offsets.tolist()
    norm = lambda v, w: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * w  # noqa: E731
    x = torch.cat(shards).double()
    a = torch.nn.functional.gelu(norm(x, p["norm_w"]) @ p["w1"].t() + p["b1"])
    y = a @ p["w2"].t() + p["b2"]
    gates = p["gate"].shape[0]
    r = x + p["gate"].repeat_interleave(len(x) // gates, 0) * norm(y, p["post_w"])
    he = norm(r, p["pre_w"])[order]
    parts = [torch.nn.functional.silu(he[i:j] @ p["e1"][e].t()) @ p["e2"][e].t()
             for e, (i, j) in enumerate(zip(off, off[1:]))]
    back = torch.empty_like(order)
    back[order] = torch.arange(len(order), device=order.device)
    return r + torch.cat(parts)[back] * weight.double()


def test_block_gradients_match_autograd():
    """Every tensor between the operators is rounded to bf16 (2^-9 each, relative), some ten of them
    along a gradient's longest way: 2^-9 * 10 = 2 % of a gradient's norm bounds their sum."""
    m = example()
    D, hidden, E, ranks = 128, 256, 5, 4
    g = torch.Generator(device="cuda").manual_seed(0)
    shards = [torch.randn(62, D, generator=g, device="cuda").to(m.BF) for _ in range(ranks)]
    p = m.make_params(D, hidden, E, 2, "cuda")
    routing = m.route(62 * ranks, E, "cuda")
    out, kept = m.forward(p, shards, routing)
    dout = torch.randn(62 * ranks, D, generator=g, device="cuda").to(m.BF)
    grads = m.backward(p, kept, routing, dout)
    leaf = {k: v.double().requires_grad_() for k, v in p.items()}
    ref = reference(leaf, shards, routing)
    assert float((out.double() - ref.detach()).norm() / ref.detach().norm()) < 0.02
    for k, want in zip(leaf, torch.autograd.grad(ref, list(leaf.values()), dout.double())):
        assert float((grads[k].double() - want).norm() / want.norm()) < 0.02, k


def test_training_loss_falls():
    losses = example().main(["--steps", "6", "--tokens", "264", "--width", "64", "--experts", "3"])
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
