"""A small transformer decoding with a paged key-value cache, on the library's operators alone (torch holds the
memory, embeds and picks tokens):

  x --norm--> h --linear--> q, k, v
  q, k turned by their positions; k, v into their pages                 (tgc_kv_append)
  attention of each sequence's new token over its pages                 (tgc_paged_attention)
  --linear, + x--> r --norm--> linear + silu --> linear, + r

    python examples/decode.py [--steps 24] [--branches 3]

feeds some prompts, forks each into branches that sample on their own, ends half of them, compacts the cache
and goes on.  The cache's bookkeeping stays on the device: a step never waits for it.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tile_gather_comm_gb300 as tgc  # noqa: E402

BF = torch.bfloat16


class Model:
    def __init__(self, layers=2, heads=8, kv_heads=2, head=64, vocab=256, hidden=512, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.head = heads, kv_heads, head
        self.width = D = heads * head

        def n(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(BF)

        self.embed = torch.randn(vocab, D, generator=g, device=device).to(BF)
        self.layers = [{"norm1": torch.ones(D, device=device, dtype=BF), "qkv": n((heads + 2 * kv_heads) * head, D),
                        "out": n(D, D), "norm2": torch.ones(D, device=device, dtype=BF), "up": n(hidden, D),
                        "down": n(D, hidden)} for _ in range(layers)]
        self.final = torch.ones(D, device=device, dtype=BF)
        self.logits = n(vocab, D)
        # a context four times longer than the 4096 tokens that the model would have been trained on
        self.freqs, self.rope_scale = tgc.tgc_rope_freqs(head, scaling="yarn", factor=4.0, trained=4096.0, device=device)


class Cache:
    """Pages of keys and values for every layer, and which sequence holds which."""

    def __init__(self, model, pages, page, seqs, max_pages, device="cuda"):
        self.page = page
        shape = (pages, page, model.kv_heads, model.head)
        self.pools = [torch.zeros(shape, device=device, dtype=BF) for _ in range(2 * len(model.layers))]
        ints = dict(device=device, dtype=torch.int32)
        self.refs, self.lens = torch.zeros(pages, **ints), torch.zeros(seqs, **ints)
        self.table = torch.full((seqs, max_pages), -1, **ints)
        self.used = torch.zeros(1, **ints)

    def reserve(self, seqs, ok):
        tgc.tgc_kv_reserve(self.refs, self.table, self.lens, seqs, torch.ones_like(seqs), self.page, ok=ok)

    def fork(self, src, dst, ok=None):
        tgc.tgc_kv_fork(self.pools, self.refs, self.table, self.lens, src, dst, self.page, ok=ok)

    def free(self, seqs):
        tgc.tgc_kv_free(self.refs, self.table, self.lens, seqs)

    def compact(self):
        tgc.tgc_kv_compact(self.pools, self.refs, self.table, self.used)


def step(model, cache, tokens, live, ok=None):
    """One token of every sequence in ``live`` (int32) through the model; tokens has one for every sequence of
    the cache.  Returns logits (sequences, vocabulary).  A sequence that is not in ``live``, or that the cache has
    no room for (``ok``, int32 beside ``live``, says which it had), keeps its tokens as they are; its row of the logits
    means nothing."""
    S, H, K, E, D = len(tokens), model.heads, model.kv_heads, model.head, model.width
    new = lambda *shape: torch.empty(*shape, device=tokens.device, dtype=BF)  # noqa: E731
    ok = torch.empty_like(live) if ok is None else ok
    cache.reserve(live, ok)
    # the new token's position where there is one, -1 elsewhere: nothing of those is appended
    at = live.long().clamp(0, S - 1)  # what is no sequence, or is named again, was refused
    pos = torch.full_like(cache.lens, -1)
    pos.scatter_reduce_(0, at, torch.where(ok > 0, cache.lens[at] - 1, -1), "amax")
    x = model.embed[tokens]
    for i, w in enumerate(model.layers):
        keys, values = cache.pools[2 * i:2 * i + 2]
        h, qkv, q, a, r, u = new(S, D), new(S, H + 2 * K, E), new(S, H, E), new(S, H, E), new(S, D), new(S, len(w["up"]))
        tgc.tgc_block_norm(x, None, h, pre="rms", pre_weight=w["norm1"])
        tgc.tgc_linear(h, w["qkv"], qkv.view(S, -1))
        q.zero_()  # rows without a new token are left as they are
        tgc.tgc_kv_append(qkv[:, H:H + K], qkv[:, H + K:], keys, values, cache.table, pos, q=qkv[:, :H], q_out=q,
                          freqs=model.freqs, scale=model.rope_scale)
        tgc.tgc_paged_attention(q, a, keys, values, cache.table, cache.lens)
        tgc.tgc_linear(a.view(S, D), w["out"], r, residual=x)
        tgc.tgc_block_norm(r, None, h, pre="rms", pre_weight=w["norm2"])
        tgc.tgc_linear(h, w["up"], u, act="silu")
        x = new(S, D)
        tgc.tgc_linear(u, w["down"], x, residual=r)
    h, logits = new(S, D), new(S, len(model.logits))
    tgc.tgc_block_norm(x, None, h, pre="rms", pre_weight=model.final)
    tgc.tgc_linear(h, model.logits, logits)
    return logits


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--prompts", type=int, default=4)
    ap.add_argument("--branches", type=int, default=3)
    ap.add_argument("--page", type=int, default=16)
    a = ap.parse_args(argv)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(1)
    model = Model()
    S = a.prompts * (1 + a.branches)
    most = 40 + a.steps
    cache = Cache(model, S * (-(-most // a.page)), a.page, S, -(-most // a.page))
    prompt = torch.randint(0, len(model.embed), (40, S), generator=g, device=dev)
    parents = torch.arange(a.prompts, device=dev, dtype=torch.int32)
    refused = torch.zeros((), device=dev, dtype=torch.int64)  # tokens and branches that found no room
    ok = torch.empty_like(parents)
    for t in range(40):
        logits = step(model, cache, prompt[t], parents, ok)
        refused += (ok == 0).sum()
    children = torch.arange(a.prompts, S, device=dev, dtype=torch.int32)
    ok = torch.empty_like(children)
    cache.fork(children % a.prompts, children, ok)
    refused += (ok == 0).sum()
    live = torch.arange(S, device=dev, dtype=torch.int32)
    logits = logits[live % a.prompts]
    ok = torch.empty_like(live)
    texts = []
    for t in range(a.steps):
        p = torch.softmax(logits.float(), -1)
        tokens = torch.multinomial(p, 1, generator=g).view(-1)
        texts.append(tokens)
        if t == a.steps // 2:  # every second sequence ends
            cache.free(live[1::2].contiguous())
            live = live[::2].contiguous()
            ok = torch.empty_like(live)
            cache.compact()
            print(f"{len(live)} sequences go on in {int(cache.used)} pages")
        logits = step(model, cache, tokens, live, ok)
        refused += (ok == 0).sum()
    if int(refused):
        raise RuntimeError(f"the cache had no room for {int(refused)} tokens or branches")
    texts = torch.stack(texts, 1)
    for s in live.tolist():
        print(f"sequence {s:2d} ({int(cache.lens[s])} tokens): {texts[s].tolist()}")
    tgc.tgc_async_status()
    return texts


if __name__ == "__main__":
    main()
