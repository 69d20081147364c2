"""The decoding example: its logits against the whole model in 64 bits, through forks, frees and compactions."""
import importlib.util
import os

import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tests.helpers import requires_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    requires_gpu()
    spec = importlib.util.spec_from_file_location("decode", os.path.join(ROOT, "examples", "decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(model, tokens):
    """Logits of the last of one sequence's tokens: every position at once, masked, no cache."""
    n, H, K, E = len(tokens), model.heads, model.kv_heads, model.head
    norm = lambda v, w: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w.double()  # noqa: E731
    w = torch.arange(n, device="cuda").double()[:, None, None] * model.freqs

    def turn(v):
        a, b = v[..., :E // 2], v[..., E // 2:]
        return model.rope_scale * torch.cat([a * w.cos() - b * w.sin(), b * w.cos() + a * w.sin()], -1)

    x = model.embed[tokens].double()
    later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
    for p in model.layers:
        qkv = (norm(x, p["norm1"]) @ p["qkv"].double().t()).view(n, H + 2 * K, E)
        q, k = turn(qkv[:, :H]), turn(qkv[:, H:H + K]).repeat_interleave(H // K, 1)
        v = qkv[:, H + K:].repeat_interleave(H // K, 1)
        s = torch.einsum("ihe,jhe->hij", q, k) * E ** -0.5
        a = torch.einsum("hij,jhe->ihe", torch.softmax(s.masked_fill(later, -torch.inf), -1), v).reshape(n, H * E)
        r = x + a @ p["out"].double().t()
        x = r + torch.nn.functional.silu(norm(r, p["norm2"]) @ p["up"].double().t()) @ p["down"].double().t()
    return norm(x, model.final)[-1] @ model.logits.double().t()


@pytest.mark.parametrize("page", [4, 16, 7])
def test_decoding_matches_the_whole_model(page):
    """Some eight tensors along a logit's way are rounded to bf16 (2^-9 each, relative): a relative distance of
    8 * 2^-9 = 1.6 % bounds their sum, and with what each step's rounding adds to the next layer's, 3 %."""
    m = example()
    g = torch.Generator(device="cuda").manual_seed(page)
    model = m.Model(seed=3)
    S = 10
    cache = m.Cache(model, 64, page, S, -(-60 // page))
    ints = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    past = {0: [], 3: [], 7: []}

    def run(steps):
        for _ in range(steps):
            tokens = torch.randint(0, len(model.embed), (S,), generator=g, device="cuda")
            logits = m.step(model, cache, tokens, ints(sorted(past)))
            for s in past:
                past[s].append(int(tokens[s]))
        assert cache.lens.tolist() == [len(past.get(s, [])) for s in range(S)]
        for s in past:
            want = reference(model, torch.tensor(past[s], device="cuda"))
            assert float((logits[s].double() - want).norm() / want.norm()) < 0.03, s

    run(11)
    past[5] = []  # a sequence that joins later
    run(9)
    cache.fork(ints([3, 3, 0]), ints([1, 2, 9]))
    past.update({1: list(past[3]), 2: list(past[3]), 9: list(past[0])})
    run(6)
    cache.free(ints([3, 0]))
    del past[3], past[0]
    before = [int((cache.refs > 0).sum()), int(cache.refs.sum())]
    cache.compact()
    assert before == [int((cache.refs > 0).sum()), int(cache.refs.sum())]
    assert int(cache.used) == before[0] and bool((cache.refs[:before[0]] > 0).all())
    run(5)
    past[0] = []  # an ended sequence's place is used again
    run(3)
    tgc.tgc_async_status()


def test_attention_does_not_depend_on_where_the_pages_lie():
    """The same bits before and after a compaction, and for a fork of the same tokens."""
    m = example()
    model = m.Model(seed=5)
    cache = m.Cache(model, 40, 8, 6, 6)
    ints = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    for t in range(21):
        m.step(model, cache, torch.full((6,), 3 * t, device="cuda"), ints([0, 2, 4]))
    cache.fork(ints([4]), ints([5]))
    q = torch.randn(6, model.heads, model.head, device="cuda").to(m.BF)
    q[5] = q[4]
    a, b = torch.empty_like(q), torch.empty_like(q)
    tgc.tgc_paged_attention(q, a, cache.pools[0], cache.pools[1], cache.table, cache.lens)
    assert torch.equal(a[4], a[5])
    cache.free(ints([0]))
    cache.compact()
    tgc.tgc_paged_attention(q, b, cache.pools[0], cache.pools[1], cache.table, cache.lens)
    assert torch.equal(a[1:], b[1:]) and not bool(b[0].any())


def test_a_captured_step():
    """Reserve, append and attention in one graph: every replay is the next token."""
    m = example()
    model = m.Model(layers=1, seed=6)
    K, E, H, S = model.kv_heads, model.head, model.heads, 3
    eager, graphed = m.Cache(model, 30, 4, S, 9), m.Cache(model, 30, 4, S, 9)
    live, one, ok = (torch.tensor(v, device="cuda", dtype=torch.int32) for v in ([0, 2], [1, 1], [0, 0]))
    qkv, out = torch.zeros(S, H + 2 * K, E, device="cuda", dtype=m.BF), torch.zeros(S, H, E, device="cuda", dtype=m.BF)
    q, pos = torch.zeros_like(out), torch.zeros(S, device="cuda", dtype=torch.int32)
    ws = torch.empty(tgc.tgc_kv_reserve_workspace_bytes(graphed.refs, graphed.table, graphed.lens, live, one, 4), device="cuda", dtype=torch.uint8)

    def token(c):
        tgc.tgc_kv_reserve(c.refs, c.table, c.lens, live, one, 4, ok=ok, workspace=ws)
        torch.sub(c.lens, 1, out=pos)
        tgc.tgc_kv_append(qkv[:, H:H + K], qkv[:, H + K:], c.pools[0], c.pools[1], c.table, pos, q=qkv[:, :H], q_out=q, freqs=model.freqs)
        tgc.tgc_paged_attention(q, out, c.pools[0], c.pools[1], c.table, c.lens)

    g = torch.Generator(device="cuda").manual_seed(0)
    inputs = torch.randn(20, S, H + 2 * K, E, generator=g, device="cuda").to(m.BF)
    want = []
    for x in inputs:
        qkv.copy_(x)
        token(eager)
        want.append(out.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token(graphed)
    for x, w in zip(inputs, want):
        qkv.copy_(x)
        graph.replay()
        assert torch.equal(out, w)
    assert torch.equal(graphed.table, eager.table) and torch.equal(graphed.lens, eager.lens)


def test_the_example_runs():
    texts = example().main(["--steps", "6", "--prompts", "2", "--branches", "2"])
    assert texts.shape == (6, 6) and bool((texts >= 0).all()) and bool((texts < 256).all())
