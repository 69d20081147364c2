"""The attention and cache operators, and the example that decodes with them, at the edges of what they accept."""
import ctypes
import importlib.util
import math
import os
from fractions import Fraction

import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tile_gather_comm_gb300 import _lib
from tests import test_gpu_paged_attention as attention
from tests.helpers import requires_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    requires_gpu()


def ints(v):
    return torch.tensor(v, device="cuda", dtype=torch.int32)


# ---------------------------------------------------------------- the decoding example


def example():
    spec = importlib.util.spec_from_file_location("decode", os.path.join(ROOT, "examples", "decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def tokens_of(cache, s, n):
    """The first n tokens' bytes of sequence s, in every pool."""
    j = torch.arange(n, device="cuda")
    at = cache.table[s, j // cache.page].long()
    return [p[at, j % cache.page].view(torch.int16) for p in cache.pools]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_sequence_left_out_of_a_step_keeps_its_tokens():
    """Six tokens of three sequences, then steps without the second: its length, its bytes, and, when it goes on, the
    same logits as a cache in which nobody paused."""
    m = example()
    model = m.Model(seed=3)
    paused, straight = (m.Cache(model, 16, 4, 4, 5) for _ in range(2))
    for t in range(6):
        for c in (paused, straight):
            m.step(model, c, torch.full((4,), 3 * t + 1, device="cuda"), ints([0, 1, 2]))
    before = tokens_of(paused, 1, 6)
    for t in range(3):
        m.step(model, paused, torch.full((4,), 99 + t, device="cuda"), ints([2, 0]))
        assert paused.lens.tolist() == [7 + t, 6, 7 + t, 0]
        assert same(tokens_of(paused, 1, 6), before)
    got = m.step(model, paused, torch.full((4,), 42, device="cuda"), ints([1]))
    want = m.step(model, straight, torch.full((4,), 42, device="cuda"), ints([1]))
    assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("held", [8, 7])
def test_a_step_that_finds_no_room_keeps_every_token(held):
    """Two branches whose pages are full (shared, or one shared and one of each) and one free page: the first
    branch has it, the second is told so, and nobody's old tokens change."""
    m = example()
    model = m.Model(seed=3)
    cache = m.Cache(model, 3 if held == 8 else 4, 4, 2, 5)
    for t in range(held):
        m.step(model, cache, torch.full((2,), 3 * t + 1, device="cuda"), ints([0]))
    cache.fork(ints([0]), ints([1]))
    if held == 7:
        m.step(model, cache, torch.tensor([50, 60], device="cuda"), ints([0, 1]))
    before = [tokens_of(cache, s, 8) for s in range(2)]
    ok = ints([-1, -1])
    m.step(model, cache, torch.tensor([5, 77], device="cuda"), ints([0, 1]), ok)
    assert ok.tolist() == [1, 0] and cache.lens.tolist() == [9, 8]
    for s in range(2):
        assert same(tokens_of(cache, s, 8), before[s])


def test_a_step_that_names_sequences_twice_and_none():
    """The same as one that names each sequence once."""
    m = example()
    model = m.Model(seed=3)
    caches = [m.Cache(model, 16, 4, 4, 5) for _ in range(2)]
    for t in range(6):
        tokens = torch.full((4,), 3 * t + 1, device="cuda")
        want = m.step(model, caches[0], tokens, ints([0, 2, 3]))
        ok = ints([9] * 7)
        got = m.step(model, caches[1], tokens, ints([0, 3, 2, 0, -1, 4, 2]), ok)
        assert ok.tolist() == [1, 1, 1, 0, 0, 0, 0] and caches[1].lens.tolist() == [t + 1, 0, t + 1, t + 1]
        assert torch.equal(got[[0, 2, 3]], want[[0, 2, 3]])


def test_the_example_says_when_its_cache_is_too_small():
    """Pages for the prompts and no branch's copy of a part-filled one: the run ends with an error, not with tokens of
    sequences that were never made."""
    m = example()

    class Small(m.Cache):
        def __init__(self, model, pages, page, seqs, max_pages):
            super().__init__(model, 2 * -(-40 // page), page, seqs, max_pages)

    m.Cache = Small
    with pytest.raises(RuntimeError, match="no room"):
        m.main(["--steps", "2", "--prompts", "2", "--branches", "1"])


# ---------------------------------------------------------------- attention


@pytest.mark.parametrize("scale,cap", [(8.0, 2.3e38), (0.125, 1e37), (1.0, 1e-30), (0.125, 1e-38), (-0.5, 40.0)])
@pytest.mark.parametrize("S", [1, 300])
def test_the_largest_and_smallest_caps(scale, cap, S):
    """A cap that no score comes near changes nothing; one that all pass by far leaves +-cap, 0 for softmax.  Products
    of -1, 0 and 1: scores are exact before they are scaled, 2^9.6 in powers of two at most.  Quotient, product and the
    cap's factor round by 2^-24 each and tanh by 2^-22: 2^-11.6 of a score and as much of the reference, times ln 2 2^-11.1
    of a probability, twice (product and sum) 2^-10.1; what is left to 2^-9 is for the sums and parts."""
    g = torch.Generator(device="cuda").manual_seed(S)
    n, D, page = 70, 64, 16
    kp = torch.randint(-1, 2, (S * 5, page, 1, D), generator=g, device="cuda").to(BF)
    vp = torch.randn(S * 5, page, 1, D, generator=g, device="cuda").to(BF)
    table = torch.arange(S * 5, device="cuda", dtype=torch.int32).view(S, 5)
    q = torch.randint(-1, 2, (S, 2, D), generator=g, device="cuda").to(BF)
    out = torch.empty_like(q)
    tgc.tgc_paged_attention(q, out, kp, vp, table, ints([n] * S), scale=scale, softcap=cap)
    k, v = (p[table.long()].reshape(S, 80, D)[:, :n].double() for p in (kp, vp))
    x = q.double() @ k.transpose(1, 2) * scale
    p = torch.softmax(cap * torch.tanh(x / cap), -1)
    want, size = p @ v, p @ v.abs()
    assert bool(((out.double() - want).abs() <= 2 ** -9 * size + 2 ** -8 * want.abs()).all())


@pytest.mark.parametrize("late", [0, 500, 900, 999])
@pytest.mark.parametrize("S,Hk", [(400, 1), (40, 4), (1, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_near_the_end_of_fp32(late, S, Hk, D):
    """A key of e^5.25 times the others' weight (2^7.6: under any step of the reference) with values of 2^122 among zeros:
    what comes out is finite, and so has to be the way there.  Scores are 0 and 5.25: off by 2^-22 in powers of two; the
    parts of a probability by 2^-17, sums of 1000 by 2^-14, one rounding."""
    n, page, wide = 1000, 16, 63
    kp = torch.zeros(S * wide, page, Hk, D, device="cuda", dtype=BF)
    vp = torch.zeros_like(kp)
    table = torch.arange(S * wide, device="cuda", dtype=torch.int32).view(S, wide)
    at = table[:, late // page].long()
    kp[at, late % page, :, 0] = 5.25
    vp[at, late % page] = 2.0 ** 122
    q = torch.zeros(S, 2 * Hk, D, device="cuda", dtype=BF)
    q[..., 0] = 1
    out = torch.empty_like(q)
    tgc.tgc_paged_attention(q, out, kp, vp, table, ints([n] * S), scale=1.0)
    want = 2.0 ** 122 * math.exp(5.25) / (math.exp(5.25) + n - 1)
    assert bool(((out.double() - want).abs() <= want * (2 ** -8 + 2 ** -13)).all())


@pytest.mark.parametrize("shape", [(6, 8, 1, 64), (1, 8, 2, 64), (6, 1, 2, 64)])
def test_strides_of_one_entry_mean_nothing(shape):
    """Keys and values whose strides differ only where a dimension has one entry."""
    g = torch.Generator(device="cuda").manual_seed(4)
    kp, vp = (torch.randn(shape, generator=g, device="cuda").to(BF) for _ in range(2))
    strides = [s if n > 1 else 40 for n, s in zip(shape, vp.stride())]
    odd = vp.as_strided(shape, strides)
    table = ints([[0, min(3, shape[0] - 1), -1]])
    n = ints([2 * shape[1]])
    q = torch.randn(1, 2 * shape[2], 64, generator=g, device="cuda").to(BF)
    want, out = torch.empty_like(q), torch.empty_like(q)
    tgc.tgc_paged_attention(q, want, kp, vp, table, n)
    tgc.tgc_paged_attention(q, out, kp, odd, table, n)
    assert torch.equal(out, want)
    x = torch.randn(1, shape[2], 64, generator=g, device="cuda").to(BF)
    tgc.tgc_kv_append(x, x, kp, odd, table, ints([0]))
    assert torch.equal(vp[0, 0], x[0]) and torch.equal(kp[0, 0], x[0])
    with pytest.raises(ValueError):  # and where they mean something they have to be the same
        tgc.tgc_paged_attention(q, out, kp, vp.transpose(1, 2).contiguous().transpose(1, 2) if shape[1] > 1 and shape[2] > 1 else vp[..., :32], table, n)


@pytest.mark.parametrize("lens,Hk,group,D,page", attention.FOURS + [([200, 0, 7, 33] * 6, 8, 8, 64, 8), ([300, 1] * 20, 4, 7, 104, 16)])
@pytest.mark.parametrize("dtype", list(attention.DT))
def test_key_heads_by_fours_under_wide_tables(lens, Hk, group, D, page, dtype):
    """Tables wide enough that every warp takes a key head of its own, whatever the lengths are."""
    g = attention.gen(sum(lens) + D)
    items = len(lens) * Hk
    wide = 2 * 304 * 900 * group // items // page + 1
    kp, vp, table, n, keys = attention.cache(lens, page, Hk, D, attention.DT[dtype], g, wide=wide)
    q = torch.randn(len(lens), Hk * group, D, generator=g, device="cuda").to(attention.DT[dtype])
    for window, cap in ((0, 0.0), (37, 5.0)):
        out, lse = torch.full_like(q, 7.0), torch.full((len(lens), Hk * group), 7.0, device="cuda")
        tgc.tgc_paged_attention(q, out, kp, vp, table, n, lse=lse, window=window, softcap=cap)
        attention.check(out, lse, q, keys, D ** -0.5, window, cap)


@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_two_parts_of_a_probability(dtype):
    """Hundreds of keys of one weight against 16 of another (one of every 32, so that every warp's reference comes of
    them), whose values nearly cancel: what is left shows what the two 16-bit parts of a probability lose, 2^-17 of it in bf16 (8 bits, then 8 bits of a rest below 2^-8) and 2^-23 in fp16.
    Beside that: scores are exact, times log2(e) off by 2^-24 of 2^3, the exponential by 2^-22, 25 sums of a lane and
    of the lanes by 2^-24 each, 16 products of 16 keys by 2^-22 each: 2^-17 in all, and one rounding of the result."""
    n, D, page, wide = 512, 64, 16, 32
    scores = [float(torch.tensor(-k / 64).to(dtype)) for k in range(3, 250, 5)]
    S = len(scores)
    keys, values = torch.full((S, n), -64.0, dtype=torch.float64), torch.zeros(S, n, dtype=torch.float64)
    for s, x in enumerate(scores):
        _, m, c = min((abs(m * math.exp(x) - c), m, c) for m in range(200, 496)
                      for c in [float(torch.tensor(m * math.exp(x)).to(dtype))])
        light = torch.arange(n)[torch.arange(n) % 32 != 0][:m]
        keys[s, ::32], values[s, ::32] = 0.0, -c / 16
        keys[s, light], values[s, light] = x, 1.0
    p = torch.softmax(keys, 1)
    want, size = (p * values).sum(1), (p * values.abs()).sum(1)
    assert float((want.abs() / size).max()) < 2 ** -10  # the result's own rounding: 2^-18 of size
    kp = torch.zeros(S * wide, page, 1, D, device="cuda", dtype=dtype)
    kp[..., 0] = keys.view(S * wide, page, 1).cuda().to(dtype)
    vp = values.view(S * wide, page, 1, 1).cuda().to(dtype).expand(-1, -1, -1, D).contiguous()
    q = torch.zeros(S, 1, D, device="cuda", dtype=dtype)
    q[..., 0] = 1
    out = torch.empty_like(q)
    tgc.tgc_paged_attention(q, out, kp, vp, torch.arange(S * wide, device="cuda", dtype=torch.int32).view(S, wide), ints([n] * S), scale=1.0)
    err = (out[:, 0].double() - want.cuda()[:, None]).abs().amax(1).cpu()
    lost = {BF: 2 ** -17, torch.float16: 2 ** -23}[dtype]
    assert dtype != BF or float((err / size).max()) > 2 ** -20  # what the parts lose is seen here
    assert bool((err <= (lost + 2 ** -17) * size + torch.finfo(dtype).eps / 2 * want.abs() + 2 ** -25).all())


# ---------------------------------------------------------------- the cache's upkeep


def test_upkeep_without_pools():
    """npools = 0: the same bookkeeping as with pools, and no bytes."""
    tables = []
    for pools in (True, False):
        refs, lens = torch.zeros(40, device="cuda", dtype=torch.int32), ints([0] * 6)
        table, ws = torch.full((6, 8), -1, device="cuda", dtype=torch.int32), torch.empty(1 << 16, device="cuda", dtype=torch.uint8)
        src, dst, used = ints([0, 1, 1]), ints([4, 5, 3]), ints([-1])
        tgc.tgc_kv_reserve(refs, table, lens, ints([0, 1, 2]), ints([13, 16, 30]), 4)
        if pools:
            pool = [torch.zeros(40, 4, 8, device="cuda", dtype=BF)]
            tgc.tgc_kv_fork(pool, refs, table, lens, src, dst, 4)
            tgc.tgc_kv_free(refs, table, lens, ints([0, 1]))
            tgc.tgc_kv_compact(pool, refs, table, used)
        else:
            a = _lib.KvArgs(refs=refs.data_ptr(), table=table.data_ptr(), lens=lens.data_ptr(), num_pages=40, page_size=4,
                            num_seqs=6, max_pages=8, src=src.data_ptr(), dst=dst.data_ptr(), n=3, workspace=ws.data_ptr(),
                            workspace_bytes=ws.numel(), used=used.data_ptr(), stream=torch.cuda.current_stream().cuda_stream)
            assert _lib.lib().tgc_kv_fork(ctypes.byref(a)) == _lib.TGC_OK
            tgc.tgc_kv_free(refs, table, lens, ints([0, 1]))
            assert _lib.lib().tgc_kv_compact(ctypes.byref(a)) == _lib.TGC_OK
        tables.append([t.tolist() for t in (refs, table, lens, used)])
    assert tables[0] == tables[1] and tables[0][3] == [8 + 3 + 1 + 4]


# ---------------------------------------------------------------- positions


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("back", [False, True])
def test_angles_keep_their_bits(layout, back):
    """Fast and slow pairs at near and far positions against whole-number arithmetic.  The fraction of a turn is off by
    2^-64 a position (2^-61.3 radians, with its product's 2^-106); the angle is rounded to fp32 twice, 2^-23 of itself,
    sine and cosine by 2 units (2^-23 each): 2^-23 |w cos w| + 2^-22 |sin w|, below 2^-21 up to w = pi and below
    2^-21 w for a small one, and the same with sine and cosine the other way round."""
    freqs = [1.0, 0.7310585786300049, 0.11, 0.5, math.pi, 100.3, 12345.678, -0.9, 1e-3, 1e-7, 1e-9, 3e-12, -1e-10, 2.0 ** 40 + 0.5, 0.0]
    pos = [0, 1, 3, 4097, 999983, 16777217, 2 ** 31 - 1]
    R = 2 * len(freqs)
    q = torch.zeros(len(pos), 1, R, device="cuda")
    a, b = (q[..., :R // 2], q[..., R // 2:]) if layout == "half" else (q[..., 0::2], q[..., 1::2])
    a.fill_(1.0)  # (1, 0) turns into (cos, sin)
    (tgc.tgc_rope_bwd if back else tgc.tgc_rope)(q, q, ints(pos), torch.tensor(freqs, dtype=torch.float64, device="cuda"), layout=layout)
    turn = Fraction(2 * 31415926535897932384626433832795028841971693993751, 10 ** 49)
    for t, p in enumerate(pos):
        for i, f in enumerate(freqs):
            w = Fraction(f) * p * (-1 if back else 1)
            w = float(w - turn * round(w / turn))
            far = p * 2 ** -61
            assert abs(float(a[t, 0, i]) - math.cos(w)) <= 2 ** -21 + far, (p, f)
            assert abs(float(b[t, 0, i]) - math.sin(w)) <= 2 ** -21 * min(1.0, abs(w)) + far, (p, f)


def test_append_where_no_page_can_be():
    """An empty pool (its pointer is NULL), a table without pages, one without sequences: the queries are turned, and keys
    and values dropped."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(3, 2, 8, generator=g, device="cuda")
    freqs, _ = tgc.tgc_rope_freqs(8)
    pos, want, seqs = ints([1, 2, 3]), torch.empty_like(x), ints([0, 0, 0])
    tgc.tgc_rope(x, want, pos, freqs)
    for pages, seq_n, wide in ((0, 3, 2), (2, 3, 0), (2, 0, 2), (0, 0, 0)):
        pool = torch.zeros(pages, 4, 2, 8, device="cuda")
        out = torch.full_like(x, 7.0)
        tgc.tgc_kv_append(x, x, pool, pool, torch.zeros(seq_n, wide, device="cuda", dtype=torch.int32), pos, seqs=seqs, q=x,
                          q_out=out, freqs=freqs)
        assert torch.equal(out, want) and not bool(pool.any())


@pytest.mark.parametrize("seed", range(8))
def test_corrupt_bookkeeping_moves_bytes_of_the_pool_alone(seed):
    """Table entries, lengths and references that no history gives, and a pool between two pages that are not its own:
    those stay, and every 16 bytes of the pool are some page's of it (a page may be a source and a destination at once
    then, so not every page is one page's)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages, seqs, wide, page = 32, 6, 8, 4

    def mixed(n, low, high):
        v = torch.randint(low, high, (n,), generator=g, device="cuda", dtype=torch.int32)
        bad = torch.tensor([-1, -(2 ** 31), 2 ** 31 - 1, pages, pages + 1, -2], device="cuda", dtype=torch.int32)
        pick = torch.randint(0, 24, (n,), generator=g, device="cuda")
        return torch.where(pick < 6, bad[pick.clamp(max=5)], v)

    refs, table, lens = mixed(pages, -2, 3), mixed(seqs * wide, 0, pages).view(seqs, wide), mixed(seqs, 0, wide * page)
    lens[:2] = 0  # children that can be
    pools = [torch.empty(pages + 2, page, 8, device="cuda", dtype=BF) for _ in range(2)]
    for p in pools:
        p.copy_(torch.arange(pages + 2, device="cuda")[:, None, None].expand_as(p))
        p[0], p[-1] = -100, -200
    inner = [p[1:-1] for p in pools]
    tgc.tgc_kv_reserve(refs, table, lens, mixed(8, 2, seqs), mixed(8, 0, 9), page)
    tgc.tgc_kv_fork(inner, refs, table, lens, mixed(7, 2, seqs), mixed(7, 0, seqs), page)
    tgc.tgc_kv_compact(inner, refs, table)
    tgc.tgc_kv_copy(inner, inner, mixed(4, 0, pages // 2), pages - 1 - mixed(4, 0, pages // 2))
    tgc.tgc_kv_free(refs, table, lens, mixed(7, 0, seqs))
    torch.cuda.synchronize()
    for p, a in zip(pools, inner):
        assert bool((p[0] == -100).all()) and bool((p[-1] == -200).all())
        assert bool((a == a[..., :1]).all()) and bool((a >= 1).all()) and bool((a <= pages).all())
        assert bool((a[:, 0, 0] != torch.arange(1, pages + 1, device="cuda")).any())  # something was moved
