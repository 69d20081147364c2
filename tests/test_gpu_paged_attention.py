"""Attention of single tokens over a paged cache, against softmax in 64 bits.

Tolerance, worst case: a score is a sum of D products in fp32, off by at most (D + 4) 2^-23 sum |q k| scale = dx (the
capped one by no more: tanh's slope is at most 1, its own error 2^-22 of the cap).  A probability is then off by a factor
of 1 + 2 dx + 2^-20 (exponential, its argument's rounding below 2^6 in powers of two, two 16-bit parts); sums over n
keys add n 2^-24, so out is off by (2 dx + n 2^-23 + 2^-19) sum p |v|, and then rounded once."""
import math

import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tests.helpers import requires_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def _gpu():
    requires_gpu()


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def cache(lens, page, Hk, D, dt, g, spare=3, heads_first=False, wide=0):
    """Shuffled pages with garbage (NaN) behind each sequence's end and on pages that nobody has."""
    counts = [-(-n // page) for n in lens]
    n = sum(counts) + spare
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(counts), 1) + wide), -1, device="cuda", dtype=torch.int32)
    stores = [torch.full((n, Hk, page, D) if heads_first else (n, page, Hk, D), float("nan"), device="cuda", dtype=dt)
              for _ in range(2)]
    kp, vp = (s.transpose(1, 2) if heads_first else s for s in stores)
    keys, at = [], 0
    for s, (m, c) in enumerate(zip(lens, counts)):
        table[s, :c] = order[at:at + c]
        at += c
        kv = torch.randn(2, m, Hk, D, generator=g, device="cuda").to(dt)
        j = torch.arange(m, device="cuda")
        where = table[s, j // page].long()
        kp[where, j % page], vp[where, j % page] = kv[0], kv[1]
        keys.append(kv)
    return kp, vp, table, torch.tensor(lens, device="cuda", dtype=torch.int32), keys


def expect(q, kv, scale, window=0, cap=0.0, gone=None):
    """One sequence: out, lse, their tolerances before rounding.  gone: keys left out."""
    Hq, D = q.shape
    _, n, Hk, _ = kv.shape
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    if window:
        keep[:max(0, n - window)] = False
    if gone is not None:
        keep &= ~gone
    if not bool(keep.any()):
        z = torch.zeros(Hq, D, dtype=torch.float64, device="cuda")
        return z, torch.full((Hq,), -math.inf, dtype=torch.float64, device="cuda"), z, z[:, 0]
    k, v = kv[:, keep].double()
    k, v = (t.repeat_interleave(Hq // Hk, 1) for t in (k, v))
    x = torch.einsum("hd,jhd->hj", q.double(), k) * scale
    dx = float((torch.einsum("hd,jhd->hj", q.double().abs(), k.abs()) * abs(scale)).max()) * (D + 4) * 2 ** -23
    if cap:
        x = cap * torch.tanh(x / cap)
        dx += cap * 2 ** -22
    p = torch.softmax(x, 1)
    lse = torch.logsumexp(x, 1)
    rel = 2 * dx + int(keep.sum()) * 2 ** -23 + 2 ** -19
    return torch.einsum("hj,jhd->hd", p, v), lse, rel * torch.einsum("hj,jhd->hd", p, v.abs()), rel + lse.abs() * 2 ** -22


def check(out, lse, q, keys, scale, window=0, cap=0.0):
    half = torch.finfo(out.dtype).eps / 2
    for s, kv in enumerate(keys):
        want, want_lse, tol, tol_lse = expect(q[s], kv, scale, window, cap)
        err = (out[s].double() - want).abs()
        assert bool((err <= tol + half * (want.abs() + tol) + 2 ** -25).all()), (s, float((err - tol).max()))
        if lse is not None:
            inf = torch.isinf(want_lse)
            assert torch.equal(lse[s][inf].double(), want_lse[inf])
            assert bool(((lse[s].double() - want_lse).abs()[~inf] <= tol_lse[~inf]).all()), s


CASES = [  # lens, key heads, group, D, page
    ([1], 1, 1, 8, 1), ([5, 0, 17], 2, 1, 64, 16), ([900], 8, 4, 128, 16), ([64, 65, 63, 1, 0, 128], 2, 8, 128, 64),
    ([1000, 3, 257], 1, 16, 128, 7), ([4000, 20], 2, 5, 80, 24), ([2000], 1, 32, 128, 32), ([333, 1200], 1, 17, 64, 100),
    ([700, 41], 3, 8, 256, 16), ([1500], 1, 40, 256, 33), ([50] * 40, 2, 2, 96, 13), ([300, 0, 300], 2, 71, 16, 8),
    ([20000], 1, 4, 64, 16), ([9000, 1, 12000], 2, 8, 128, 128), ([511] * 9, 4, 3, 144, 3), ([1] * 300, 1, 1, 64, 4)]


# many items, or long ones, with more than 8 heads a key or more than 128 elements a head
WIDE = [([20000, 300], 1, 16, 128, 16), ([9000, 1, 8000], 2, 32, 96, 24), ([700, 5] * 85, 2, 12, 64, 16),
        ([500, 0, 1, 127, 128, 129] * 30, 2, 9, 72, 7), ([300] * 160, 1, 4, 256, 16), ([12000], 1, 16, 256, 33),
        ([130, 0, 257] * 60, 1, 40, 200, 5), ([25000], 1, 33, 128, 64), ([1, 2, 3] * 110, 1, 20, 8, 1)]


# many items of key heads by fours
FOURS = [([1] * 200, 4, 1, 64, 1), ([700, 5, 0, 33, 32, 31, 64] * 12, 4, 3, 40, 16), ([1, 2, 15, 16, 17] * 30, 8, 8, 128, 5),
         ([6000, 1, 9000, 16] * 4, 16, 1, 64, 24), ([0, 0, 3000] * 11, 4, 8, 120, 16), ([257, 0, 1000] * 6, 12, 5, 72, 7),
         ([50] * 170, 32, 1, 8, 64), ([20000, 3, 1200, 7] * 8, 4, 4, 128, 64), ([0] * 60 + [900] * 4 + [0] * 60, 8, 2, 96, 16)]


@pytest.mark.parametrize("lens,Hk,group,D,page", CASES + WIDE + FOURS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("window,cap", [(0, 0.0), (100, 0.0), (37, 5.0)])
def test_attention(lens, Hk, group, D, page, dtype, window, cap):
    g = gen(sum(lens) + D)
    kp, vp, table, n, keys = cache(lens, page, Hk, D, DT[dtype], g)
    q = torch.randn(len(lens), Hk * group, D, generator=g, device="cuda").to(DT[dtype])
    out, lse = torch.full_like(q, 7.0), torch.full((len(lens), Hk * group), 7.0, device="cuda")
    tgc.tgc_paged_attention(q, out, kp, vp, table, n, lse=lse, window=window, softcap=cap)
    check(out, lse, q, keys, D ** -0.5, window, cap)


@pytest.mark.parametrize("dtype", list(DT))
def test_strides_and_layouts(dtype):
    g = gen(9)
    lens, Hk, group, D, page = [130, 0, 77, 300], 2, 4, 64, 16
    for heads_first in (False, True):
        kp, vp, table, n, keys = cache(lens, page, Hk, D, DT[dtype], g, heads_first=heads_first, wide=9)
        rows = torch.randn(len(lens), Hk * group + 5, D + 8, generator=g, device="cuda").to(DT[dtype])
        before = rows.clone()
        q = rows[:, 2:2 + Hk * group, :D]
        tgc.tgc_paged_attention(q, q, kp, vp, table, n, scale=0.3)  # over its own queries
        check(q, None, before[:, 2:2 + Hk * group, :D], keys, 0.3)
        around = torch.ones_like(rows, dtype=torch.bool)
        around[:, 2:2 + Hk * group, :D] = False
        assert torch.equal(rows[around], before[around])
        out = torch.empty(len(lens), Hk * group, D, device="cuda", dtype=DT[dtype])
        tgc.tgc_paged_attention(before[:, 2:2 + Hk * group, :D], out, kp, vp, table[:, :table.shape[1] - 5], n)
        check(out, None, before[:, 2:2 + Hk * group, :D], keys, D ** -0.5)
    # keys and values of a page side by side
    both = torch.randn(20, 2, page, Hk, D, generator=g, device="cuda").to(DT[dtype])
    table = torch.randperm(20, generator=g, device="cuda").to(torch.int32).view(2, 10)
    n = torch.tensor([150, 90], device="cuda", dtype=torch.int32)
    q = torch.randn(2, Hk, D, generator=g, device="cuda").to(DT[dtype])
    out = torch.empty_like(q)
    tgc.tgc_paged_attention(q, out, both[:, 0], both[:, 1], table, n)
    keys = [both[table[s].long()].transpose(0, 1).reshape(2, 10 * page, Hk, D)[:, :int(n[s])] for s in range(2)]
    check(out, None, q, keys, D ** -0.5)


@pytest.mark.parametrize("n", [1, 2, 64, 256, 4096, 32768])
@pytest.mark.parametrize("dtype", list(DT))
def test_whole_numbers_are_exact(n, dtype):
    """A query of zeros weighs n = 2^k keys alike: the mean of whole numbers, rounded once.  A query that meets one key
    by 2^10 more than the others takes its value alone."""
    g = gen(n)
    Hk, group, D, page = 2, 4, 64, 16
    kp, vp, table, lens, _ = cache([n], page, Hk, D, DT[dtype], g)
    j = torch.arange(n, device="cuda")
    at = table[0, j // page].long()
    v = torch.randint(-8, 9, (n, Hk, D), generator=g, device="cuda").to(DT[dtype])
    k = torch.zeros(n, Hk, D, device="cuda", dtype=DT[dtype])
    picked = torch.randint(0, n, (Hk * group,), generator=g, device="cuda")
    for h in range(Hk * group):
        k[picked[h], h // group, h] = 64.0
    kp[at, j % page], vp[at, j % page] = k, v
    q = torch.zeros(1, Hk * group, D, device="cuda", dtype=DT[dtype])
    out, lse = torch.empty_like(q), torch.empty(1, Hk * group, device="cuda")
    tgc.tgc_paged_attention(q, out, kp, vp, table, lens, lse=lse)
    mean = (v.double().sum(0) / n).repeat_interleave(group, 0).to(DT[dtype])
    assert torch.equal(out[0], mean)
    assert bool((lse - math.log(n)).abs().max() <= 2 ** -22 * max(1.0, math.log(n)))
    for h in range(Hk * group):
        q[0, h, h] = 64.0
    tgc.tgc_paged_attention(q, out, kp, vp, table, lens, scale=0.25)
    want = torch.stack([v[picked[h], h // group] for h in range(Hk * group)])
    same = torch.stack([(k[:, h // group, h] != 0).sum() for h in range(Hk * group)])
    assert bool((same == 1).all()) and torch.equal(out[0], want)


def test_bad_pages_and_lengths():
    """Numbers outside the pool leave their keys out; lengths are taken as what the table can hold."""
    g = gen(4)
    Hk, group, D, page = 2, 2, 64, 16
    kp, vp, table, lens, keys = cache([300, 200, 64, 100], page, Hk, D, torch.bfloat16, g)
    q = torch.randn(4, Hk * group, D, generator=g, device="cuda").bfloat16()
    table[0, 3], table[0, 18], table[1, 0], table[2, :] = -1, kp.shape[0], 2 ** 31 - 1, -(2 ** 31)
    lens[3] = -5
    out, lse = torch.empty_like(q), torch.empty(4, Hk * group, device="cuda")
    tgc.tgc_paged_attention(q, out, kp, vp, table, lens, lse=lse)
    for s, bad in enumerate([(3, 18), (0,), range(4)]):
        gone = torch.zeros(keys[s].shape[1], dtype=torch.bool, device="cuda")
        for b in bad:
            gone[b * page:(b + 1) * page] = True
        want, want_lse, tol, _ = expect(q[s], keys[s], D ** -0.5, gone=gone)
        assert bool(((out[s].double() - want).abs() <= tol + 2 ** -8 * (want.abs() + tol)).all())
        assert bool((torch.isinf(lse[s]) == torch.isinf(want_lse)).all())
    assert bool((out[3] == 0).all()) and bool((lse[3] == -math.inf).all())
    # longer than the table: every page that it has
    kp, vp, table, lens, keys = cache([160], page, Hk, D, torch.bfloat16, g)
    lens[0] = 2 ** 31 - 1
    tgc.tgc_paged_attention(q[:1], out[:1], kp, vp, table, lens)
    check(out[:1], None, q[:1], keys, D ** -0.5)


def test_bad_pages_of_many_sequences():
    """The same where every warp has a key head of its own, heads and tokens in either order."""
    g = gen(14)
    Hk, group, D, page = 8, 3, 64, 16
    for heads_first in (False, True):
        lens = [(s * 53) % 400 for s in range(48)]
        kp, vp, table, n, keys = cache(lens, page, Hk, D, torch.bfloat16, g, heads_first=heads_first)
        q = torch.randn(48, Hk * group, D, generator=g, device="cuda").bfloat16()
        bad = torch.rand(table.shape, generator=g, device="cuda") < 0.3
        table[bad] = torch.tensor([-1, kp.shape[0], 2 ** 31 - 1, -(2 ** 31)], device="cuda", dtype=torch.int32)[
            torch.randint(0, 4, (int(bad.sum()),), generator=g, device="cuda")]
        out, lse = torch.full_like(q, 7.0), torch.full((48, Hk * group), 7.0, device="cuda")
        tgc.tgc_paged_attention(q, out, kp, vp, table, n, lse=lse)
        for s in range(48):
            gone = bad[s].repeat_interleave(page)[:lens[s]]
            want, want_lse, tol, tol_lse = expect(q[s], keys[s], D ** -0.5, gone=gone)
            assert bool(((out[s].double() - want).abs() <= tol + 2 ** -8 * (want.abs() + tol)).all()), s
            assert torch.equal(torch.isinf(lse[s]), torch.isinf(want_lse))
            live = ~torch.isinf(want_lse)
            assert bool(((lse[s].double() - want_lse).abs()[live] <= tol_lse[live]).all()), s


def test_nothing_to_attend_to():
    """No sequences; a table without pages; a pool without pages; all lengths zero, in runs and in clusters."""
    ints = dict(device="cuda", dtype=torch.int32)
    kp = torch.full((3, 4, 2, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    for S, table, pool, n in ((0, torch.zeros(0, 2, **ints), kp, 0), (3, torch.zeros(3, 0, **ints), kp, 5),
                              (3, torch.zeros(3, 2, **ints), kp[:0], 5), (3, torch.zeros(3, 2, **ints), kp, 0),
                              (400, torch.zeros(400, 2, **ints), kp, 0), (400, torch.zeros(400, 0, **ints), kp, 9)):
        q = torch.randn(S, 4, 64, device="cuda").bfloat16()
        out, lse = torch.full_like(q, 7.0), torch.full((S, 4), 7.0, device="cuda")
        tgc.tgc_paged_attention(q, out, pool, pool, table, torch.full((S,), n, **ints), lse=lse)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_many_sequences():
    """More sequences than threads look at in one go, most of them empty."""
    g = gen(12)
    lens = [0] * 3000
    for s in (0, 5, 31, 32, 700, 1500, 2998, 2999):
        lens[s] = 1 + s % 97
    kp, vp, table, n, keys = cache(lens, 16, 2, 64, torch.bfloat16, g)
    q = torch.randn(3000, 4, 64, generator=g, device="cuda").bfloat16()
    out, lse = torch.full_like(q, 7.0), torch.full((3000, 4), 7.0, device="cuda")
    tgc.tgc_paged_attention(q, out, kp, vp, table, n, lse=lse)
    some = [s for s in range(3000) if lens[s]]
    check(out[some], lse[some], q[some], [keys[s] for s in some], 0.125)
    gone = [s for s in range(3000) if not lens[s]]
    assert bool((out[gone] == 0).all()) and bool((lse[gone] == -math.inf).all())


def test_large_scores_and_infinities():
    """Scores of thousands do not overflow; a row whose scores fall from step to step keeps its first maximum."""
    g = gen(6)
    n, D, page = 700, 64, 16
    kp, vp, table, lens, keys = cache([n], page, 1, D, torch.bfloat16, g)
    j = torch.arange(n, device="cuda")
    at = table[0, j // page].long()
    for k in (torch.linspace(-200, 200, n, device="cuda"), torch.linspace(200, -200, n, device="cuda")):
        keys[0][0] = k.bfloat16()[:, None, None].expand(n, 1, D)
        kp[at, j % page] = keys[0][0]
        q = torch.full((1, 2, D), 4.0, device="cuda", dtype=torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty(1, 2, device="cuda")
        tgc.tgc_paged_attention(q, out, kp, vp, table, lens, lse=lse, scale=1.0)
        # scores are whole multiples of 2^-1 up to 51200: exact in fp32; times log2(e), 2^-24 of 73866 off: 2^-7.8 in powers
        # of two, twice (score and maximum), so probabilities by a factor of 1 + 2^-7.3
        want, want_lse, _, _ = expect(q[0], keys[0], 1.0)
        p_abs = keys[0][1].double().abs().max()
        assert bool(((out[0].double() - want).abs() <= (2 ** -7 + 2 ** -8) * p_abs).all())
        assert bool(((lse[0].double() - want_lse).abs() <= want_lse.abs() * 2 ** -22).all())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("at", [0, 500, 999])
def test_small_probabilities_count(dtype, at):
    """One key, whose value is zero, weighs e^17.7 as much as each of the others: what is left of those 999 is below fp16's
    normal range, and is the output."""
    g = gen(at)
    n, D, page, S = 1000, 64, 16, 200
    kp, vp, table, lens, keys = cache([n] * S, page, 1, D, DT[dtype], g)
    j = torch.arange(n, device="cuda")
    for s, kv in enumerate(keys):
        kv[0] = 0.0
        kv[0, at, 0, 0] = 17.6875 if dtype == "f16" else 17.75
        kv[1] = kv[1].abs() * 64
        kv[1, at] = 0.0
        where = table[s, j // page].long()
        kp[where, j % page], vp[where, j % page] = kv[0], kv[1]
    q = torch.zeros(S, 2, D, device="cuda", dtype=DT[dtype])
    q[:, :, 0] = 1.0
    out, lse = torch.empty_like(q), torch.empty(S, 2, device="cuda")
    tgc.tgc_paged_attention(q, out, kp, vp, table, lens, lse=lse, scale=1.0)
    check(out, lse, q, keys, 1.0)


def test_same_bits_streams_and_graphs():
    g = gen(8)
    lens, Hk, group, D, page = [3000, 10, 5000, 777, 0, 64], 4, 4, 128, 16
    kp, vp, table, n, keys = cache(lens, page, Hk, D, torch.bfloat16, g)
    q = torch.randn(len(lens), Hk * group, D, generator=g, device="cuda").bfloat16()
    first = torch.empty_like(q)
    tgc.tgc_paged_attention(q, first, kp, vp, table, n)
    for _ in range(20):
        out = torch.empty_like(q)
        tgc.tgc_paged_attention(q, out, kp, vp, table, n)
        assert torch.equal(out, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    tgc.tgc_paged_attention(q, out, kp, vp, table, n, stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    # captured: the lengths are read when it is replayed
    ws = torch.empty(tgc.tgc_paged_attention_workspace_bytes(q, out, kp, vp, table, n), device="cuda", dtype=torch.uint8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tgc.tgc_paged_attention(q, out, kp, vp, table, n, workspace=ws)
    graph.replay()
    assert torch.equal(out, first)
    n.copy_(torch.tensor([17, 10, 1234, 0, 0, 1], device="cuda"))
    graph.replay()
    check(out, None, q, [kv[:, :m] for kv, m in zip(keys, n.tolist())], D ** -0.5)


def test_two_calls_at_once():
    """Two streams, a workspace each (torch's allocator gives each stream its own)."""
    g = gen(10)
    sets = []
    for i in range(2):
        kp, vp, table, n, _ = cache([20000 + i, 300], 16, 2, 128, torch.bfloat16, g)
        q = torch.randn(2, 8, 128, generator=g, device="cuda").bfloat16()
        alone = torch.empty_like(q)
        tgc.tgc_paged_attention(q, alone, kp, vp, table, n)
        sets.append((q, kp, vp, table, n, alone, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[torch.empty_like(s[0]) for _ in range(30)] for s in sets]
    for i in range(30):
        for s, o in zip(sets, outs):
            tgc.tgc_paged_attention(s[0], o[i], *s[1:5], stream=s[6])
    torch.cuda.synchronize()
    for s, o in zip(sets, outs):
        assert all(torch.equal(x, s[5]) for x in o)


def test_a_long_cache_far_into_its_pool():
    """Keys more than 2^31 elements from the pool's start."""
    D, Hk, page = 128, 8, 64
    n = (1 << 31) // (D * Hk * page) + 40
    kp, vp = (torch.zeros(n, page, Hk, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    g = gen(2)
    table = (n - 1 - torch.arange(30, device="cuda", dtype=torch.int32))[None]
    kv = torch.randn(2, 30 * page, Hk, D, generator=g, device="cuda").bfloat16()
    j = torch.arange(30 * page, device="cuda")
    kp[table[0, j // page].long(), j % page], vp[table[0, j // page].long(), j % page] = kv[0], kv[1]
    q = torch.randn(1, 2 * Hk, D, generator=g, device="cuda").bfloat16()
    out = torch.empty_like(q)
    lens = torch.tensor([30 * page - 5], device="cuda", dtype=torch.int32)
    tgc.tgc_paged_attention(q, out, kp, vp, table, lens)
    check(out, None, q, [kv[:, :30 * page - 5]], D ** -0.5)


def test_the_binding_refuses():
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    kp = torch.zeros(5, 8, 2, 64, device="cuda", dtype=torch.bfloat16)
    table, n = torch.zeros(2, 3, device="cuda", dtype=torch.int32), torch.zeros(2, device="cuda", dtype=torch.int32)
    for call in (lambda: tgc.tgc_paged_attention(q, q, kp, kp, table[:1], n), lambda: tgc.tgc_paged_attention(q, q, kp, kp, table, n[:1]),
                 lambda: tgc.tgc_paged_attention(q, q, kp.half(), kp.half(), table, n), lambda: tgc.tgc_paged_attention(q, q, kp, kp[:4], table, n),
                 lambda: tgc.tgc_paged_attention(q, q, kp[..., :32], kp[..., :32], table, n),
                 lambda: tgc.tgc_paged_attention(q, q[:, :2], kp, kp, table, n), lambda: tgc.tgc_paged_attention(q, q, kp, kp, table, n.long()),
                 lambda: tgc.tgc_paged_attention(q, q, kp, kp, table, n, lse=torch.zeros(2, 4, device="cuda").half()),
                 lambda: tgc.tgc_paged_attention(q, q, kp[:, :, :1].expand(5, 8, 2, 64), kp[:, :, :1].expand(5, 8, 2, 64), table, n)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: tgc.tgc_paged_attention(q[:, :3], q[:, :3], kp, kp, table, n), lambda: tgc.tgc_paged_attention(q, q, kp, kp, table, n, window=-1),
                 lambda: tgc.tgc_paged_attention(q.float(), q.float(), kp.float(), kp.float(), table, n),
                 lambda: tgc.tgc_paged_attention(q, q, kp, kp, table.repeat(1, 3000), n, workspace=torch.zeros(8, device="cuda", dtype=torch.uint8))):
        with pytest.raises(tgc.TGCError):
            call()
