"""Rotary positions and appending to a paged cache, against the formulas in 64 bits.

Tolerance: an output a cos - b sin (times scale) is rounded once, by half a step of its type.  Before that fp32:
the angle's remainder in turns is rounded (2^-26 turns, 2^-23.3 radians), sine and cosine are off by at most 2
units (2^-23 each), scaled (2^-24), multiplied and added (3 times 2^-24): together under 2^-21 of |a| + |b| times scale.
f16 keeps 2^-25 absolute near zero."""
import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tests.helpers import requires_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    requires_gpu()


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def split(x, R, layout):
    return (x[..., :R // 2], x[..., R // 2:R]) if layout == "half" else (x[..., 0:R:2], x[..., 1:R:2])


def turned(x, pos, freqs, layout, scale=1.0, back=False):
    """The result in 64 bits and its tolerance before the last rounding."""
    R, x = 2 * len(freqs), x.double()
    w = pos.double()[:, None, None] * freqs * (-1 if back else 1)
    a, b = split(x, R, layout)
    out, tol = x.clone(), torch.zeros_like(x)
    oa, ob = split(out, R, layout)
    na, nb = scale * (a * w.cos() - b * w.sin()), scale * (b * w.cos() + a * w.sin())
    oa.copy_(na)
    ob.copy_(nb)
    for t in split(tol, R, layout):
        t.copy_((a.abs() + b.abs()) * abs(scale) * 2 ** -21)
    return out, tol


def check(got, x, pos, freqs, layout, scale=1.0, back=False):
    want, tol = turned(x, pos, freqs, layout, scale, back)
    half = torch.finfo(got.dtype).eps / 2
    tol = tol + half * (want.abs() + tol) + (2 ** -25 if got.dtype == torch.float16 else 0)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    R = 2 * len(freqs)
    assert torch.equal(got[..., R:], x[..., R:])


def positions(T, far, g):
    return torch.randint(0, far + 1, (T,), generator=g, device="cuda", dtype=torch.int32)


SIZES = [(1, 1, 1, 2, 2), (1, 32, 8, 128, 128), (5, 3, 1, 64, 32), (7, 6, 3, 90, 34), (33, 4, 2, 80, 20), (3, 2, 2, 66, 66),
         (2, 1, 1, 1024, 1024), (2500, 4, 1, 64, 64), (1300, 5, 0, 36, 12), (2, 300, 7, 16, 16), (6000, 2, 2, 24, 8), (1, 1, 0, 3, 2)]


@pytest.mark.parametrize("T,Hq,Hk,D,R", SIZES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("back", [False, True])
def test_rope(T, Hq, Hk, D, R, layout, dtype, back):
    g = gen(T + D)
    rows = torch.randn(T, Hq + Hk, D, generator=g, device="cuda").to(DT[dtype])
    q, k = rows[:, :Hq], rows[:, Hq:] if Hk else None
    pos = positions(T, 1000000, g)
    freqs, scale = tgc.tgc_rope_freqs(R, 10000.0, scaling="yarn", factor=4.0, trained=4096.0)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan")) if Hk else None
    if back:
        tgc.tgc_rope_bwd(q, qo, pos, freqs, dk_out=k, dk=ko, layout=layout, scale=scale)
    else:
        tgc.tgc_rope(q, qo, pos, freqs, k=k, k_out=ko, layout=layout, scale=scale)
    check(qo, q, pos, freqs, layout, scale, back)
    if Hk:
        check(ko, k, pos, freqs, layout, scale, back)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions_against_extended_angles(layout):
    """pos * freq with every bit of the product, modulo a turn, by whole-number arithmetic in Python."""
    import math
    from fractions import Fraction
    R, pos = 8, [0, 1, 4097, 999983, 16777217, 2 ** 31 - 1]
    freqs, _ = tgc.tgc_rope_freqs(R)
    q = torch.zeros(len(pos), 1, R, device="cuda")
    a, b = split(q, R, layout)
    a.fill_(1.0)  # (1, 0) turns into (cos, sin)
    tgc.tgc_rope(q, q, torch.tensor(pos, device="cuda", dtype=torch.int32), freqs, layout=layout)
    turn = Fraction(2 * 31415926535897932384626433832795028841971, 10 ** 40)
    for t, p in enumerate(pos):
        for i, f in enumerate(freqs.tolist()):
            w = Fraction(f) * p
            w = float(w - turn * (w // turn))
            # beyond the tolerance above: the product in 64 bits is off by 2^-53 of itself, its turns by 2^-52
            tol = 2 ** -21 + 3 * 2 ** -53 * p * f
            assert abs(float(a[t, 0, i]) - math.cos(w)) <= tol and abs(float(b[t, 0, i]) - math.sin(w)) <= tol, (p, i)


@pytest.mark.parametrize("dtype", list(DT))
def test_in_place_strides_and_padding(dtype):
    g = gen(3)
    T, H, D, R = 11, 5, 64, 32
    freqs, _ = tgc.tgc_rope_freqs(R)
    pos = positions(T, 500, g)
    pos[4], pos[10] = -1, -7
    for view in (lambda s: s[:, :H, :D], lambda s: s[:, 1:H + 1, 8:D + 8], lambda s: s[:, :H, 1:D + 1],
                 lambda s: s.permute(0, 1, 2)[:, 2:H + 2, :D]):
        store = torch.randn(T, H + 3, D + 16, generator=g, device="cuda").to(DT[dtype])
        before = store.clone()
        x = view(store)
        tgc.tgc_rope(x, x, pos, freqs)
        live = pos >= 0
        check(view(store)[live], view(before)[live], pos[live], freqs, "half")
        assert torch.equal(view(store)[~live], view(before)[~live])
        mask = torch.ones_like(store, dtype=torch.bool)
        view(mask).fill_(False)
        assert torch.equal(store[mask], before[mask])  # nothing around it is written
    # heads outside tokens: (H, T, D) memory
    store = torch.randn(H, T, D, generator=g, device="cuda").to(DT[dtype])
    x, out = store.transpose(0, 1), torch.empty(T, H, D, device="cuda", dtype=DT[dtype])
    tgc.tgc_rope(x, out, pos.abs(), freqs, layout="interleaved")
    check(out, x, pos.abs(), freqs, "interleaved")


def test_rotating_back_and_gradients():
    """The backward pass is the transpose: <rope(x), y> = <x, rope_bwd(y)>, and differences of rope along a direction
    are its values (it is linear): in fp32, sums of 4096 products, each off by 2^-20 of its size."""
    g = gen(5)
    T, H, D, R = 16, 4, 64, 48
    freqs, scale = tgc.tgc_rope_freqs(R, scaling="yarn", factor=2.0, trained=100.0)
    pos = positions(T, 100000, g)
    for layout in ("half", "interleaved"):
        x, y = (torch.randn(T, H, D, generator=g, device="cuda") for _ in range(2))
        fx, by = torch.empty_like(x), torch.empty_like(x)
        tgc.tgc_rope(x, fx, pos, freqs, layout=layout, scale=scale)
        tgc.tgc_rope_bwd(y, by, pos, freqs, layout=layout, scale=scale)
        left, right = (fx.double() * y.double()).sum(), (x.double() * by.double()).sum()
        assert abs(float(left - right)) <= 2 ** -19 * float((fx.double() * y.double()).abs().sum() + (x.double() * by.double()).abs().sum())
        leaf = x.double().requires_grad_()
        w = pos.double()[:, None, None] * freqs
        a, b = split(leaf, R, layout)
        na, nb = scale * (a * w.cos() - b * w.sin()), scale * (b * w.cos() + a * w.sin())
        ya, yb = split(y.double(), R, layout)
        ((na * ya).sum() + (nb * yb).sum() + (leaf[..., R:] * y[..., R:]).sum()).backward()
        assert float((by.double() - leaf.grad).abs().max()) <= 2 ** -20 * float(y.abs().max()) * 2 * scale


def paged(S, max_pages, spare, g):
    """A shuffled table in which every sequence has all its pages, and the number of pages."""
    n = S * max_pages + spare
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)[:S * max_pages].view(S, max_pages).contiguous(), n


@pytest.mark.parametrize("T,S,Hq,Hk,D,R,page,dtype,layout", [
    (1, 1, 32, 8, 128, 128, 16, "bf16", "half"), (64, 64, 8, 2, 128, 64, 64, "f16", "interleaved"),
    (100, 3, 4, 4, 64, 64, 5, "bf16", "half"), (37, 4, 3, 1, 90, 34, 1, "f32", "interleaved"),
    (900, 7, 0, 2, 80, 0, 24, "f16", "half"), (3000, 2, 2, 2, 64, 64, 100, "bf16", "interleaved"),
    (9, 2, 5, 1, 33, 22, 3, "bf16", "half")])
@pytest.mark.parametrize("heads_first", [False, True])
def test_append(T, S, Hq, Hk, D, R, page, dtype, layout, heads_first):
    g = gen(T)
    dt = DT[dtype]
    rows = torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda").to(dt)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
    max_pages = -(-(T // S + 40) // page)
    table, n = paged(S, max_pages, 3, g)
    seqs = (torch.arange(T, device="cuda") % S).to(torch.int32)
    pos = (torch.arange(T, device="cuda") // S + 7).to(torch.int32)
    if T > 20:
        pos[3] = -1                        # padding
        pos[5] = max_pages * page          # past the table
        seqs[6], seqs[8] = S, -1           # no such sequence
        table[int(seqs[9]), int(pos[9]) // page] = n  # a page that is none
    shape = (n, Hk, page, D) if heads_first else (n, page, Hk, D)
    stores = [torch.randn(*shape, generator=g, device="cuda").to(dt) for _ in range(2)]
    kp, vp = (s.transpose(1, 2) if heads_first else s for s in stores)
    want_k, want_v = kp.double().clone(), vp.clone()
    freqs = tgc.tgc_rope_freqs(R)[0] if R else None
    qo = torch.full_like(q, 9.0) if Hq else None
    tgc.tgc_kv_append(k, v, kp, vp, table, pos, seqs=None if S == T else seqs, q=q if Hq else None, q_out=qo, freqs=freqs, layout=layout)
    f = freqs if R else torch.zeros(0, device="cuda", dtype=torch.float64)
    rk, tk = turned(k, pos, f, layout)
    tol = torch.zeros_like(want_k)
    for t in range(T):
        s, p = t if S == T else int(seqs[t]), int(pos[t])
        if p < 0 or not 0 <= s < S or p // page >= max_pages or int(table[s, p // page]) >= n:
            continue
        at = int(table[s, p // page])
        want_k[at, p % page], want_v[at, p % page] = rk[t], v[t]
        tol[at, p % page] = tk[t] + torch.finfo(dt).eps / 2 * (rk[t].abs() + tk[t]) + 2 ** -25
    assert bool(((kp.double() - want_k).abs() <= tol).all())
    assert torch.equal(vp, want_v)
    if Hq:
        live = pos >= 0
        check(qo[live], q[live], pos[live], f, layout)
        assert bool((qo[~live] == 9.0).all())


def test_the_most_heads_and_none():
    freqs, _ = tgc.tgc_rope_freqs(2)
    q = torch.randn(1, 65536, 1024, generator=gen(), device="cuda").half()
    out, pos = torch.empty_like(q), torch.tensor([5], device="cuda", dtype=torch.int32)
    tgc.tgc_rope(q, out, pos, freqs)
    for h in (slice(0, 40), slice(32700, 32800), slice(65500, 65536)):
        check(out[:, h], q[:, h], pos, freqs, "half")
    nothing = torch.zeros(0, dtype=torch.int32, device="cuda")
    tgc.tgc_rope(q[:0], q[:0], nothing, freqs)
    kp = torch.full((2, 4, 3, 8), 7.0, device="cuda")
    tgc.tgc_kv_append(kp[0, :0], kp[0, :0], kp, kp.clone(), torch.zeros(1, 2, device="cuda", dtype=torch.int32), nothing)
    assert bool((kp == 7).all())


def test_another_stream_and_a_graph():
    """Rotation, its gradients and appending on another stream and replayed from a graph: the same bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    ints = dict(device="cuda", dtype=torch.int32)
    T, H, K, D = 37, 6, 2, 64
    rows = torch.randn(T, H + 2 * K, D, generator=g, device="cuda").bfloat16()
    pos, seqs = torch.randint(0, 60, (T,), generator=g, **ints), torch.arange(T, **ints)
    table = torch.randperm(T * 4, generator=g, device="cuda").to(torch.int32).view(T, 4)
    freqs, _ = tgc.tgc_rope_freqs(D, device="cuda")

    def work(stream=None):
        o = [torch.zeros(T, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
        pools = [torch.zeros(T * 4, 16, K, D, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        here = torch.cuda.current_stream()
        if stream is not None:
            stream.wait_stream(here)
        on = {} if stream is None else dict(stream=stream)
        tgc.tgc_rope(rows[:, :H], o[0], pos, freqs, **on)
        tgc.tgc_rope_bwd(o[0], o[1], pos, freqs, **on)
        tgc.tgc_kv_append(rows[:, H:H + K], rows[:, H + K:], *pools, table, pos, seqs=seqs, q=rows[:, :H], q_out=o[2], freqs=freqs, **on)
        if stream is not None:
            here.wait_stream(stream)
        return o + pools

    want = work()
    assert torch.equal(want[0], want[2]) and bool(want[3].any())
    for a, b in zip(want, work(torch.cuda.Stream())):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(2):
        graph.replay()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_a_far_page_of_a_large_pool():
    """Pages more than 2^31 elements from the pool's start."""
    D, Hk, page = 128, 8, 64
    n = (1 << 31) // (D * Hk * page) + 3
    kp = torch.zeros(n, page, Hk, D, device="cuda", dtype=torch.bfloat16)
    vp = torch.zeros_like(kp)
    k, v = (torch.randn(2, Hk, D, generator=gen(s), device="cuda").bfloat16() for s in (1, 2))
    table = torch.tensor([[n - 1], [n - 2]], device="cuda", dtype=torch.int32)
    pos = torch.tensor([63, 0], device="cuda", dtype=torch.int32)
    tgc.tgc_kv_append(k, v, kp, vp, table, pos)
    for s, (p, o) in enumerate(((n - 1, 63), (n - 2, 0))):
        assert torch.equal(kp[p, o], k[s]) and torch.equal(vp[p, o], v[s])
    assert int(torch.count_nonzero(kp[:n - 2])) == 0


def test_the_binding_refuses():
    x = torch.zeros(4, 2, 8, device="cuda")
    pos = torch.zeros(4, device="cuda", dtype=torch.int32)
    f = torch.zeros(4, device="cuda", dtype=torch.float64)
    kp, table = torch.zeros(3, 2, 2, 8, device="cuda"), torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    for call in (lambda: tgc.tgc_rope(x, x[:3], pos, f), lambda: tgc.tgc_rope(x, x, pos.long(), f),
                 lambda: tgc.tgc_rope(x, x, pos, f.float()), lambda: tgc.tgc_rope(x, x, pos[:3], f),
                 lambda: tgc.tgc_rope(x, x, pos, f, k=x), lambda: tgc.tgc_rope(x, x.half(), pos, f),
                 lambda: tgc.tgc_rope(x[..., ::2], x[..., ::2], pos, f[:2]), lambda: tgc.tgc_rope(x[:1].expand(4, 2, 8), x, pos, f),
                 lambda: tgc.tgc_kv_append(x, x, kp, kp[:2], table, pos), lambda: tgc.tgc_kv_append(x, x, kp.half(), kp, table, pos),
                 lambda: tgc.tgc_kv_append(x, x, kp, kp, table.long(), pos), lambda: tgc.tgc_kv_append(x[:, :1], x[:, :1], kp, kp, table, pos),
                 lambda: tgc.tgc_kv_append(x, x, kp, kp, table, pos, q=x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(tgc.TGCError):  # more elements to turn than a head has
        tgc.tgc_rope(x, x, pos, torch.zeros(5, device="cuda", dtype=torch.float64))
    with pytest.raises(tgc.TGCError):  # four tokens, two sequences, and no seqs
        tgc.tgc_kv_append(x, x, kp, kp, table[:2], pos)
