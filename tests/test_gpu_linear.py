"""tgc_linear and tgc_linear_bwd on the GPU against the formulas in 64 bits.

Two kinds of comparison.  With small whole numbers as inputs every product and sum is exact in
fp32, so the output has to be the 64-bit result rounded once: bit equality, at every size, stride
and grouping where an index can go wrong.  With normal inputs the bound is the worst case of the
roundings: u |result| for the output (u = 2^-8 bf16, 2^-10 f16: one unit in the last place), 2^-23 a step of a sum of
n terms against the sum of their magnitudes, 2^-20 for an activation's exp and division."""
import math

import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tests.helpers import requires_gpu

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, F16: 2.0 ** -10}
TINY = {BF: 1e-38, F16: 2.0 ** -24}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(autouse=True)
def _gpu():
    requires_gpu()


def act64(z, act):
    return {"none": lambda v: v, "relu": torch.relu,  # derivative 0 at 0
            "gelu": lambda v: 0.5 * v * (1 + torch.erf(v / math.sqrt(2))),
            "gelu_tanh": lambda v: 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))),
            "silu": lambda v: v / (1 + torch.exp(-v))}[act](z)


def act_grad64(z, act):
    z = z.clone().requires_grad_()
    return torch.autograd.grad(act64(z, act).sum(), z)[0] if act != "none" else torch.ones_like(z)


def ints(g, *shape, lo=-2, hi=3, dtype=BF):
    return torch.randint(lo, hi, shape, generator=g, device="cuda").to(dtype)


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def groups_of(offsets, M):
    return [(offsets[i], offsets[i + 1]) for i in range(len(offsets) - 1)]


def forward64(x, w, b, res, act, offsets=None):
    x, w = x.double(), w.double()
    if offsets is None:
        z = x @ w.t() + (b.double() if b is not None else 0)
    else:
        z = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
        for e, (i, j) in enumerate(groups_of(offsets, x.shape[0])):
            z[i:j] = x[i:j] @ w[e].t() + (b[e].double() if b is not None else 0)
    return z, act64(z, act) + (res.double() if res is not None else 0)


def backward64(dy, x, w, z, act, offsets=None):
    x, w, dz = x.double(), w.double(), dy.double()
    if act != "none":
        dz = dz * act_grad64(z.double(), act)
    if offsets is None:
        return dz @ w, dz.t() @ x, dz.sum(0), dz
    dx = torch.zeros_like(x)
    dw, db = torch.zeros_like(w), torch.zeros_like(w[:, :, 0])
    for e, (i, j) in enumerate(groups_of(offsets, x.shape[0])):
        dx[i:j], dw[e], db[e] = dz[i:j] @ w[e], dz[i:j].t() @ x[i:j], dz[i:j].sum(0)
    return dx, dw, db, dz


SHAPES = [(1, 8, 8), (1, 64, 256), (2, 72, 264), (7, 200, 136), (31, 512, 64), (33, 4104, 24), (64, 136, 520),
          (127, 320, 128), (128, 64, 512), (129, 1000, 200), (255, 96, 1032), (257, 648, 264), (300, 8, 2048),
          (513, 192, 768), (1000, 1024, 520), (2050, 72, 136), (48, 7168, 1024), (4096, 64, 64), (5, 16384, 128)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F16])
def test_forward_is_exact_on_whole_numbers(M, K, N, dtype):
    g = gen(M + K + N)
    x, w = ints(g, M, K, dtype=dtype), ints(g, N, K, dtype=dtype, lo=-1, hi=2)
    b, res = ints(g, N, dtype=dtype), ints(g, M, N, dtype=dtype)
    for act, bias, residual, keep in [("none", None, None, False), ("relu", b, None, True), ("none", b, res, True)]:
        y = torch.full((M, N), float("nan"), device="cuda", dtype=dtype)
        z = torch.full_like(y, float("nan")) if keep else None
        tgc.tgc_linear(x, w, y, bias=bias, act=act, residual=residual, z=z)
        z64, y64 = forward64(x, w, bias, residual, act)
        assert torch.equal(y, y64.to(dtype)), (act, residual is not None)
        assert z is None or torch.equal(z, z64.to(dtype))


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype,act", [(BF, "relu"), (F16, "none")])
def test_backward_is_exact_on_whole_numbers(M, K, N, dtype, act):
    g = gen(M + K + N)
    x, w = ints(g, M, K, dtype=dtype, lo=-1, hi=2), ints(g, N, K, dtype=dtype, lo=-1, hi=2)
    dy, z = ints(g, M, N, dtype=dtype), ints(g, M, N, dtype=dtype)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda", dtype=dtype)
    for t in (dx, dw, db):
        t.fill_(float("nan"))
    tgc.tgc_linear_bwd(dy, x, w, z=z, act=act, dx=dx, dw=dw, dbias=db)
    rx, rw, rb, _ = backward64(dy, x, w, z, act)
    assert torch.equal(dx, rx.to(dtype))
    assert torch.equal(dw, rw.to(dtype))
    assert torch.equal(db, rb.to(dtype))


# rows of each expert: empty ones, single rows, odd counts, more than a tile, all rows in one
GROUPS = [[5], [0, 3], [1, 0, 0, 1, 1], [128, 128], [130, 0, 7, 255, 64, 1], [0, 0, 700, 0], [33] * 17, [1] * 70,
          [300, 513, 1, 0, 90, 256, 2], [0, 0, 0]]


@pytest.mark.parametrize("sizes", GROUPS)
@pytest.mark.parametrize("dtype,K,N", [(BF, 136, 264), (F16, 64, 520), (BF, 1032, 72)])
@pytest.mark.parametrize("before,after", [(0, 0), (3, 70)])
def test_experts_are_exact_on_whole_numbers(sizes, dtype, K, N, before, after):
    """Rows before the first and after the last expert hold NaN and are neither read nor written."""
    g = gen(sum(sizes) + K)
    offsets = [before]
    for n in sizes:
        offsets.append(offsets[-1] + n)
    M, En = offsets[-1] + after, len(sizes)
    if M == 0:
        return
    x, w = ints(g, M, K, dtype=dtype, lo=-1, hi=2), ints(g, En, N, K, dtype=dtype, lo=-1, hi=2)
    b, dy, z = ints(g, En, N, dtype=dtype), ints(g, M, N, dtype=dtype), ints(g, M, N, dtype=dtype)
    rx, rw, rb, _ = backward64(dy, x, w, z, "relu", offsets)
    z64, y64 = forward64(x, w, b, None, "relu", offsets)
    for t in (x, dy, z):
        t[:before] = t[offsets[-1]:] = float("nan")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y, zo = (torch.full((M, N), 77.0, device="cuda", dtype=dtype) for _ in range(2))
    tgc.tgc_linear(x, w, y, bias=b, act="relu", z=zo, offsets=off)
    for got, ref in ((y, y64), (zo, z64)):
        ref = ref.to(dtype)
        ref[:before] = ref[offsets[-1]:] = 77.0
        assert torch.equal(got, ref)
    dx, dw, db = torch.full_like(x, 77.0), torch.full_like(w, float("nan")), torch.full_like(b, float("nan"))
    tgc.tgc_linear_bwd(dy, x, w, z=z, act="relu", dx=dx, dw=dw, dbias=db, offsets=off)
    rx = rx.to(dtype)
    rx[:before] = rx[offsets[-1]:] = 77.0
    assert torch.equal(dx, rx)
    assert torch.equal(dw, rw.to(dtype))
    assert torch.equal(db, rb.to(dtype))


# Sizes at which each form of the products is taken: CTA pairs with wide and narrow tiles, single
# CTAs, split reductions of several parts, full tiles with a ragged end's rows beside them.
FORMS = [(777, 4104, 5000), (300, 4096, 4096), (2048, 2048, 2048), (4100, 1032, 2056), (9, 14336, 1024),
         (520, 8192, 520), (1, 4096, 14336), (6000, 264, 3000)]


@pytest.mark.parametrize("M,K,N", FORMS)
def test_every_form_is_exact_on_whole_numbers(M, K, N):
    g = gen(M + N)
    x, w = ints(g, M, K, lo=-1, hi=2), ints(g, N, K, lo=-1, hi=2)
    b, res, dy = ints(g, N), ints(g, M, N), ints(g, M, N, lo=-1, hi=2)
    y, z = (torch.full((M, N), float("nan"), device="cuda", dtype=BF) for _ in range(2))
    tgc.tgc_linear(x, w, y, bias=b, act="relu", residual=res, z=z)
    z64, y64 = forward64(x, w, b, res, "relu")
    assert torch.equal(z, z64.to(BF)) and torch.equal(y, y64.to(BF))
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    tgc.tgc_linear_bwd(dy, x, w, z=z, act="relu", dx=dx, dw=dw, dbias=db)
    rx, rw, rb, _ = backward64(dy, x, w, z, "relu")
    assert torch.equal(dx, rx.to(BF)) and torch.equal(dw, rw.to(BF)) and torch.equal(db, rb.to(BF))


@pytest.mark.parametrize("sizes,K,N", [([700, 0, 1500, 33, 257, 1], 1032, 2056), ([3000, 40], 520, 4096)])
def test_large_experts_are_exact_on_whole_numbers(sizes, K, N):
    g = gen(K)
    offsets = [0]
    for n in sizes:
        offsets.append(offsets[-1] + n)
    M, En = offsets[-1], len(sizes)
    x, w = ints(g, M, K, lo=-1, hi=2), ints(g, En, N, K, lo=-1, hi=2)
    dy, off = ints(g, M, N, lo=-1, hi=2), torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = torch.full((M, N), float("nan"), device="cuda", dtype=BF)
    tgc.tgc_linear(x, w, y, offsets=off)
    assert torch.equal(y, forward64(x, w, None, None, "none", offsets)[1].to(BF))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db = torch.empty(En, N, device="cuda", dtype=BF)
    tgc.tgc_linear_bwd(dy, x, w, dx=dx, dw=dw, dbias=db, offsets=off)
    rx, rw, rb, _ = backward64(dy, x, w, None, "none", offsets)
    assert torch.equal(dx, rx.to(BF)) and torch.equal(dw, rw.to(BF)) and torch.equal(db, rb.to(BF))


def test_many_experts_and_offsets_out_of_range():
    g = gen(1)
    En, K, N = 1024, 64, 64
    sizes = torch.randint(0, 3, (En,), generator=torch.Generator().manual_seed(3)).tolist()
    offsets = [0]
    for n in sizes:
        offsets.append(offsets[-1] + n)
    M = offsets[-1]
    x, w = ints(g, M, K), ints(g, En, N, K)
    y = torch.full((M, N), float("nan"), device="cuda", dtype=BF)
    tgc.tgc_linear(x, w, y, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, forward64(x, w, None, None, "none", offsets)[1].to(BF))
    # values outside [0, M] count as the nearer bound, a group that ends before it begins as empty
    y.fill_(5.0)
    tgc.tgc_linear(x, w[:3], y, offsets=torch.tensor([-40, 10, 4, 1 << 30], dtype=torch.int32, device="cuda"))
    ref = forward64(x, w[:3], None, None, "none", [0, 10, 10, M])[1]
    ref[4:] = forward64(x[4:], w[2], None, None, "none")[1]
    assert torch.equal(y[10:], ref[10:].to(BF)) and torch.equal(y[:4], ref[:4].to(BF))


@pytest.mark.parametrize("M,K,N", [(3, 64, 128), (150, 264, 200), (700, 128, 520)])
def test_strided_operands(M, K, N):
    """Row strides on every operand, NaN in what lies between the rows, and nothing written there."""
    g = gen(5)

    def wide(t, extra, fill):
        buf = torch.full((t.shape[0], t.shape[1] + extra), fill, device="cuda", dtype=t.dtype)
        buf[:, :t.shape[1]] = t
        return buf[:, :t.shape[1]], buf

    nan = float("nan")
    x, _ = wide(ints(g, M, K), 8, nan)
    w, _ = wide(ints(g, N, K), 24, nan)
    res, _ = wide(ints(g, M, N), 16, nan)
    y, ybuf = wide(torch.zeros(M, N, device="cuda", dtype=BF), 40, 9.0)
    z, zbuf = wide(torch.zeros(M, N, device="cuda", dtype=BF), 8, 9.0)
    tgc.tgc_linear(x, w, y, residual=res, z=z)
    z64, y64 = forward64(x, w, None, res, "none")
    assert torch.equal(y, y64.to(BF)) and torch.equal(z, z64.to(BF))
    assert bool((ybuf[:, N:] == 9).all()) and bool((zbuf[:, N:] == 9).all())
    dy, _ = wide(ints(g, M, N), 8, nan)
    zz, _ = wide(ints(g, M, N), 16, nan)
    dx, dxbuf = wide(torch.zeros(M, K, device="cuda", dtype=BF), 8, 9.0)
    dw = torch.empty(N, K, device="cuda", dtype=BF)
    tgc.tgc_linear_bwd(dy, x, w, z=zz, act="relu", dx=dx, dw=dw)
    rx, rw, _, _ = backward64(dy, x, w, zz, "relu")
    assert torch.equal(dx, rx.to(BF)) and torch.equal(dw, rw.to(BF)) and bool((dxbuf[:, K:] == 9).all())


def test_rows_past_32_bit_offsets():
    """Rows that lie more than 2^31 elements apart."""
    g = gen(6)
    M, K, N, ld = 3, 64, 64, (1 << 30) + 8
    buf = torch.empty(2 * ld + 64, device="cuda", dtype=BF)
    x = buf.as_strided((M, K), (ld, 1))
    x.copy_(ints(g, M, K))
    w, y = ints(g, N, K), torch.empty(M, N, device="cuda", dtype=BF)
    tgc.tgc_linear(x, w, y)
    ref = forward64(x, w, None, None, "none")[1].to(BF)
    assert torch.equal(y, ref)
    dy, dw = ints(g, M, N), torch.empty_like(w)
    tgc.tgc_linear_bwd(dy, x, w, dw=dw)
    assert torch.equal(dw, backward64(dy, x, w, None, "none")[1].to(BF))
    out = buf.as_strided((M, N), (ld, 1))
    xs = ints(g, M, K)
    tgc.tgc_linear(xs, w, out)
    assert torch.equal(out, forward64(xs, w, None, None, "none")[1].to(BF))


def test_experts_weights_with_a_stride_between_them():
    g = gen(7)
    big = torch.full((3, 80, 72), float("nan"), device="cuda", dtype=BF)
    big[:, :40, :64] = ints(g, 3, 40, 64)
    w = big[:, :40, :64]
    x, offsets = ints(g, 50, 64), [0, 20, 20, 50]
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = torch.empty(50, 40, device="cuda", dtype=BF)
    tgc.tgc_linear(x, w, y, offsets=off)
    assert torch.equal(y, forward64(x, w, None, None, "none", offsets)[1].to(BF))
    dy, dx = ints(g, 50, 40), torch.empty_like(x)
    tgc.tgc_linear_bwd(dy, x, w, dx=dx, offsets=off)
    assert torch.equal(dx, backward64(dy, x, w, None, "none", offsets)[0].to(BF))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("M,K,N", [(5, 512, 264), (200, 1032, 392)])
def test_activations_and_gradients(act, dtype, M, K, N):
    g = gen(11)
    r = lambda *s, k=1.0: (torch.randn(*s, generator=g, device="cuda") * k).to(dtype)
    x, w, b, res = r(M, K), r(N, K, k=2 / math.sqrt(K)), r(N), r(M, N)
    y, z = (torch.empty(M, N, device="cuda", dtype=dtype) for _ in range(2))
    tgc.tgc_linear(x, w, y, bias=b, act=act, residual=res, z=z)
    z64, y64 = forward64(x, w, b, res, act)
    mag = x.double().abs() @ w.double().abs().t() + b.double().abs()
    ez = (K + 2) * 2.0 ** -23 * mag
    u, tiny = U[dtype], TINY[dtype]
    assert bool(((z.double() - z64).abs() <= u * z64.abs() + ez + tiny).all())
    ey = 1.2 * ez + 2.0 ** -20 * z64.abs() + 2.0 ** -23 * (y64.abs() + res.double().abs())
    assert bool(((y.double() - y64).abs() <= u * y64.abs() + ey + tiny).all())

    dy = r(M, N)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    tgc.tgc_linear_bwd(dy, x, w, z=z, act=act, dx=dx, dw=dw, dbias=db)
    rx, rw, rb, dz = backward64(dy, x, w, z, act)
    edz = dz.abs() * 2.0 ** -20 + dy.double().abs() * 2.0 ** -20 * (1 + z.double().abs())  # fp32 derivative
    rdz = dz.abs() * u + edz + tiny                                                      # and its rounding
    wa, xa = w.double().abs(), x.double().abs()
    assert bool(((dx.double() - rx).abs() <= u * rx.abs() + (rdz + N * 2.0 ** -23 * dz.abs()) @ wa + tiny).all())
    assert bool(((dw.double() - rw).abs() <= u * rw.abs() + (rdz + M * 2.0 ** -23 * dz.abs()).t() @ xa + tiny).all())
    assert bool(((db.double() - rb).abs() <= u * rb.abs() + (edz + M * 2.0 ** -23 * dz.abs()).sum(0) + tiny).all())


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """d/dp of sum(dy * y) by central differences of the 64-bit formula in a random direction p,
    against the same direction of the kernels' gradients (rounded z and dz: 2^-8 a term)."""
    g = gen(12)
    M, K, N, dtype = 24, 64, 40, F16
    r = lambda *s, k=1.0: (torch.randn(*s, generator=g, device="cuda") * k).to(dtype)
    x, w, b, dy = r(M, K), r(N, K, k=0.2), r(N), r(M, N)
    y, z = (torch.empty(M, N, device="cuda", dtype=dtype) for _ in range(2))
    tgc.tgc_linear(x, w, y, bias=b, act=act, z=z)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    tgc.tgc_linear_bwd(dy, x, w, z=z, act=act, dx=dx, dw=dw, dbias=db)
    args = [x.double(), w.double(), b.double()]
    for k, grad in enumerate((dx, dw, db)):
        p = torch.randn(args[k].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        f = []
        for s in (h, -h):
            a = list(args)
            a[k] = a[k] + s * p
            f.append((dy.double() * forward64(*a, None, act)[1]).sum())
        diff = (f[0] - f[1]) / (2 * h)
        scale = (grad.double().abs() * p.abs()).sum()
        kinks = 0.02 if act == "relu" else 0.0  # a step may cross a kink of relu
        assert float((diff - (grad.double() * p).sum()).abs()) <= (2.0 ** -8 + kinks) * float(scale)


def test_nan_and_infinity_stay_in_their_rows():
    g = gen(13)
    for M in (6, 300):
        x, w = ints(g, M, 128), ints(g, 264, 128)
        x[1, 3], x[4, 7] = float("nan"), float("inf")
        w[5, 7] = 1.0
        y = torch.zeros(M, 264, device="cuda", dtype=BF)
        tgc.tgc_linear(x, w, y, act="relu")
        ref = x.clone()
        ref[1], ref[4] = 0, 0
        good = [i for i in range(M) if i not in (1, 4)]
        assert torch.equal(y[good], forward64(ref, w, None, None, "relu")[1].to(BF)[good])
        assert bool(y[1].isnan().all()) and float(y[4, 5]) == float("inf")


def test_residual_in_place_partial_gradients_and_empty():
    g = gen(14)
    for M in (3, 400):
        x, w, y = ints(g, M, 72), ints(g, 136, 72), ints(g, M, 136)
        ref = forward64(x, w, None, y, "none")[1].to(BF)
        tgc.tgc_linear(x, w, y, residual=y)
        assert torch.equal(y, ref)
        dy = ints(g, M, 136)
        rx, rw, rb, _ = backward64(dy, x, w, None, "none")
        dx = torch.empty_like(x)
        tgc.tgc_linear_bwd(dy, x, w, dx=dx)
        assert torch.equal(dx, rx.to(BF))
        db = torch.empty(136, device="cuda", dtype=BF)
        tgc.tgc_linear_bwd(dy, x, w, dbias=db)
        assert torch.equal(db, rb.to(BF))
    dw, db = torch.full_like(w, 3.0), torch.full_like(db, 3.0)
    tgc.tgc_linear_bwd(dy[:0], x[:0], w, dw=dw, dbias=db)
    assert not dw.any() and not db.any()
    tgc.tgc_linear(x[:0], w, y[:0])


def test_same_bits_every_time_on_a_side_stream_and_in_a_graph():
    g = gen(15)
    x = torch.randn(333, 2056, generator=g, device="cuda").to(BF)
    w = torch.randn(520, 2056, generator=g, device="cuda").to(BF)
    dy = torch.randn(333, 520, generator=g, device="cuda").to(BF)
    z = torch.randn(333, 520, generator=g, device="cuda").to(BF)
    bufs = lambda: (torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w[:, 0]).contiguous())

    def run(o, stream=None):
        tgc.tgc_linear(x, w, o[0], act="gelu", stream=stream)
        tgc.tgc_linear_bwd(dy, x, w, z=z, act="gelu", dx=o[1], dw=o[2], dbias=o[3], stream=stream)

    first, other, graphed = bufs(), bufs(), bufs()
    run(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(other, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    run(graphed)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(graphed)
    for t in graphed:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, graphed))


def test_the_binding_refuses_operands_that_do_not_fit():
    x, w = torch.zeros(4, 64, device="cuda", dtype=BF), torch.zeros(32, 64, device="cuda", dtype=BF)
    for y in (torch.zeros(4, 64, device="cuda", dtype=BF), torch.zeros(4, 32, device="cuda", dtype=F16),
              torch.zeros(32, 4, device="cuda", dtype=BF).t()):
        with pytest.raises(ValueError):
            tgc.tgc_linear(x, w, y)
    y = torch.zeros(4, 32, device="cuda", dtype=BF)
    with pytest.raises(ValueError):
        tgc.tgc_linear(x, w, y, bias=torch.zeros(31, device="cuda", dtype=BF))
    with pytest.raises(ValueError):
        tgc.tgc_linear(x, w, y, offsets=torch.zeros(2, device="cuda", dtype=torch.int32))
    with pytest.raises(ValueError):
        tgc.tgc_linear(x, w, y, offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        tgc.tgc_linear_bwd(y, x, w, dw=torch.zeros(64, 32, device="cuda", dtype=BF))
    with pytest.raises(tgc.TGCError):
        tgc.tgc_linear(torch.zeros(4, 63, device="cuda", dtype=BF), torch.zeros(32, 63, device="cuda", dtype=BF), y)


@pytest.mark.parametrize("M,groups", [(1, 0), (300, 0), (300, 3)])
def test_a_workspace_of_the_queried_size_serves_and_a_smaller_one_is_refused(M, groups):
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy, z = ints(g, M, 64), ints(g, M, 48), ints(g, M, 48)
    lead = (groups,) if groups else ()
    w = ints(g, *lead, 48, 64)
    offsets = torch.tensor([0, 7, 7, M], device="cuda", dtype=torch.int32) if groups else None
    out = lambda: dict(dx=torch.empty_like(x), dw=torch.empty_like(w),
                       dbias=torch.empty(*lead, 48, device="cuda", dtype=x.dtype))
    kw, one, own = dict(z=z, act="relu", offsets=offsets), out(), out()
    n = tgc.tgc_linear_bwd_workspace_bytes(dy, x, w, **kw, **one)
    assert n > 0
    tgc.tgc_linear_bwd(dy, x, w, **kw, **one)
    tgc.tgc_linear_bwd(dy, x, w, **kw, **own, workspace=torch.empty(n, device="cuda", dtype=torch.uint8))
    assert all(torch.equal(one[k], own[k]) for k in one)
    with pytest.raises(tgc.TGCError):
        tgc.tgc_linear_bwd(dy, x, w, **kw, **own, workspace=torch.empty(n - 1, device="cuda", dtype=torch.uint8))
