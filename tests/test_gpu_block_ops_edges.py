"""What the transformer-block operators do at the edges of what they accept, on the GPU: offsets that decrease,
host threads that call at the same time, infinities where a term has no factor for them, waits, activations
far from zero."""
import ctypes
import math
import os
import threading

import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tile_gather_comm_gb300 import _build, _lib
from tests.helpers import requires_gpu

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF: 2.0 ** -8, F16: 2.0 ** -10}  # a unit in the last place


@pytest.fixture(autouse=True)
def _gpu():
    requires_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---------------------------------------------------------------- offsets


@pytest.mark.parametrize("M,groups", [(300, 16), (1000, 7), (300, 1000)])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_offsets_that_decrease_stay_inside_the_workspace(M, groups, act):
    """Offsets 0, M, 0, M, ...: every even group has all rows, more chunks in all than the workspace has partial
    sums.  What lies behind the queried size is NaN, far past any place those chunks would have had."""
    g, K, N = gen(M + groups), 64, 48
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(BF)  # noqa: E731
    x, dy, z, w1 = ints(M, K), ints(M, N), ints(M, N), ints(N, K)
    w = w1.expand(groups, N, K).contiguous()
    offsets = torch.tensor([0, M] * ((groups + 2) // 2), device="cuda", dtype=torch.int32)[:groups + 1]
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db = torch.empty(groups, N, device="cuda", dtype=BF)
    kw = dict(z=z, act=act, dx=dx, dw=dw, dbias=db, offsets=offsets)
    n = tgc.tgc_linear_bwd_workspace_bytes(dy, x, w, **kw)
    chunks = (M + 63) // 64
    ws = torch.full((n + 4 * N * chunks * groups,), 0xff, device="cuda", dtype=torch.uint8)
    tgc.tgc_linear_bwd(dy, x, w, workspace=ws, **kw)
    dz = dy.double() * (z > 0) if act == "relu" else dy.double()
    assert torch.equal(dx, (dz @ w1.double()).to(BF))
    full = (dz.t() @ x.double()).to(BF)
    assert bool((dw[0::2] == full).all()) and not dw[1::2].any()
    assert not db.isnan().any() and bool((ws[n:] == 0xff).all())
    whole = [e for e in range(0, groups, 2) if (e // 2 + 1) * chunks <= chunks + groups]
    assert 0 in whole and bool((db[whole] == dz.sum(0).to(BF)).all()) and not db[1::2].any()
    y = torch.empty(M, N, device="cuda", dtype=BF)
    tgc.tgc_linear(x, w, y, offsets=offsets)
    assert torch.equal(y, (x.double() @ w1.double().t()).to(BF))


# ---------------------------------------------------------------- host threads


def test_host_threads_with_rows_of_two_widths():
    """Two threads, each with a width of its own and a stream of its own: every call is accepted."""
    L, rounds, M = _lib.lib(), 4000, 200
    bad, done = [], []

    def work(D, backward):
        y, r, h, dr, dh = (torch.ones(M, D, device="cuda", dtype=BF) for _ in range(5))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        kw = dict(M=M, D=D, post=1, pre=1, eps=1e-5, dtype=3, res_scale=1.0, branch_scale=1.0, stream=s.cuda_stream)
        p = lambda t: t.data_ptr()  # noqa: E731
        if backward:
            a = _lib.BlockNormBwdArgs(y=p(y), r=p(r), dr=p(dr), dh=p(dh), dx=p(h), **kw)
            f = L.tgc_block_norm_bwd
        else:
            a = _lib.BlockNormArgs(y=p(y), r=p(r), h=p(h), **kw)
            f = L.tgc_block_norm
        torch.cuda.synchronize()
        start.wait()
        for i in range(rounds):
            rc = f(ctypes.byref(a))
            if rc != _lib.TGC_OK:
                bad.append((D, backward, rc))
            if i % 200 == 199:
                s.synchronize()
        done.append((y, r, h, dr, dh))

    for backward, widths in ((True, (4104, 8192)), (False, (6400, 8192))):
        start = threading.Barrier(2)
        ts = [threading.Thread(target=work, args=(D, backward)) for D in widths]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
    torch.cuda.synchronize()
    assert len(done) == 4 and not bad, (len(bad), bad[:3])


# ---------------------------------------------------------------- block norm


@pytest.mark.parametrize("D", [64, 777, 1191, 2501, 4096, 8192, 16384])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_without_a_post_norm_dy_does_not_depend_on_y(D, dtype, pre):
    """r = a x + c gate y: dy = c gate t whatever y holds, with and without the gate's gradient."""
    g, M, gates = gen(D), 6, 2
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    y, r, dr, dh, gate = n(M, D), n(M, D), n(M, D), n(M, D) if pre != "none" else None, n(gates, D)
    y[1, 3], y[4, D - 1], y[5, 0] = math.inf, -math.inf, math.nan
    kw = dict(gate=gate, pre=pre, branch_scale=0.5, res_scale=0.75)
    dy, alone, dg, dgf = (torch.full_like(t, 7.0) for t in (y, y, gate, gate))
    tgc.tgc_block_norm_bwd(y, r, dr, dh, dy=dy, dgate=dg, **kw)
    tgc.tgc_block_norm_bwd(None, r, dr, dh, dy=alone, **kw)
    assert bool(alone.isfinite().all())
    assert torch.equal(dy, alone)
    # and the gate's gradient is what it would be without those columns' values
    finite = torch.where(y.isfinite(), y, torch.zeros_like(y))
    tgc.tgc_block_norm_bwd(finite, r, dr, dh, dgate=dgf, **kw)
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[3] = keep[D - 1] = keep[0] = False
    assert torch.equal(dg[:, keep], dgf[:, keep])


# ---------------------------------------------------------------- waits


@pytest.fixture(scope="module")
def short_waits():
    """The library with its limits on waits made so short that a pass outlasts them: a millisecond for the products,
    nothing for the norms' rows."""
    requires_gpu()
    path = _build.build_variant(os.path.join(_build.PKG, "_build", "variant_short_waits"),
                                {"TGC_LINEAR_TIMEOUT_NS": 1000000, "TGC_ROW_TIMEOUT_NS": 0},
                                ["linear_gemm.cu", "linear_split.cu", "block_norm.cu"])
    return _lib.load_library(path)


@pytest.fixture(scope="module")
def one_look():
    """The library with products that give up where the first look at a barrier finds it open."""
    requires_gpu()
    path = _build.build_variant(os.path.join(_build.PKG, "_build", "variant_one_look"), {"TGC_LINEAR_TIMEOUT_NS": 0},
                                ["linear_gemm.cu", "linear_split.cu"])
    return _lib.load_library(path)


def test_a_reduction_may_outlast_the_limit_of_a_wait(short_waits):
    """Reductions of 65536 steps and more of a tile, several milliseconds each: a wait for all of it counts from the
    last step.  Whole numbers, so sums below 2^24 are exact."""
    L, g = short_waits, gen(21)
    ints = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda", dtype=torch.int8).to(BF)  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream

    def status(rc):
        assert rc == _lib.TGC_OK
        return L.tgc_async_status(stream)

    # few tiles: the depth is split over the CTAs of a cluster
    M, K, N = 8, 1 << 25, 8
    x, w = ints(M, K), ints(N, K)
    y = torch.empty(M, N, device="cuda", dtype=BF)
    a = _lib.LinearArgs(x=x.data_ptr(), w=w.data_ptr(), y=y.data_ptr(), M=M, K=K, N=N, dtype=3, stream=stream)
    assert status(L.tgc_linear(ctypes.byref(a))) == _lib.TGC_OK
    assert torch.equal(y, (x.float() @ w.float().t()).to(BF))
    del x, w
    # experts' weight gradients: one CTA or a pair for each tile, rows of another group behind the last step
    for M, K, N in (((1 << 22) + 7, 64, 64), ((1 << 21) + 7, 512, 512)):
        x, dy = ints(M, K), ints(M, N)
        x[M - 9:], dy[M - 9:] = math.nan, math.nan
        off = torch.tensor([0, M - 9], device="cuda", dtype=torch.int32)
        dw = torch.empty(1, N, K, device="cuda", dtype=BF)
        b = _lib.LinearBwdArgs(dy=dy.data_ptr(), x=x.data_ptr(), dw=dw.data_ptr(), M=M, K=K, N=N, dtype=3,
                               offsets=off.data_ptr(), ngroups=1, stream=stream)
        assert status(L.tgc_linear_bwd(ctypes.byref(b))) == _lib.TGC_OK
        assert torch.equal(dw[0], (dy[:M - 9].float().t() @ x[:M - 9].float()).to(BF))


@pytest.mark.parametrize("D", [256, 4096, 8192])
@pytest.mark.parametrize("full", [False, True])
def test_norms_whose_wait_expires_end_and_say_so(short_waits, D, full):
    """Rows that have not landed at the first look: the kernels go on without them, let them land, end and mark
    the fault; every later call is right."""
    g, M = gen(D), 20000
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    y, x, r, h, dr, dh, dx, dy = (n(M, D) for _ in range(8))
    dw, db = (torch.empty(D, device="cuda", dtype=BF) for _ in range(2))
    ws = torch.empty(1 << 25, device="cuda", dtype=torch.uint8)
    stream = torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()  # noqa: E731
    kw = dict(M=M, D=D, post=2 if full else 1, pre=1, eps=1e-5, dtype=3, res_scale=1.0, branch_scale=1.0, stream=stream)
    fwd = dict(y=p(y), x=p(x), pre_bias=p(db) if full else None)
    bwd = dict(y=p(y), r=p(r), dr=p(dr), dh=p(dh), workspace=p(ws), workspace_bytes=ws.numel(), dpre_weight=p(dw),
               dpre_bias=p(db) if full else None)
    db.zero_()
    seen = []
    for _ in range(3):
        rc = short_waits.tgc_block_norm(ctypes.byref(_lib.BlockNormArgs(r=p(dx), h=p(dy), **fwd, **kw)))
        assert rc == _lib.TGC_OK
        seen.append(short_waits.tgc_async_status(stream))
        rc = short_waits.tgc_block_norm_bwd(ctypes.byref(_lib.BlockNormBwdArgs(dx=p(dx), dy=p(dy), **bwd, **kw)))
        assert rc == _lib.TGC_OK
        seen.append(short_waits.tgc_async_status(stream))
    assert set(seen) <= {_lib.TGC_OK, _lib.TGC_ERR_TIMEOUT}
    assert D < 4096 or seen[0] == seen[1] == _lib.TGC_ERR_TIMEOUT
    tgc.tgc_block_norm(y, dx, dy, x=x, post="layer" if full else "rms", pre="rms", pre_bias=db if full else None)
    tgc.tgc_async_status()
    v = y.float() - (y.float().mean(1, keepdim=True) if full else 0)
    want = x.float() + v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-5)
    assert bool(((dx.float() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all())


@pytest.mark.parametrize("M,K,N,groups", [(4, 4096, 1024, 0), (2048, 2048, 2048, 0), (2048, 1024, 1024, 3), (300, 512, 264, 0)])
def test_products_whose_wait_expires_end_and_say_so(one_look, M, K, N, groups):
    """Loads that have not landed at the first look: the kernels give up, let them land, end and mark the
    fault; every later call is right."""
    L, g = one_look, gen(M + N)
    ints = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda", dtype=torch.int8).to(BF)  # noqa: E731
    lead = (groups,) if groups else ()
    x, w, dy = ints(M, K), ints(*lead, N, K), ints(M, N)
    off = torch.tensor([0, M // 3 + 5, M // 3 + 5, M - 7], device="cuda", dtype=torch.int32) if groups else None
    y, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(w)
    stream = torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
    kw = dict(M=M, K=K, N=N, dtype=3, offsets=p(off), ngroups=groups, stream=stream)
    assert L.tgc_linear(ctypes.byref(_lib.LinearArgs(x=p(x), w=p(w), y=p(y), **kw))) == _lib.TGC_OK
    assert L.tgc_async_status(stream) == _lib.TGC_ERR_TIMEOUT
    for out in (dict(dx=p(dx)), dict(dw=p(dw)), dict(dx=p(dx), dw=p(dw))):
        a = _lib.LinearBwdArgs(dy=p(dy), x=p(x), w=p(w), **out, **kw)
        assert L.tgc_linear_bwd(ctypes.byref(a)) == _lib.TGC_OK
        assert L.tgc_async_status(stream) == _lib.TGC_ERR_TIMEOUT
    assert L.tgc_async_status(stream) == _lib.TGC_OK  # read, and cleared
    tgc.tgc_linear(x, w, y, offsets=off)
    tgc.tgc_linear_bwd(dy, x, w, dx=dx, dw=dw, offsets=off)
    tgc.tgc_async_status()
    spans = list(zip(off.tolist(), off.tolist()[1:])) if groups else [(0, M)]
    for e, (i, j) in enumerate(spans):
        we, dwe = (w[e], dw[e]) if groups else (w, dw)
        assert torch.equal(y[i:j], (x[i:j].float() @ we.float().t()).to(BF))
        assert torch.equal(dx[i:j], (dy[i:j].float() @ we.float()).to(BF))
        assert torch.equal(dwe, (dy[i:j].float().t() @ x[i:j].float()).to(BF))


# ---------------------------------------------------------------- activations

FAR = [50.0, 1e3, 1e9, 1e15, 1e19, 2e19, 1e20, 1e30, 3e38]


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [4, 300])
def test_activations_far_from_zero(act, M):
    """|z| >= 50: act(z) is z, or next to nothing, and its derivative 1, or next to nothing."""
    K = 8
    values = torch.tensor([v * s for v in FAR for s in (1, -1)], device="cuda")
    N = (len(values) + 7) // 8 * 8
    values = torch.cat([values, torch.full((N - len(values),), 60.0, device="cuda")]).to(BF)
    v64 = values.double()
    gate = torch.sigmoid(v64) if act == "silu" else (v64 > 0).double()
    want, slope = v64 * gate, gate * (1 + v64 * (1 - gate)) if act == "silu" else gate
    x, w = torch.zeros(M, K, device="cuda", dtype=BF), torch.zeros(N, K, device="cuda", dtype=BF)
    x[:, 0], w[:, 0] = 1.0, values
    y, z = (torch.empty(M, N, device="cuda", dtype=BF) for _ in range(2))
    tgc.tgc_linear(x, w, y, act=act, z=z)
    assert torch.equal(z, values.expand(M, N))
    assert bool(((y.double() - want).abs() <= U[BF] * want.abs()).all())
    dy, db = torch.ones(M, N, device="cuda", dtype=BF), torch.empty(N, device="cuda", dtype=BF)
    tgc.tgc_linear_bwd(dy, x, w, z=z, act=act, dbias=db)
    assert bool(((db.double() - M * slope).abs() <= U[BF] * M * slope.abs()).all())


@pytest.mark.parametrize("dtype", [BF, F16])
def test_gelu_of_negative_values(dtype):
    """Phi(z) is off by 2^-21 at most: 0.75e-7 by its formula; half of 2^-22 by the exponential, as Phi <= 1/2
    here; 2^-22 times a slope below 0.6 by the reciprocal; five roundings of values below 0.75 by the polynomial."""
    z = torch.linspace(-12, 0, 4096, device="cuda").to(dtype)
    M, K, N = 8, 8, len(z)
    x, w = torch.zeros(M, K, device="cuda", dtype=dtype), torch.zeros(N, K, device="cuda", dtype=dtype)
    x[:, 0], w[:, 0] = 1.0, z
    y = torch.empty(M, N, device="cuda", dtype=dtype)
    tgc.tgc_linear(x, w, y, act="gelu")
    z64 = z.double()
    ref = z64 * 0.5 * torch.special.erfc(-z64 / math.sqrt(2))
    err = (y.double() - ref).abs()
    assert bool((err <= U[dtype] * ref.abs() + 2.0 ** -21 * z64.abs() + (2.0 ** -24 if dtype == F16 else 0)).all())
