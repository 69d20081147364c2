"""tgc_block_norm and tgc_block_norm_bwd on the GPU against the formulas in 64 bits.

Tolerance, from the roundings: u |result| for the output's type (one unit in the last place: 2^-8
bf16, 2^-10 f16, 2^-23 f32) and 1e-5 of the largest magnitude that a row's (for sums over rows: a
column's) terms reach -- a fp32 value goes through fewer than 80 roundings of 2^-23 there."""
import math

import pytest
import torch

import tile_gather_comm_gb300 as tgc
from tests.helpers import requires_gpu

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF: 2.0 ** -8, F16: 2.0 ** -10, F32: 2.0 ** -23}
EPS = 1e-5
A, C = 0.75, 0.5  # residual and branch scale


@pytest.fixture(autouse=True)
def _gpu():
    requires_gpu()


def norm64(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    v = v * w if w is not None else v
    return v + b if b is not None else v


def forward64(d, post, pre):
    u = norm64(d["y"], post, d["post_w"], d["post_b"])
    if d["gate"] is not None:
        u = u * d["gate"].repeat_interleave(u.shape[0] // d["gate"].shape[0], 0)
    r = C * u + (A * d["x"] if d["x"] is not None else 0)
    return r, norm64(r, pre, d["pre_w"], d["pre_b"])


def inputs(M, D, dtype, post, pre, gates, weights=True, biases=True, residual=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + M + D)
    n = lambda *s, k=1.0, m=0.0: (torch.randn(*s, generator=g, device="cuda") * k + m).to(dtype)
    return {"y": n(M, D, m=0.3), "x": n(M, D) if residual else None, "gate": n(gates, D) if gates else None,
            "post_w": n(D, k=0.3, m=1) if weights and post != "none" else None,
            "post_b": n(D) if biases and post != "none" else None,
            "pre_w": n(D, k=0.3, m=1) if weights and pre != "none" else None,
            "pre_b": n(D) if biases and pre != "none" else None, "dr": n(M, D), "dh": n(M, D), "kept": n(M, D, m=-0.2)}


def run(s, post, pre, r, h, **kw):
    tgc.tgc_block_norm(s["y"], r, h, x=s["x"], gate=s["gate"], post=post, post_weight=s["post_w"], post_bias=s["post_b"],
                       pre=pre, pre_weight=s["pre_w"], pre_bias=s["pre_b"], res_scale=A, branch_scale=C, eps=EPS, **kw)


def close(got, ref, mag, dtype):
    """mag: the magnitude the fp32 roundings act on, broadcastable to ref."""
    err = (got.double() - ref).abs() - U[dtype] * ref.abs() - 1e-5 * mag - (2.0 ** -24 if dtype == F16 else 0)
    return float(err.max()) <= 0


# widths: one element, no vector divides it, one warp, its edges, a block, several vectors a thread
WIDTHS = [1, 7, 32, 64, 255, 256, 257, 777, 1000, 1024, 2056, 4096, 5000, 8192, 12296, 16383, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("post,pre,gates,M", [("rms", "rms", 3, 12), ("layer", "layer", 1, 5), ("none", "rms", 0, 9),
                                              ("rms", "none", 7, 7)])
def test_forward(D, dtype, post, pre, gates, M):
    s = inputs(M, D, dtype, post, pre, gates)
    r = torch.full((M, D), float("nan"), device="cuda", dtype=dtype)
    h = torch.full_like(r, float("nan")) if pre != "none" else None
    run(s, post, pre, r, h)
    d = {k: v.double() if v is not None else None for k, v in s.items()}
    r64, h64 = forward64(d, post, pre)
    top = r64.abs().amax(1, keepdim=True) + d["x"].abs().amax(1, keepdim=True)
    assert close(r, r64, top, dtype)
    if h is not None:
        # a row of nearly equal values: the norm enlarges r's own roundings by 1 / its deviation
        v = r64 - r64.mean(1, keepdim=True) if pre == "layer" else r64
        grow = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
        w = s["pre_w"].double().abs().amax() if s["pre_w"] is not None else 1
        assert close(h, h64, h64.abs().amax(1, keepdim=True) + grow * top * w, dtype)


GRADS = ["dx", "dy", "dgate", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"]


def backward64(d, post, pre, M, gates):
    """By autograd: pre's at the kept r, the rest through the forward formula."""
    names = [k for k in ("x", "y", "gate", "post_w", "post_b") if d[k] is not None]
    leaf = {k: d[k].clone().requires_grad_() for k in names + ["pre_w", "pre_b", "kept"] if d[k] is not None}
    full = {**d, **leaf}
    t, out = d["dr"], {}
    if pre != "none":
        hs = [k for k in ("kept", "pre_w", "pre_b") if k in leaf]
        got = torch.autograd.grad(norm64(full["kept"], pre, full["pre_w"], full["pre_b"]), [leaf[k] for k in hs], d["dh"])
        out.update(zip(hs, got))
        t = t + out.pop("kept")
    out.update(zip(names, torch.autograd.grad(forward64({**full, "pre_w": None, "pre_b": None}, post, "none")[0],
                                              [leaf[k] for k in names], t)))
    rename = {"post_w": "dpost_weight", "post_b": "dpost_bias", "pre_w": "dpre_weight", "pre_b": "dpre_bias"}
    return {rename.get(k, "d" + k): v for k, v in out.items()}, t


def run_bwd(s, post, pre, outs, **kw):
    tgc.tgc_block_norm_bwd(s["y"], s["kept"], s["dr"], s["dh"] if pre != "none" else None, gate=s["gate"], post=post,
                           post_weight=s["post_w"], post_bias=s["post_b"], pre=pre, pre_weight=s["pre_w"], res_scale=A,
                           branch_scale=C, eps=EPS, **outs, **kw)


@pytest.mark.parametrize("D", [8, 31, 64, 256, 264, 777, 1024, 2056, 4096, 5000, 8192, 16383, 16384])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("post,pre,gates,M,biases", [("rms", "rms", 2, 38, False), ("layer", "layer", 1, 29, True),
                                                     ("none", "rms", 5, 5, False), ("layer", "none", 0, 3, True),
                                                     ("rms", "layer", 400, 800, False)])
def test_backward(D, dtype, post, pre, gates, M, biases):
    if M * D > 1 << 22:
        M, gates = M // 100, max(1, gates // 100)
    s = inputs(M, D, dtype, post, pre, gates, biases=biases)
    d = {k: v.double() if v is not None else None for k, v in s.items()}
    ref, t = backward64(d, post, pre, M, gates)
    outs = {k: torch.full(v.shape, float("nan"), device="cuda", dtype=dtype) for k, v in ref.items()}
    run_bwd(s, post, pre, outs)

    def rstd(v, kind):
        if kind == "none":
            return torch.ones_like(v[:, :1])
        v = v - v.mean(1, keepdim=True) if kind == "layer" else v
        return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)

    big = lambda k: d[k].abs().amax() if d[k] is not None else 1.0
    # what the roundings of a row act on: the terms before they cancel
    grow = rstd(d["kept"], pre) if pre != "none" else 0
    mt = d["dr"].abs().amax(1, keepdim=True) + (3 * grow * big("dh") * big("pre_w") if pre != "none" else 0)
    mu = C * mt * big("gate")
    my = 3 * rstd(d["y"], post) * mu * (big("post_w") if post != "none" else 1)
    hat = lambda v, k: norm64(v, k, None, None).abs().amax(1, keepdim=True) + (rstd(v, k) * v.abs().amax(1, keepdim=True)
                                                                             if k != "none" else 0)
    yh, rh = hat(d["y"], post), hat(d["kept"], pre)
    bounds = {"dx": mt, "dy": my, "dgate": None, "dpost_weight": (mu * yh).sum(), "dpost_bias": mu.sum(),
              "dpre_weight": (big("dh") * rh).sum(), "dpre_bias": big("dh") * M}
    if gates:
        u = yh * big("post_w") + big("post_b") if post != "none" else d["y"].abs().amax(1, keepdim=True)
        bounds["dgate"] = (C * mt * u).view(gates, -1).sum(1, keepdim=True)
    for k, v in ref.items():
        assert close(outs[k], v, bounds[k], dtype), (k, float((outs[k].double() - v).abs().max()))


@pytest.mark.parametrize("D", [513, 2047, 2049, 2501, 4095, 4097, 8191, 8193])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("post,pre,gates,M,biases", [("rms", "rms", 2, 38, False), ("layer", "layer", 1, 29, True),
                                                     ("none", "rms", 5, 5, False), ("layer", "none", 0, 3, True),
                                                     ("rms", "layer", 4, 400, False)])
def test_odd_widths_of_every_length(D, dtype, post, pre, gates, M, biases):
    """Single elements, 4 to 32 a thread, on both sides of each step."""
    test_forward(D, dtype, post, pre, gates, M)
    test_backward(D, dtype, post, pre, gates, M, biases)


@pytest.mark.parametrize("M,gates", [(1, 1), (1, 0), (4096, 4096), (4096, 2), (4099, 1), (4099, 4099), (3000, 600)])
@pytest.mark.parametrize("dtype,D", [(BF, 256), (F32, 33), (BF, 1024)])
def test_backward_over_many_rows(M, gates, dtype, D):
    """Every way the rows are dealt: single rows, whole gate segments, segments cut into units."""
    post, pre = "rms", "rms"
    s = inputs(M, D, dtype, post, pre, gates, biases=False)
    d = {k: v.double() if v is not None else None for k, v in s.items()}
    ref, t = backward64(d, post, pre, M, gates)
    outs = {k: torch.full(v.shape, float("nan"), device="cuda", dtype=dtype) for k, v in ref.items()}
    run_bwd(s, post, pre, outs)
    again = {k: torch.empty_like(v) for k, v in outs.items()}
    run_bwd(s, post, pre, again)
    for k, v in ref.items():
        n = M // max(gates, 1) if k == "dgate" else M if v.dim() == 1 else 1
        mag = (40 * n if k == "dgate" or v.dim() == 1 else 20) * t.abs().amax()
        assert close(outs[k], v, mag, dtype), k
        assert torch.equal(outs[k], again[k])


@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms")])
def test_gradients_against_differences(post, pre):
    """Central differences of the 64-bit formula along random directions, against the kernels' f32 gradients."""
    M, D, gates = 6, 48, 3
    s = inputs(M, D, F32, post, pre, gates)
    d = {k: v.double() for k, v in s.items()}
    r64 = forward64(d, post, pre)[0]
    s["kept"] = r64.float()
    names = {"x": "dx", "y": "dy", "gate": "dgate", "post_w": "dpost_weight", "post_b": "dpost_bias",
             "pre_w": "dpre_weight", "pre_b": "dpre_bias"}
    outs = {n: torch.empty_like(s[k]) for k, n in names.items()}
    run_bwd(s, post, pre, outs)
    g = torch.Generator(device="cuda").manual_seed(4)
    for k, n in names.items():
        p = torch.randn(d[k].shape, generator=g, device="cuda", dtype=torch.float64)
        loss = []
        for h in (1e-6, -1e-6):
            r, hh = forward64({**d, k: d[k] + h * p}, post, pre)
            loss.append((r * d["dr"]).sum() + (hh * d["dh"]).sum())
        diff = float((loss[0] - loss[1]) / 2e-6)
        scale = float((outs[n].double() * p).abs().sum())
        assert abs(diff - float((outs[n].double() * p).sum())) <= 1e-5 * scale + 1e-6


@pytest.mark.parametrize("D,off", [(256, 0), (256, 1), (777, 0), (4096, 3)])
def test_strides_alignment_and_in_place(D, off):
    """Rows with a stride and a start that no vector fits, NaN around them; outputs over inputs."""
    M, dtype = 10, BF
    s = inputs(M, D, dtype, "rms", "rms", 2, biases=False)

    def wide(t):
        buf = torch.full((M, D + 16 + off), float("nan"), device="cuda", dtype=dtype)
        buf[:, off:off + D] = t
        return buf[:, off:off + D], buf

    # in place against out of place on the same layout (another alignment may sum in another order)
    q = dict(s)
    q["y"], ybuf = wide(s["y"])
    q["x"], xbuf = wide(s["x"])
    r, rbuf = wide(s["x"])
    h, hbuf = wide(s["x"])
    run(q, "rms", "rms", r, h)
    d = {k: v.double() if v is not None else None for k, v in s.items()}
    r64, h64 = forward64(d, "rms", "rms")
    assert close(r, r64, r64.abs().amax(), dtype) and close(h, h64, h64.abs().amax(), dtype)
    run(q, "rms", "rms", q["x"], q["y"])  # r over x, h over y
    assert torch.equal(q["x"], r) and torch.equal(q["y"], h)
    for buf in (ybuf, xbuf, rbuf, hbuf):
        assert bool(buf[:, off + D:].isnan().all()) and bool(buf[:, :off].isnan().all())
    q = dict(s)
    q["dr"], _ = wide(s["dr"])
    q["dh"], _ = wide(s["dh"])
    q["kept"], _ = wide(s["kept"])
    ref = {"dx": wide(s["x"])[0], "dy": wide(s["x"])[0]}
    run_bwd(q, "rms", "rms", ref)
    run_bwd(q, "rms", "rms", {"dx": q["dr"], "dy": q["dh"]})
    assert torch.equal(q["dr"], ref["dx"]) and torch.equal(q["dh"], ref["dy"])


def test_special_rows_large_strides_and_empty():
    s = inputs(6, 512, F32, "layer", "layer", 0)
    s["y"][1] = 3.25            # no deviation: the norm is its bias
    s["y"][2], s["y"][3, 5] = 0.0, float("nan")
    s["y"][4] *= 1e15           # squares near the top of fp32
    r, h = torch.empty_like(s["y"]), torch.empty_like(s["y"])
    run(s, "layer", "layer", r, h)
    d = {k: v.double() if v is not None else None for k, v in s.items()}
    r64, h64 = forward64(d, "layer", "layer")
    good = [0, 1, 2, 4, 5]
    assert close(r[good], r64[good], 10.0, F32) and close(h[good], h64[good], 10.0, F32)
    assert bool(r[3].isnan().all()) and bool(h[3].isnan().all())
    # rows more than 2^31 elements apart
    ld = (1 << 30) + 8
    buf = torch.empty(2 * ld + 512, device="cuda", dtype=BF)
    y = buf.as_strided((3, 512), (ld, 1))
    y.copy_(s["x"][:3])
    out = torch.empty(3, 512, device="cuda", dtype=BF)
    tgc.tgc_block_norm(y, None, out, pre="rms")
    ref = norm64(y.double(), "rms", None, None)
    assert close(out, ref, ref.abs().amax(), BF)
    # no rows: parameter gradients are zeros
    dw, dg = torch.ones(8, device="cuda"), torch.ones(2, 8, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    tgc.tgc_block_norm(e, e, e, pre="rms")
    tgc.tgc_block_norm_bwd(e, e, e, e, gate=torch.ones(2, 8, device="cuda"), dgate=dg, dpre_weight=dw)
    assert not dw.any() and not dg.any()


def test_partial_outputs_and_the_plain_norm():
    s = inputs(40, 256, BF, "rms", "rms", 2, biases=False)
    full = {k: None for k in ("dx", "dy")}
    full = {"dx": torch.empty_like(s["y"]), "dy": torch.empty_like(s["y"]), "dgate": torch.empty_like(s["gate"]),
            "dpost_weight": torch.empty_like(s["post_w"]), "dpre_weight": torch.empty_like(s["pre_w"])}
    run_bwd(s, "rms", "rms", full)
    for k, v in full.items():
        one = {k: torch.full_like(v, float("nan"))}
        run_bwd(s, "rms", "rms", one)
        assert torch.equal(one[k], v), k
    h, h2 = torch.empty_like(s["y"]), torch.empty_like(s["y"])
    tgc.tgc_block_norm(s["y"], None, h, pre="rms", pre_weight=s["pre_w"])
    tgc.tgc_block_norm(s["y"], h2, None, post="rms", post_weight=s["pre_w"], pre="none")
    assert torch.equal(h, h2)


def test_side_stream_and_graph():
    s = inputs(500, 1024, BF, "rms", "rms", 4, biases=False)
    outs = lambda: {"dx": torch.empty_like(s["y"]), "dgate": torch.empty_like(s["gate"]),
                    "dpre_weight": torch.empty_like(s["pre_w"])}
    first, other, graphed = outs(), outs(), outs()
    run_bwd(s, "rms", "rms", first)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    run_bwd(s, "rms", "rms", other, stream=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_bwd(s, "rms", "rms", graphed)
    graph.replay()
    torch.cuda.synchronize()
    for k in first:
        assert torch.equal(first[k], other[k]) and torch.equal(first[k], graphed[k])


@pytest.mark.parametrize("M,D", [(1, 64), (300, 64), (300, 777)])
def test_a_workspace_of_the_queried_size_serves_and_a_smaller_one_is_refused(M, D):
    gen = torch.Generator(device="cuda").manual_seed(5)
    y, r, dh = (torch.randn(M, D, device="cuda", generator=gen) for _ in range(3))
    w = torch.ones(D, device="cuda")
    out = lambda: dict(dy=torch.empty_like(y), dpre_weight=torch.empty_like(w))
    kw, one, own = dict(pre="rms", pre_weight=w), out(), out()
    n = tgc.tgc_block_norm_bwd_workspace_bytes(y, r, None, dh, **kw, **one)
    assert n > 0
    tgc.tgc_block_norm_bwd(y, r, None, dh, **kw, **one)
    tgc.tgc_block_norm_bwd(y, r, None, dh, **kw, **own, workspace=torch.empty(n, device="cuda", dtype=torch.uint8))
    assert all(torch.equal(one[k], own[k]) for k in one)
    with pytest.raises(tgc.TGCError):
        tgc.tgc_block_norm_bwd(y, r, None, dh, **kw, **own,
                               workspace=torch.empty(n - 1, device="cuda", dtype=torch.uint8))
