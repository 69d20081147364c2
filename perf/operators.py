"""The work the transformer-block operators are measured on.

Three operators around the library's matrix product:
  linear      y = act(x w^T + b) + residual, and its gradients
  grouped     the same product for experts: rows sorted by expert, a weight each, ragged sizes
  block norm  r = a x + c g * post(y), h = pre(r): the norms before and after a block with its
              gate and residual scale, and their gradients

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU from a seed, ``run`` makes one
pass (in plain 32-bit torch operations, or through the library where ``own`` is true), ``exact``
computes the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------------------ cases


def _linear(op, M, K, N, dtype, act, bias=True, residual=False, keep_z=False):
    return {"op": op, "M": M, "K": K, "N": N, "dtype": dtype, "act": act, "bias": bias, "residual": residual,
            "keep_z": keep_z}


def _grouped(op, rows, experts, K, N, dtype, act, mix, bias=True, keep_z=False):
    return {"op": op, "M": rows, "E": experts, "K": K, "N": N, "dtype": dtype, "act": act, "mix": mix, "bias": bias,
            "keep_z": keep_z}


def _norm(op, M, D, dtype, post, pre, gates, affine_bias, residual=True):
    return {"op": op, "M": M, "D": D, "dtype": dtype, "post": post, "pre": pre, "gates": gates,
            "affine_bias": affine_bias, "residual": residual}


def listed():
    return [
        # one new token through the up projection of the MLP: the weight is read once for a single row
        {"name": "linear token", **_linear("linear", 1, 4096, 14336, "bf16", "gelu_tanh")},
        # a batch of 48 running sequences through the down projection, added to the residual stream
        {"name": "linear batch 48", **_linear("linear", 48, 14336, 4096, "f16", "none", residual=True)},
        # a short prompt, no size a multiple of a tile
        {"name": "linear prompt 777", **_linear("linear", 777, 4104, 5000, "bf16", "silu", residual=True)},
        # the up projection of a training step: the pre-activation is kept for the backward pass
        {"name": "linear train", **_linear("linear", 8192, 4096, 14336, "bf16", "gelu", keep_z=True)},
        # and its gradients: input, weight and bias
        {"name": "linear train backward", **_linear("linear_bwd", 8192, 4096, 14336, "bf16", "gelu")},
        # one decoding step of 24 sequences, two experts each out of 16: most of the weights for few rows
        {"name": "experts batch 24x2", **_grouped("grouped", 48, 16, 4096, 14336, "bf16", "silu", 1, bias=False)},
        # a training batch over 16 experts, unevenly loaded
        {"name": "experts train", **_grouped("grouped", 16384, 16, 4096, 4096, "bf16", "gelu_tanh", 2, keep_z=True)},
        # gradients over 8 experts, odd row counts and an expert that no row chose
        {"name": "experts train backward", **_grouped("grouped_bwd", 8191, 8, 4096, 4096, "f16", "silu", 3)},
        # a decoding step's block boundary: four tokens, where the call itself is what costs
        {"name": "norm tokens 4", **_norm("norm", 4, 4096, "bf16", "rms", "rms", 1, False)},
        # the boundary between two blocks for a long prompt: eight sequences, a gate vector for each
        {"name": "norm prompt", **_norm("norm", 8192, 4096, "bf16", "rms", "rms", 8, False)},
        # and its gradients in training
        {"name": "norm train backward", **_norm("norm_bwd", 8192, 4096, "bf16", "rms", "rms", 8, False)},
        # mean-and-variance norms with biases in 32 bits, an odd width that no vector divides, one gate for all rows
        {"name": "norm odd backward", **_norm("norm_bwd", 1000, 777, "f32", "layer", "layer", 1, True)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    return max(lo, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "grouped", "grouped_bwd", "norm", "norm_bwd"])
    if op.startswith("norm"):
        M, D = _log(rng, 1, 8192), _log(rng, 16, 8192)  # narrower rows leave a norm nothing but rounding
        while M * D > 8192 * 4096:
            M = (M + 1) // 2
        divisors = [g for g in range(1, M + 1) if M % g == 0]
        return _norm(op, M, D, rng.choice(["bf16", "f16", "f32"]), rng.choice(["none", "rms", "layer"]),
                     rng.choice(["rms", "layer"]), rng.choice([0, 1, M, rng.choice(divisors)]), rng.random() < 0.5,
                     residual=rng.random() < 0.8)
    dtype = rng.choice(["bf16", "f16"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    K, N = _eights(rng, 64, 14336), _eights(rng, 64, 14336)
    if op.startswith("linear"):
        M = _log(rng, 1, 8192)
        while M * K * N > 8192 * 4096 * 14336:
            K = max(64, K // 2 // 8 * 8)
        fwd = op == "linear"
        return _linear(op, M, K, N, dtype, act, rng.random() < 0.7, fwd and rng.random() < 0.5,
                       fwd and rng.random() < 0.3)
    E, M = _log(rng, 1, 64), _log(rng, 1, 16384)
    while E * K * N > 16 * 4096 * 14336 or M * K * N > 16384 * 4096 * 4096:
        K, N = max(64, K // 2 // 8 * 8), max(64, N // 2 // 8 * 8)
    return _grouped(op, M, E, K, N, dtype, act, rng.randrange(1, 1000), rng.random() < 0.5,
                    op == "grouped" and rng.random() < 0.3)


def _group_sizes(case):
    """Rows of each expert: uneven shares, some of them empty, drawn from the case alone."""
    rng = random.Random(case["mix"])
    E, M = case["E"], case["M"]
    share = [0.0 if E > 3 and rng.random() < 0.1 else rng.gammavariate(1.5, 1.0) + 1e-3 for _ in range(E)]
    if not any(share):
        share[0] = 1.0
    total, sizes, done, acc = sum(share), [], 0, 0.0
    for s in share:
        acc += s
        upto = int(round(M * acc / total))
        sizes.append(upto - done)
        done = upto
    sizes[-1] += M - sum(sizes)
    return sizes


# ------------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(sigma).add_(mean).to(dt)

    s = {"case": case}
    if case["op"].startswith("norm"):
        M, D, G = case["M"], case["D"], case["gates"]
        s["y"] = normal(M, D, sigma=0.7, mean=0.1)
        s["x"] = normal(M, D, sigma=2.0) if case["residual"] else None
        s["gate"] = normal(G, D, sigma=0.5, mean=0.3) if G else None
        for which in ("post", "pre"):
            s[which + "_w"] = normal(D, sigma=0.2, mean=1.0) if case[which] != "none" else None
            s[which + "_b"] = normal(D, sigma=0.2) if case[which] == "layer" and case["affine_bias"] else None
        s["res_scale"], s["branch_scale"] = 0.9, 0.5
        s["r"] = torch.empty(M, D, device="cuda", dtype=dt)
        if case["op"] == "norm":
            s["h"] = torch.empty(M, D, device="cuda", dtype=dt)
        else:
            s["r"] = normal(M, D, sigma=2.0, mean=0.05)  # the residual stream that the forward pass kept
            s["dr"], s["dh"] = normal(M, D), normal(M, D)
            s["dx"] = torch.empty_like(s["y"]) if case["residual"] else None
            s["dy"] = torch.empty_like(s["y"])
            s["dgate"] = torch.empty_like(s["gate"]) if G else None
            for k in ("post_w", "post_b", "pre_w", "pre_b"):
                s["d" + k] = torch.empty_like(s[k]) if s[k] is not None else None
        return s
    M, K, N = case["M"], case["K"], case["N"]
    lead = (case["E"],) if "E" in case else ()
    s["x"] = normal(M, K)
    s["w"] = normal(*lead, N, K, sigma=0.02)
    s["b"] = normal(*lead, N, sigma=0.1) if case["bias"] else None
    s["sizes"] = _group_sizes(case) if lead else [M]
    if lead:
        edges = [0]
        for n in s["sizes"]:
            edges.append(edges[-1] + n)
        s["offsets"] = torch.tensor(edges, dtype=torch.int32, device="cuda")
    if case["op"].endswith("_bwd"):
        s["dy"] = normal(M, N, sigma=0.1)
        s["z"] = normal(M, N, sigma=0.02 * math.sqrt(K)) if case["act"] != "none" else None
        s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
        s["db"] = torch.empty_like(s["b"]) if case["bias"] else None
    else:
        s["res"] = normal(M, N) if case.get("residual") else None
        s["y"] = torch.empty(M, N, device="cuda", dtype=dt)
        s["z"] = torch.empty(M, N, device="cuda", dtype=dt) if case["keep_z"] else None
    return s


# ------------------------------------------------------------------------------------------ one pass


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _plain_linear(s, case):
    x, w = s["x"].float(), s["w"].float()
    b = s["b"].float() if s["b"] is not None else None
    if "E" in case:
        parts = zip(x.split(s["sizes"]), w, b if b is not None else [0.0] * len(w))
        z = torch.cat([xe @ we.t() + be for xe, we, be in parts])
    else:
        z = x @ w.t()
        z = z + b if b is not None else z
    y = _act(z, case["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(s["x"].dtype)}
    if case["keep_z"]:
        out["z"] = z.to(s["x"].dtype)
    return out


def _plain_linear_bwd(s, case):
    dt = s["x"].dtype
    x, w, dz = s["x"].float(), s["w"].float(), s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(s["z"].float(), case["act"])
    if "E" in case:
        dzs, xs = dz.split(s["sizes"]), x.split(s["sizes"])
        dx = torch.cat([de @ we for de, we in zip(dzs, w)])
        dw = torch.stack([de.t() @ xe for de, xe in zip(dzs, xs)])
        db = torch.stack([de.sum(0) for de in dzs])
    else:
        dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    out = {"dx": dx.to(dt), "dw": dw.to(dt)}
    if s["db"] is not None:
        out["db"] = db.to(dt)
    return out


def _plain_hat(v, kind):
    """Normalised rows and the reciprocal deviations."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * rstd, rstd


def _plain_norm(s, kind, which, v):
    if kind == "none":
        return v
    out = _plain_hat(v, kind)[0] * s[which + "_w"].float()
    return out + s[which + "_b"].float() if s[which + "_b"] is not None else out


def _plain_norm_grad(s, kind, which, v, d):
    """The gradient of a norm's input, weight and bias."""
    hat, rstd = _plain_hat(v, kind)
    q = d * s[which + "_w"].float()
    dv = q - hat * (q * hat).mean(1, keepdim=True)
    if kind == "layer":
        dv = dv - q.mean(1, keepdim=True)
    return rstd * dv, (d * hat).sum(0), d.sum(0)


def _spread(gate, M):
    return gate.float().repeat_interleave(M // gate.shape[0], 0)


def _plain_block_norm(s, case):
    dt = s["y"].dtype
    r = s["branch_scale"] * _plain_norm(s, case["post"], "post", s["y"].float())
    if s["gate"] is not None:
        r = r * _spread(s["gate"], case["M"])
    if s["x"] is not None:
        r = r + s["res_scale"] * s["x"].float()
    return {"r": r.to(dt), "h": _plain_norm(s, case["pre"], "pre", r).to(dt)}


def _plain_block_norm_bwd(s, case):
    dt, out = s["y"].dtype, {}
    dv, dw, db = _plain_norm_grad(s, case["pre"], "pre", s["r"].float(), s["dh"].float())
    out["dpre_w"], out["dpre_b"] = dw, db
    t = s["dr"].float() + dv
    if s["x"] is not None:
        out["dx"] = s["res_scale"] * t
    du = s["branch_scale"] * t
    if s["gate"] is not None:
        u = _plain_norm(s, case["post"], "post", s["y"].float())
        out["dgate"] = (du * u).reshape(case["gates"], -1, case["D"]).sum(1)
        du = du * _spread(s["gate"], case["M"])
    if case["post"] == "none":
        out["dy"] = du
    else:
        out["dy"], out["dpost_w"], out["dpost_b"] = _plain_norm_grad(s, case["post"], "post", s["y"].float(), du)
    return {k: v.to(dt) for k, v in out.items() if s[k] is not None}


def _own_pass(s, case):
    import tile_gather_comm_gb300 as tgc
    op = case["op"]
    if op == "linear":
        tgc.tgc_linear(s["x"], s["w"], s["y"], bias=s["b"], act=case["act"], residual=s["res"], z=s["z"])
    elif op == "grouped":
        tgc.tgc_linear(s["x"], s["w"], s["y"], bias=s["b"], act=case["act"], z=s["z"], offsets=s["offsets"])
    elif op == "linear_bwd":
        tgc.tgc_linear_bwd(s["dy"], s["x"], s["w"], z=s["z"], act=case["act"], dx=s["dx"], dw=s["dw"], dbias=s["db"])
    elif op == "grouped_bwd":
        tgc.tgc_linear_bwd(s["dy"], s["x"], s["w"], z=s["z"], act=case["act"], dx=s["dx"], dw=s["dw"], dbias=s["db"],
                           offsets=s["offsets"])
    elif op == "norm":
        tgc.tgc_block_norm(s["y"], s["r"], s["h"], x=s["x"], gate=s["gate"], post=case["post"],
                           post_weight=s["post_w"], post_bias=s["post_b"], pre=case["pre"], pre_weight=s["pre_w"],
                           pre_bias=s["pre_b"], res_scale=s["res_scale"], branch_scale=s["branch_scale"], eps=EPS)
    else:
        tgc.tgc_block_norm_bwd(s["y"], s["r"], s["dr"], s["dh"], gate=s["gate"], post=case["post"],
                               post_weight=s["post_w"], post_bias=s["post_b"], pre=case["pre"],
                               pre_weight=s["pre_w"], res_scale=s["res_scale"], branch_scale=s["branch_scale"],
                               eps=EPS, dx=s["dx"], dy=s["dy"], dgate=s["dgate"], dpost_weight=s["dpost_w"],
                               dpost_bias=s["dpost_b"], dpre_weight=s["dpre_w"], dpre_bias=s["dpre_b"])
    return {k: s[k] for k in _outputs(case) if s[k] is not None}


def _outputs(case):
    return {"linear": ("y", "z"), "grouped": ("y", "z"), "linear_bwd": ("dx", "dw", "db"),
            "grouped_bwd": ("dx", "dw", "db"), "norm": ("r", "h"),
            "norm_bwd": ("dx", "dy", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b")}[case["op"]]


def run(state):
    case = state["case"]
    if own:
        return _own_pass(state, case)
    op = case["op"]
    if op == "norm":
        out = _plain_block_norm(state, case)
    elif op == "norm_bwd":
        out = _plain_block_norm_bwd(state, case)
    elif op.endswith("_bwd"):
        out = _plain_linear_bwd(state, case)
    else:
        out = _plain_linear({"res": None, **state}, case)
    return {k: out[k] for k in _outputs(case) if k in out}


# ------------------------------------------------------------------------------------------ its cost


def work(case):
    if case["op"].startswith("norm"):
        es = 4 if case["dtype"] == "f32" else 2
        M, D, x = case["M"], case["D"], int(case["residual"])
        gate = case["gates"] * D
        vectors = sum((1 + int(case[k] == "layer" and case["affine_bias"])) * D for k in ("post", "pre") if case[k] != "none")
        if case["op"] == "norm":  # reads y, x, gate, weights; writes r, h
            return {"bytes": es * (M * D * (3 + x) + gate + vectors), "flops": 14 * M * D}
        # reads y (where a post norm or a gate needs it), r, dr, dh, gate, weights; writes dx, dy and the parameters' gradients
        y = int(case["post"] != "none" or case["gates"] > 0)
        return {"bytes": es * (M * D * (4 + x + y) + 2 * gate + 2 * vectors), "flops": 30 * M * D}
    M, K, N = case["M"], case["K"], case["N"]
    act, bias = int(case["act"] != "none"), int(case["bias"])
    used, E = 1, 1
    if "E" in case:
        used, E = sum(n > 0 for n in _group_sizes(case)), case["E"]
    if case["op"].endswith("_bwd"):  # reads dy, z, x, the weights in use; writes dx, dw, db
        return {"bytes": 2 * (M * N * (1 + act) + 2 * M * K + (used + E) * N * K + bias * E * N), "flops": 4 * M * N * K}
    y = M * N * (1 + int(case["keep_z"]) + int(case.get("residual", False)))
    return {"bytes": 2 * (M * K + used * N * K + y + bias * used * N), "flops": 2 * M * N * K}


# ------------------------------------------------------------------------------------------ in 64 bits


def _exact_act(z, act):
    f = torch.nn.functional
    return {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"),
            "silu": f.silu}[act](z)


def _exact_norm(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        return torch.nn.functional.layer_norm(v, (v.shape[1],), w, b, EPS)
    return v * torch.rsqrt(v.pow(2).mean(-1, keepdim=True) + EPS) * w


def exact(case, seed):
    if case["op"].startswith("norm") is False and case["M"] * case["K"] * case["N"] > 5e12:
        return None
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    M = case["M"]
    if case["op"].startswith("norm"):
        leaf = {k: d[k].requires_grad_() for k in ("x", "y", "gate", "post_w", "post_b", "pre_w", "pre_b")
                if d[k] is not None}
        branch = _exact_norm(d["y"], case["post"], d["post_w"], d["post_b"])
        if d["gate"] is not None:
            G = case["gates"]
            branch = (branch.view(G, M // G, -1) * d["gate"][:, None, :]).reshape(M, -1)
        r = s["branch_scale"] * branch
        if d["x"] is not None:
            r = r + s["res_scale"] * d["x"]
        if case["op"] == "norm":
            return {"r": r.detach(), "h": _exact_norm(r, case["pre"], d["pre_w"], d["pre_b"]).detach()}
        kept = d["r"].requires_grad_()
        h = _exact_norm(kept, case["pre"], d["pre_w"], d["pre_b"])
        pre = [k for k in ("pre_w", "pre_b") if k in leaf]
        first = torch.autograd.grad(h, [kept] + [leaf[k] for k in pre], d["dh"])
        rest = [k for k in leaf if k not in pre]
        second = torch.autograd.grad(r, [leaf[k] for k in rest], d["dr"] + first[0])
        found = {"d" + k: v for k, v in [*zip(pre, first[1:]), *zip(rest, second)]}
        return {k: found[k] for k in _outputs(case) if k in found}
    w = d["w"] if "E" in case else d["w"][None]
    starts = [0]
    for n in s["sizes"]:
        starts.append(starts[-1] + n)
    if case["op"].endswith("_bwd"):
        dz = d["dy"]
        if d["z"] is not None:
            z = d["z"].requires_grad_()
            dz = torch.autograd.grad(_exact_act(z, case["act"]), z, dz)[0]
        dx, dw = torch.zeros_like(d["x"]), torch.zeros_like(w)
        db = torch.zeros(w.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
        for e, (i, j) in enumerate(zip(starts, starts[1:])):
            dx[i:j] = torch.einsum("mn,nk->mk", dz[i:j], w[e])
            dw[e] = torch.einsum("mn,mk->nk", dz[i:j], d["x"][i:j])
            db[e] = torch.einsum("mn->n", dz[i:j])
        out = {"dx": dx, "dw": dw.view_as(d["w"])}
        if case["bias"]:
            out["db"] = db.view_as(d["b"])
        return out
    z = torch.zeros(M, case["N"], dtype=torch.float64, device="cuda")
    for e, (i, j) in enumerate(zip(starts, starts[1:])):
        z[i:j] = torch.einsum("mk,nk->mn", d["x"][i:j], w[e])
        if case["bias"]:
            z[i:j] += d["b"][e] if "E" in case else d["b"]
    y = _exact_act(z, case["act"])
    if case.get("residual"):
        y = y + d["res"]
    return {"y": y, "z": z} if case["keep_z"] else {"y": y}
