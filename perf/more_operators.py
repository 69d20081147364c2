"""The work the attention and cache operators are measured on.

  rope       rotary positions of query and key heads, and their gradients
  append     the new tokens' keys (rotated) and values into the pages of a cache, their queries rotated on the way
  attention  one new token of every sequence over its pages of the cache
  pages      copying, forking (with the room for the next tokens), freeing and compacting the cache's pages

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU from a seed, ``run`` makes one
pass (in plain torch operations, or through the library where ``own`` is true), ``exact`` computes the
same outputs from the definitions in 64 bits.  The page calls change their own bookkeeping, so a pass
over them starts by putting the saved bookkeeping back, on both sides alike.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------ cases


def _rope(op, T, Hq, Hk, D, R, layout, dtype, far, scaling):
    return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "layout": layout, "dtype": dtype, "far": far,
            "scaling": scaling}


def _append(seqs, tokens, mix, Hq, Hk, D, R, layout, dtype, page, far):
    """``tokens`` of ``seqs`` sequences in all, in uneven shares drawn from ``mix``; ``far``: the tokens they hold already."""
    return {"op": "append", "S": seqs, "T": tokens, "mix": mix, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "layout": layout,
            "dtype": dtype, "page": page, "far": far}


def _attention(seqs, most, mix, Hk, group, D, dtype, page, window=0, cap=0.0):
    """Lengths up to ``most``, drawn from ``mix``; the first sequence has the whole of it."""
    return {"op": "attention", "S": seqs, "most": most, "mix": mix, "Hk": Hk, "group": group, "D": D, "dtype": dtype,
            "page": page, "window": window, "cap": cap}


def _pages(op, pages, moved, mix, pools, page, width, dtype):
    """``pools`` (keys and values of the layers) of ``pages`` pages, each ``page`` tokens of ``width`` elements."""
    return {"op": op, "pages": pages, "moved": moved, "mix": mix, "pools": pools, "page": page, "width": width,
            "dtype": dtype}


def listed():
    return [
        # a training step: eight sequences of 1024, 32 query heads on 8 key heads
        {"name": "rope train", **_rope("rope", 8192, 32, 8, 128, 128, "half", "bf16", 0, "none")},
        # gradients in 32 bits, far positions under a scaled context, part of an odd-sized head, neighbouring pairs
        {"name": "rope odd backward", **_rope("rope_bwd", 1001, 6, 3, 90, 34, "interleaved", "f32", 900000, "yarn")},
        # one sequence's next token: the call is what costs
        {"name": "append token", **_append(1, 1, 1, 32, 8, 128, 128, "half", "bf16", 16, 1000)},
        # a decoding step of 64 sequences, half of each head rotated
        {"name": "append batch 64", **_append(64, 64, 2, 32, 8, 128, 64, "interleaved", "f16", 64, 8000)},
        # prompts of eight sequences, behind what they hold already
        {"name": "append prompts", **_append(8, 8191, 3, 32, 8, 128, 128, "half", "bf16", 16, 500)},
        # one sequence's next token over a short cache
        {"name": "attention token", **_attention(1, 900, 1, 8, 4, 128, "bf16", 16)},
        # a decoding step of 64 sequences, uneven lengths
        {"name": "attention batch 64", **_attention(64, 8192, 2, 8, 4, 128, "bf16", 64)},
        # two long contexts: few sequences, the length is what the work is split over
        {"name": "attention long", **_attention(2, 131071, 3, 8, 8, 128, "bf16", 64)},
        # a head of its own for every query head, a sliding window, capped scores, pages that no tile divides
        {"name": "attention window", **_attention(48, 5000, 4, 16, 1, 64, "f16", 24, 2000, 30.0)},
        # shared prefixes handed to another cache: 4 layers, 200 pages of each
        {"name": "pages copy", **_pages("copy", 1024, 200, 1, 8, 64, 1024, "bf16")},
        # a sampler's branches: 48 children of 12 parents, room for the next tokens of each
        {"name": "pages fork", **_pages("fork", 1500, 48, 2, 8, 16, 1024, "bf16")},
        # a third of the sequences end; what is left moves together
        {"name": "pages compact", **_pages("compact", 4000, 60, 3, 8, 16, 1024, "f16")},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _head(rng, step):
    return rng.choice([64, 128, 256, _log(rng, 16, 256) // step * step])


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "attention", "attention", "attention", "copy", "fork", "compact"])
    layout = rng.choice(["half", "interleaved"])
    if op.startswith("rope") or op == "append":
        Hk = _log(rng, 1, 16)
        Hq, D = Hk * rng.choice([1, 2, 4, 7, 8]), _head(rng, 2)
        R = rng.choice([D, D, max(2, D // 4 * 2), 2 * rng.randint(1, D // 2)])
        T = _log(rng, 1, 8192)
        while T * (Hq + 2 * Hk) * D > 8192 * 48 * 128:
            T = (T + 1) // 2
        dtype = rng.choice(["bf16", "f16", "f32"])
        while dtype == "f32" and T * (Hq + 2 * Hk) * D > 8192 * 24 * 128:
            T = (T + 1) // 2
        if op == "append":
            S, far = min(T, _log(rng, 1, 64)), rng.choice([0, 100, 20000])
            while S * far * Hk * D > 64 * 8000 * 8 * 128:
                far //= 2
            return _append(S, T, rng.randrange(1000), Hq, Hk, D, R, layout, dtype, _log(rng, 1, 256), far)
        return _rope(op, T, Hq, Hk, D, R, layout, dtype, rng.choice([0, 5000, 1000000]),
                     rng.choice(["none", "linear", "ntk", "yarn"]))
    if op == "attention":
        Hk, group, D = _log(rng, 1, 16), rng.choice([1, 2, 4, 5, 8, 16, 32]), _head(rng, 8)
        S, most = _log(rng, 1, 256), _log(rng, 1, 131072)
        while S * most * Hk * D > 2 * 131071 * 8 * 128 or S * most * Hk * max(group, 4) * D > 2 * 131071 * 64 * 128:
            S, most = (S + 1) // 2, (most + 1) // 2
        return _attention(S, most, rng.randrange(1000), Hk, group, D, rng.choice(["bf16", "f16"]), _log(rng, 1, 256),
                          rng.choice([0, 0, _log(rng, 1, 5000)]), rng.choice([0.0, 0.0, 20.0, 50.0]))
    pages, pools = _log(rng, 64, 20000), 2 * _log(rng, 1, 16)
    page, width = _log(rng, 1, 128), _log(rng, 8, 2048) // 8 * 8
    while pages * pools * page * width > 4000 * 8 * 16 * 1024:
        pages = max(64, pages // 2)
        page = max(1, page // 2)
    return _pages(op, pages, max(1, pages // rng.randint(8, 40)), rng.randrange(1000), pools, page, width,
                  rng.choice(["bf16", "f16", "f32"]))


# What a case's numbers stand for, drawn from the case alone.


def _shares(case):
    """Tokens of each sequence of an append: at least one, unevenly."""
    rng, S, T = random.Random(case["mix"]), case["S"], case["T"]
    cuts = sorted(rng.sample(range(1, T), S - 1)) if S > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def _held(case):
    rng = random.Random(case["mix"] + 1)
    return [rng.randint(0, case["far"]) for _ in range(case["S"])]


def _lengths(case):
    rng = random.Random(case["mix"])
    most, S = case["most"], case["S"]
    return [most] + [0 if S > 8 and rng.random() < 0.02 else 1 + int((most - 1) * rng.random() ** 0.7)
                     for _ in range(S - 1)]


def _tenants(case):
    """The lengths of the sequences that fill about two thirds of a cache's pages."""
    rng, left, lens = random.Random(case["mix"]), case["pages"] * 2 // 3, []
    while left > 0:
        n = min(left, _log(rng, 1, max(2, case["pages"] // 16)))
        left -= n
        lens.append(n * case["page"] - rng.randrange(case["page"]))
    return lens


def _fork_lists(case):
    """Parents, children and the tokens that each child is given room for."""
    rng, held = random.Random(case["mix"] + 7), len(_tenants(case))
    parents = [rng.randrange(held) for _ in range(max(1, min(held, case["moved"] // 4)))]
    src = [rng.choice(parents) for _ in range(case["moved"])]
    return src, [held + i for i in range(case["moved"])], [rng.randint(1, 2 * case["page"]) for _ in src]


def _ended(case):
    rng, held = random.Random(case["mix"] + 9), len(_tenants(case))
    return sorted(rng.sample(range(held), max(1, held // 3)))


# ------------------------------------------------------------------------------------------ inputs


def _frequencies(R, scaling):
    """Radians a position, in 64 bits, and the factor on the rotated values: base 10000, a context of 4096 stretched 8 times."""
    i = torch.arange(R // 2, dtype=torch.float64)
    plain = 10000.0 ** (-2.0 * i / R)
    if scaling == "linear":
        return plain / 8, 1.0
    if scaling == "ntk" and R > 2:
        return (10000.0 * 8.0 ** (R / (R - 2))) ** (-2.0 * i / R), 1.0
    if scaling == "yarn":
        turns = 4096 * plain / (2 * math.pi)  # of a pair over the context it was trained on
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        return plain * keep + plain / 8 * (1 - keep), 0.1 * math.log(8) + 1
    return plain, 1.0


def _paged(case, need, g, spare=5):
    """A shuffled block table for sequences of ``need`` tokens, and the number of pages behind it."""
    page = case["page"]
    counts = [-(-n // page) for n in need]
    total = sum(counts) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    wide = max(max(counts), 1)
    c = torch.tensor(counts, device="cuda")
    at = torch.arange(wide, device="cuda")[None] + (torch.cumsum(c, 0) - c)[:, None]
    table = torch.where(torch.arange(wide, device="cuda")[None] < c[:, None], order[at.clamp(max=total - 1)], -1)
    return table.to(torch.int32).contiguous(), total


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = {"case": case}
    if op.startswith("rope") or op == "append":
        T, Hq, Hk, D, R = case["T"], case["Hq"], case["Hk"], case["D"], case["R"]
        # heads lie side by side in the rows that the projection wrote
        rows = normal(T, Hq + 2 * Hk, D)
        s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
        s["q_out"] = torch.empty(T, Hq, D, device="cuda", dtype=dt)
        freqs, s["scale"] = _frequencies(R, case.get("scaling", "none"))
        s["freqs"] = freqs.cuda()
    if op.startswith("rope"):
        s["k_out"] = torch.empty(T, Hk, D, device="cuda", dtype=dt)
        start = torch.randint(0, case["far"] + 1, (1,), generator=g, device="cuda", dtype=torch.int32)
        s["pos"] = torch.arange(T, device="cuda", dtype=torch.int32) % 1024 + start
    elif op == "append":
        held, shares = ints(_held(case)), ints(_shares(case))
        s["table"], pages = _paged(case, [a + b for a, b in zip(_held(case), _shares(case))], g)
        s["seqs"] = torch.repeat_interleave(torch.arange(case["S"], device="cuda", dtype=torch.int32), shares)
        first = torch.cumsum(shares, 0) - shares
        s["pos"] = (torch.arange(T, device="cuda") - first[s["seqs"]] + held[s["seqs"]]).to(torch.int32)
        s["k_pages"], s["v_pages"] = normal(pages, case["page"], Hk, D), normal(pages, case["page"], Hk, D)
    elif op == "attention":
        S, Hk, D = case["S"], case["Hk"], case["D"]
        lens = _lengths(case)
        s["lens"] = ints(lens)
        s["table"], pages = _paged(case, lens, g)
        s["k_pages"], s["v_pages"] = normal(pages, case["page"], Hk, D), normal(pages, case["page"], Hk, D)
        s["q"] = normal(S, Hk * case["group"], D)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(S, Hk * case["group"], device="cuda")
    else:
        P, page = case["pages"], case["page"]
        s["pools"] = [normal(P, page, case["width"]) for _ in range(case["pools"])]
        if op == "copy":
            order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
            s["src"], s["dst"] = order[:case["moved"]].contiguous(), torch.flip(order, (0,))[:case["moved"]].contiguous()
            s["other"] = [normal(P, page, case["width"]) for _ in range(case["pools"])]
            return s
        lens = _tenants(case)
        src, dst, add = _fork_lists(case)
        table, used = _paged(case, lens, g, spare=P - sum(-(-n // page) for n in lens))
        rows = len(lens) + len(dst)
        wide = table.shape[1] + 3
        full = torch.full((rows, wide), -1, device="cuda", dtype=torch.int32)
        full[:len(lens), :table.shape[1]] = table
        refs = torch.zeros(P, device="cuda", dtype=torch.int32)
        refs[full[full >= 0].long()] = 1
        s["saved"] = {"table": full, "refs": refs, "lens": ints(lens + [0] * len(dst))}
        for k, v in s["saved"].items():
            s[k] = v.clone()
        if op == "fork":
            s["src"], s["dst"], s["add"] = ints(src), ints(dst), ints(add)
            s["forked"], s["grown"] = torch.empty_like(s["src"]), torch.empty_like(s["src"])
        else:
            s["ended"] = ints(_ended(case))
            s["used"] = torch.zeros(1, device="cuda", dtype=torch.int32)
    return s


# ------------------------------------------------------------------------------------------ one pass


def _plain_rotate(x, s, case, back=False):
    """Heads (T, H, D) rotated in 32 bits; the angles in 64."""
    R, T = case["R"], x.shape[0]
    angle = s["pos"].double()[:, None] * s["freqs"][None]
    cos = (torch.cos(angle) * s["scale"]).float()[:, None]
    sin = (torch.sin(angle) * s["scale"]).float()[:, None]
    if back:
        sin = -sin
    x = x.float()
    if case["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).reshape(T, -1, R)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_rope(s, case):
    dt, back = s["q"].dtype, case["op"] == "rope_bwd"
    return {"q_out": _plain_rotate(s["q"], s, case, back).to(dt), "k_out": _plain_rotate(s["k"], s, case, back).to(dt)}


def _plain_append(s, case):
    dt, page = s["q"].dtype, case["page"]
    pos = s["pos"].long()
    at = s["table"][s["seqs"].long(), pos // page].long()
    s["k_pages"][at, pos % page] = _plain_rotate(s["k"], s, case).to(dt)
    s["v_pages"][at, pos % page] = s["v"]
    return {"q_out": _plain_rotate(s["q"], s, case).to(dt), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attention(s, case):
    S, Hk, G, D, page = case["S"], case["Hk"], case["group"], case["D"], case["page"]
    at = s["table"].long().clamp(min=0)
    n = at.shape[1] * page
    k = s["k_pages"][at].reshape(S, n, Hk, D).permute(0, 2, 3, 1).float()
    v = s["v_pages"][at].reshape(S, n, Hk, D).permute(0, 2, 1, 3).float()
    x = (s["q"].float().view(S, Hk, G, D) @ k) * D ** -0.5
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    j, lens = torch.arange(n, device="cuda")[None], s["lens"][:, None]
    keep = j < lens
    if case["window"]:
        keep = keep & (j >= lens - case["window"])
    x = torch.where(keep[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return {"out": out.reshape(S, Hk * G, D).to(s["q"].dtype), "lse": lse.reshape(S, Hk * G)}


def _put_back(s):
    for k, v in s["saved"].items():
        s[k].copy_(v)


def _plain_copy(s, case):
    src, dst = s["src"].long(), s["dst"].long()
    for a, b in zip(s["pools"], s["other"]):
        b[dst] = a[src]
    return {"other": s["other"]}


def _plain_take(s, page, rows, have, get):
    """``get`` new pages for the sequences ``rows`` behind the ``have`` they hold: the lowest free ones, in order of the list."""
    refs, table = s["refs"], s["table"]
    free = torch.sort(refs != 0, stable=True).indices
    upto = torch.cumsum(get, 0)
    ok = (upto <= (refs == 0).sum()) & (have + get <= table.shape[1])
    first = upto - get
    j = torch.arange(table.shape[1], device="cuda")[None]
    new = (j >= have[:, None]) & (j < (have + get)[:, None]) & ok[:, None]
    pages = free[(first[:, None] + j - have[:, None]).clamp(0, len(free) - 1)]
    table[rows] = torch.where(new, pages.to(torch.int32), table[rows])
    refs.scatter_add_(0, torch.where(new, pages, 0).reshape(-1), new.reshape(-1).to(torch.int32))
    return ok, pages


def _plain_fork(s, case):
    page = case["page"]
    _put_back(s)
    src, dst, table, refs, lens = s["src"].long(), s["dst"].long(), s["table"], s["refs"], s["lens"]
    n = lens[src].long()
    whole, part = n // page, (n % page > 0).long()
    j = torch.arange(table.shape[1], device="cuda")[None]
    shared = torch.where(j < whole[:, None], table[src], -1)
    last = table[src, whole.clamp(max=table.shape[1] - 1)].long()
    table[dst] = shared
    ok, _ = _plain_take(s, page, dst, whole, part)
    given = (shared >= 0) & ok[:, None]
    refs.scatter_add_(0, torch.where(given, shared, 0).long().reshape(-1), given.reshape(-1).to(torch.int32))
    table[dst] = torch.where(ok[:, None], table[dst], -1)
    lens[dst] = torch.where(ok, lens[src], 0)
    s["forked"].copy_(ok)
    moves = ok & (part > 0)
    new = table[dst, whole.clamp(max=table.shape[1] - 1)].long()
    same = table[src, 0].long()  # where nothing moves, a page that nobody writes is copied onto itself
    new, last = torch.where(moves, new, same), torch.where(moves, last, same)
    for pool in s["pools"]:
        pool[new] = pool[last]
    have = -(-lens[dst].long() // page)
    get = -(-(lens[dst] + s["add"]).long() // page) - have
    ok, _ = _plain_take(s, page, dst, have, get)
    lens[dst] += torch.where(ok, s["add"], 0)
    s["grown"].copy_(ok)
    return {k: s[k] for k in ("pools", "table", "refs", "lens", "forked", "grown")}


def _plain_compact(s, case):
    _put_back(s)
    table, refs, lens, gone = s["table"], s["refs"], s["lens"], s["ended"].long()
    old = table[gone]
    refs.scatter_add_(0, old.clamp(min=0).long().reshape(-1), -(old >= 0).to(torch.int32).reshape(-1))
    table[gone] = -1
    lens[gone] = 0
    used = refs > 0
    count = used.sum()
    number = torch.arange(len(refs), device="cuda")
    movers, holes = used & (number >= count), ~used & (number < count)
    # the i-th mover goes to the i-th hole; there are at most half as many as pages, and where there are
    # fewer, a page that is neither is copied onto itself
    half = max(1, len(refs) // 2)
    src = torch.sort(torch.where(movers, 0, torch.where(holes, 2, 1)), stable=True).indices[:half]
    dst = torch.where(torch.arange(half, device="cuda") < movers.sum(),
                      torch.sort(~holes, stable=True).indices[:half], src)
    for pool in s["pools"]:
        pool[dst] = pool[src]
    number[src] = dst
    table.copy_(torch.where(table >= 0, number[table.clamp(min=0).long()].to(torch.int32), table))
    moved = refs[src]
    refs[src] = 0
    refs[dst] = moved
    s["used"].copy_(count)
    return {k: s[k] for k in ("pools", "table", "refs", "lens", "used")}


def _own_pass(s, case):
    import tile_gather_comm_gb300 as tgc
    op = case["op"]
    if op == "rope":
        tgc.tgc_rope(s["q"], s["q_out"], s["pos"], s["freqs"], k=s["k"], k_out=s["k_out"], layout=case["layout"],
                     scale=s["scale"])
        return {k: s[k] for k in ("q_out", "k_out")}
    if op == "rope_bwd":
        tgc.tgc_rope_bwd(s["q"], s["q_out"], s["pos"], s["freqs"], dk_out=s["k"], dk=s["k_out"], layout=case["layout"],
                         scale=s["scale"])
        return {k: s[k] for k in ("q_out", "k_out")}
    if op == "append":
        tgc.tgc_kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["pos"], seqs=s["seqs"], q=s["q"],
                          q_out=s["q_out"], freqs=s["freqs"], layout=case["layout"], scale=s["scale"])
        return {k: s[k] for k in ("q_out", "k_pages", "v_pages")}
    if op == "attention":
        tgc.tgc_paged_attention(s["q"], s["out"], s["k_pages"], s["v_pages"], s["table"], s["lens"], lse=s["lse"],
                                window=case["window"], softcap=case["cap"])
        return {k: s[k] for k in ("out", "lse")}
    if op == "copy":
        tgc.tgc_kv_copy(s["other"], s["pools"], s["dst"], s["src"])
        return {"other": s["other"]}
    _put_back(s)
    if op == "fork":
        tgc.tgc_kv_fork(s["pools"], s["refs"], s["table"], s["lens"], s["src"], s["dst"], case["page"], ok=s["forked"])
        tgc.tgc_kv_reserve(s["refs"], s["table"], s["lens"], s["dst"], s["add"], case["page"], ok=s["grown"])
        return {k: s[k] for k in ("pools", "table", "refs", "lens", "forked", "grown")}
    tgc.tgc_kv_free(s["refs"], s["table"], s["lens"], s["ended"])
    tgc.tgc_kv_compact(s["pools"], s["refs"], s["table"], s["used"])
    return {k: s[k] for k in ("pools", "table", "refs", "lens", "used")}


def run(state):
    case = state["case"]
    if own:
        return _own_pass(state, case)
    plain = {"rope": _plain_rope, "rope_bwd": _plain_rope, "append": _plain_append, "attention": _plain_attention,
             "copy": _plain_copy, "fork": _plain_fork, "compact": _plain_compact}
    return plain[case["op"]](state, case)


# ------------------------------------------------------------------------------------------ its cost


def _moves(case):
    """Pages that a fork or a compaction cannot do without moving (which ones move hangs on the shuffle; about how many does not)."""
    page, lens = case["page"], _tenants(case)
    if case["op"] == "fork":
        return sum(lens[p] % page > 0 for p in _fork_lists(case)[0])
    left = sum(-(-n // page) for i, n in enumerate(lens) if i not in set(_ended(case)))
    return left * (case["pages"] - left) // case["pages"]


def work(case):
    es, op = 4 if case["dtype"] == "f32" else 2, case["op"]
    if op.startswith("rope"):
        rows = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * es * rows * case["D"] + 4 * case["T"], "flops": 3 * rows * case["R"]}
    if op == "append":
        rows = case["T"] * (case["Hq"] + 2 * case["Hk"])
        return {"bytes": 2 * es * rows * case["D"] + 8 * case["T"],
                "flops": 3 * case["T"] * (case["Hq"] + case["Hk"]) * case["R"]}
    if op == "attention":
        keys = sum(min(n, case["window"] or n) for n in _lengths(case))
        q = case["S"] * case["Hk"] * case["group"]
        return {"bytes": 2 * es * keys * case["Hk"] * case["D"] + 2 * es * q * case["D"] + 4 * q,
                "flops": 4 * keys * case["Hk"] * case["group"] * case["D"]}
    moved = case["moved"] if op == "copy" else _moves(case)
    return {"bytes": 2 * es * case["pools"] * moved * case["page"] * case["width"] + 8 * case["pages"], "flops": 0}


# ------------------------------------------------------------------------------------------ in 64 bits


def _exact_turn(x, s, case, back=False):
    """Pairs as complex numbers, multiplied by scale * exp(i angle)."""
    R, x = case["R"], x.double()
    angle = torch.outer(s["pos"].double(), s["freqs"]) * (-1 if back else 1)
    turn = torch.polar(torch.full_like(angle, s["scale"]), angle)[:, None]
    out = x.clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
        out[..., :R // 2], out[..., R // 2:R] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:2], R // 2, 2).contiguous()) * turn
        out[..., :R] = torch.view_as_real(z).reshape(*x.shape[:2], R)
    return out


def _exact_attention(s, case):
    S, Hk, G, D, page = case["S"], case["Hk"], case["group"], case["D"], case["page"]
    out = torch.zeros(S, Hk * G, D, device="cuda", dtype=torch.float64)
    lse = torch.full((S, Hk * G), -math.inf, device="cuda", dtype=torch.float64)
    for b, n in enumerate(_lengths(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == first:
            continue
        j = torch.arange(first, n, device="cuda")
        at = s["table"][b, j // page].long()
        for h in range(Hk):
            k, v = s["k_pages"][at, j % page, h].double(), s["v_pages"][at, j % page, h].double()
            x = torch.einsum("gd,jd->gj", s["q"][b, h * G:(h + 1) * G].double(), k) / math.sqrt(D)
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, 1)
            out[b, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}


def _exact_pages(s, case):
    """The bookkeeping in Python, step by step."""
    page = case["page"]
    table, refs, lens = (s["saved"][k].tolist() for k in ("table", "refs", "lens"))
    pools = [p.double() for p in s["pools"]]

    def count(n):
        return -(-n // page)

    if case["op"] == "fork":
        src, dst, add = _fork_lists(case)
        forked, grown, new_lens = [], [], list(lens)
        free = [p for p, r in enumerate(refs) if r == 0]
        copies, asked = [], 0
        for a, b in zip(src, dst):
            part = lens[a] % page > 0
            asked += part
            forked.append(int(asked <= len(free)))
            if forked[-1]:
                whole = lens[a] // page
                for i in range(whole):
                    table[b][i] = table[a][i]
                    refs[table[a][i]] += 1
                if part:
                    p = free[asked - 1]
                    table[b][whole], refs[p] = p, 1
                    copies.append((p, table[a][whole]))
                new_lens[b] = lens[a]
        lens = new_lens
        for new, old in copies:
            for pool in pools:
                pool[new] = pool[old]
        free = [p for p, r in enumerate(refs) if r == 0]
        asked = 0
        for b, n in zip(dst, add):
            have = count(lens[b])
            get = count(lens[b] + n) - have
            asked += get
            grown.append(int(asked <= len(free) and have + get <= len(table[b])))
            if grown[-1]:
                for i in range(get):
                    p = free[asked - get + i]
                    table[b][have + i], refs[p] = p, 1
                lens[b] += n
        more = {"forked": forked, "grown": grown}
    else:
        for q in _ended(case):
            for p in table[q]:
                if p >= 0:
                    refs[p] -= 1
            table[q], lens[q] = [-1] * len(table[q]), 0
        used = sum(r > 0 for r in refs)
        movers = [p for p in range(used, len(refs)) if refs[p] > 0]
        holes = [p for p in range(used) if refs[p] == 0]
        to = dict(zip(movers, holes))
        for old, new in to.items():
            refs[new], refs[old] = refs[old], 0
            for pool in pools:
                pool[new] = pool[old]
        table = [[to.get(p, p) for p in row] for row in table]
        more = {"used": [used]}
    whole = {"table": table, "refs": refs, "lens": lens, **more}
    return {"pools": pools, **{k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in whole.items()}}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("rope"):
        return {k + "_out": _exact_turn(s[k], s, case, op == "rope_bwd") for k in ("q", "k")}
    if op == "append":
        k_pages, v_pages, pos = s["k_pages"].double(), s["v_pages"].double(), s["pos"].long()
        at = s["table"][s["seqs"].long(), torch.div(pos, case["page"], rounding_mode="floor")].long()
        k_pages[at, pos % case["page"]] = _exact_turn(s["k"], s, case)
        v_pages[at, pos % case["page"]] = s["v"].double()
        return {"q_out": _exact_turn(s["q"], s, case), "k_pages": k_pages, "v_pages": v_pages}
    if op == "attention":
        return _exact_attention(s, case)
    if op == "copy":
        other, src, dst = [p.double() for p in s["other"]], s["src"].tolist(), s["dst"].tolist()
        for a, b in zip(s["pools"], other):
            for i, j in zip(src, dst):
                b[j] = a[i].double()
        return {"other": other}
    return _exact_pages(s, case)
