"""What is measured of the attention step between a decoder layer's q|k|v and o linears: page assignment,
head norms with rotary positions into the paged cache, and decode attention over that cache.

``run`` computes each operator in plain torch (``own`` False) or calls the library (``own`` True) on the
same state.  Sizes are those of the two decoder layers this repository is measured on (32 query heads over
8 or 4 key/value heads of 128) and generic small, odd and wide ones."""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_WORKSPACE = 16 << 20     # bytes; the library's own query stays below this for every head layout drawn here


def listed():
    slots = {"op": "slots"}
    qk = {"op": "qk", "base": 1000000.0, "norm": True, "interleaved": False, "yarn": 1.0, "layout": "nhd"}
    att = {"op": "attention", "page": 16, "layout": "nhd", "stored": False, "lse": False, "idle": 0.0}
    return [
        # one decode step of a small server: a row for each request, now and then a new page
        dict(slots, name="slots decode 16", requests=16, rows=16, page=16, longest=4096, prompts=0.0, done=0.0, idle=0.0),
        # a mixed step: prompt chunks beside decode rows, finished and idle requests, rows padded for a captured graph
        dict(slots, name="slots mixed 256", requests=256, rows=8192, page=32, longest=8192, prompts=0.1, done=0.05,
             idle=0.05),
        # the chain's decode step: one token, fp32 from the grouped GEMV
        dict(qk, name="qk decode 1", rows=1, q_heads=32, kv_heads=8, dim=128, rot=128, x="f32", kv="f16", page=16,
             far=4096),
        # batched decode at the GEMV's widest batch, positions stretched for a long context
        dict(qk, name="qk decode 16 long", rows=16, q_heads=32, kv_heads=4, dim=128, rot=128, x="f16", kv="bf16",
             page=64, far=131072, yarn=4.0),
        # the prompt of the prefill workload, bf16 from the GEMM
        dict(qk, name="qk prompt 2048", rows=2048, q_heads=32, kv_heads=8, dim=128, rot=128, x="bf16", kv="bf16",
             page=16, far=2048),
        # odd counts: small heads, no norm, half of each head rotated in neighbouring pairs
        dict(qk, name="qk prompt 777 small heads", rows=777, q_heads=14, kv_heads=2, dim=64, rot=32, x="f32", kv="f16",
             page=24, far=30011, norm=False, interleaved=True, base=10000.0, layout="hnd"),
        # the start of one answer: latency
        dict(att, name="attention 1 x 512", requests=1, longest=512, ragged=False, q_heads=32, kv_heads=8, dim=128,
             kv="f16", out="f16"),
        # one very long context: the split over length
        dict(att, name="attention 1 x 131072", requests=1, longest=131072, ragged=False, q_heads=32, kv_heads=8, dim=128,
             kv="f16", out="f16", page=64),
        # the MoE model's heads at batch 16, written in o's stored column order
        dict(att, name="attention 16 ragged stored", requests=16, longest=4096, ragged=True, q_heads=32, kv_heads=4,
             dim=128, kv="bf16", out="f16", stored=True, layout="hnd"),
        # a full server: bandwidth
        dict(att, name="attention 128 ragged", requests=128, longest=4096, ragged=True, q_heads=32, kv_heads=8, dim=128,
             kv="f16", out="f16"),
        # small heads, seven queries to a key, pages that end inside a tile, idle requests
        dict(att, name="attention 33 odd", requests=33, longest=1999, ragged=True, q_heads=14, kv_heads=2, dim=64,
             kv="bf16", out="bf16", page=24, layout="hnd", idle=0.2, lse=True),
        # wide heads, all queries on one key head, with the softmax statistics
        dict(att, name="attention 8 wide", requests=8, longest=8192, ragged=True, q_heads=16, kv_heads=1, dim=256,
             kv="f16", out="bf16", page=32, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "qk", "attention"])
    page = rng.choice([1, 8, 16, 24, 32, 48, 64, 128])
    layout = rng.choice(["nhd", "hnd"])
    if op == "slots":
        b = _log(rng, 1, 1024)
        return {"op": op, "requests": b, "rows": b + _log(rng, 1, 16384), "page": page, "longest": _log(rng, 16, 16384),
                "prompts": rng.choice([0.0, 0.1, 0.5]), "done": rng.choice([0.0, 0.1]), "idle": rng.choice([0.0, 0.2])}
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    kv = rng.choice(["f16", "bf16"])
    if op == "qk":
        rows = max(1, _log(rng, 1, 4096) * 2048 // (max(q_heads + 2 * kv_heads, 16) * dim))
        return {"op": op, "rows": rows, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, 16]), "x": rng.choice(["f32", "f16", "bf16"]), "kv": kv,
                "page": page, "far": max(rows, _log(rng, 64, 1000000)), "norm": rng.random() < 0.7,
                "interleaved": rng.random() < 0.4, "yarn": rng.choice([1.0, 1.0, 4.0]),
                "base": rng.choice([10000.0, 1000000.0]), "layout": layout}
    b = _log(rng, 1, 300)
    most = 250000 * 1024 // (kv_heads * dim) // b           # keys a request, for at most 1 GB of cache
    return {"op": op, "requests": b, "longest": min(_log(rng, 1, 100000), most), "ragged": rng.random() < 0.7,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "kv": kv, "out": rng.choice(["f16", "bf16"]),
            "page": page, "layout": layout, "stored": rng.random() < 0.3, "lse": rng.random() < 0.5,
            "idle": rng.choice([0.0, 0.0, 0.2])}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pool(pages, page, heads, dim, layout, dtype):
    """A cache pool [pages][page][heads][dim] (any order in memory) that holds NaN until it is written."""
    if layout == "hnd":
        return torch.full((pages, heads, page, dim), float("nan"), dtype=dtype, device="cuda").transpose(1, 2)
    return torch.full((pages, page, heads, dim), float("nan"), dtype=dtype, device="cuda")


def _lengths(g, n, longest, ragged):
    if not ragged:
        return torch.full((n,), longest, dtype=torch.int32, device="cuda")
    return torch.randint(1, longest + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _frequencies(case):
    """Radians a position for each rotated pair (64 bits) and the factor on the rotated values: base^(-2i/rot),
    for a stretched context blended (YaRN) between f / s below one turn and f above 32 turns over 32768
    positions, with the factor 0.1 ln s + 1."""
    rot, s = case["rot"], case["yarn"]
    f = case["base"] ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if s == 1.0:
        return f.cuda(), 1.0
    at = lambda turns: rot * math.log(32768.0 / (turns * 2 * math.pi)) / (2 * math.log(case["base"]))
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return (f / s * ramp + f * (1 - ramp)).cuda(), 0.1 * math.log(s) + 1.0


def _prepare_slots(case, g):
    n, page, rows = case["requests"], case["page"], case["rows"]
    lens = _lengths(g, n, case["longest"], True)
    pick = torch.rand(n, generator=g, device="cuda")
    longest_chunk = max(2, (rows - n) // max(1, int(n * case["prompts"]))) if case["prompts"] else 2
    chunk = torch.randint(1, longest_chunk, (n,), generator=g, device="cuda")
    new = torch.ones(n, dtype=torch.int64, device="cuda")
    new = torch.where(pick < case["prompts"], chunk, new)
    new = torch.where(torch.cumsum(new, 0) > rows - n, torch.ones_like(new), new)      # the chunk budget is spent
    new = torch.where(pick > 1 - case["idle"], torch.zeros_like(new), new)
    new = torch.where((pick > 1 - case["idle"] - case["done"]) & (pick <= 1 - case["idle"]), -torch.ones_like(new), new)
    lens = torch.where((new > 1) & (pick < case["prompts"] / 2), torch.zeros_like(lens), lens)   # fresh prompts
    new = new.to(torch.int32)
    width = (case["longest"] + longest_chunk + page - 1) // page + 1
    used = int(((lens + page - 1) // page).sum())
    pages = n * ((case["longest"] + page - 1) // page) + (rows + page - 1) // page + n
    deal = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    held = (lens + page - 1) // page
    at = torch.arange(width, device="cuda", dtype=torch.int32)
    first = torch.cumsum(held, 0) - held
    table = torch.where(at[None, :] < held[:, None], deal[(first[:, None] + at[None, :]).clamp(max=pages - 1)],
                        torch.full((), -1, dtype=torch.int32, device="cuda"))
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - used] = deal[used:]
    i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")
    return {"lens": lens, "new": new, "table": table, "free": free,
            "n_free": torch.tensor([pages - used], dtype=torch.int32, device="cuda"), "lens_out": i32(n),
            "n_free_out": i32(1), "cu_rows": i32(n + 1), "positions": i32(rows), "slots": i32(rows)}


def _prepare_qk(case, g):
    rows, hq, hk, dim, page = case["rows"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    x = _DT[case["x"]]
    # one fused output of the three linears, channels of unequal energy
    energy = torch.exp(0.5 * torch.randn((hq + 2 * hk) * dim, generator=g, device="cuda"))
    qkv = (torch.randn((rows, (hq + 2 * hk) * dim), generator=g, device="cuda") * energy).to(x)
    gamma = lambda: (0.25 + 1.75 * torch.rand(dim, generator=g, device="cuda")).half() if case["norm"] else None
    pages = (rows + page - 1) // page + 2
    kv = _DT[case["kv"]]
    k, v = (_pool(pages, page, hk, dim, case["layout"], kv).fill_(0) for _ in range(2))
    freq, factor = _frequencies(case)
    if rows > 64:       # a prompt: rows in sequence, then a few padding rows
        first = int(torch.randint(0, case["far"] - rows + 1, (1,), generator=g, device="cuda"))
        pos = first + torch.arange(rows, device="cuda", dtype=torch.int32)
    else:
        pos = torch.randint(0, case["far"], (rows,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:rows].to(torch.int32)
    if rows > 8:
        slots[-3:] = -1
    s = {"q": qkv[:, :hq * dim], "k": qkv[:, hq * dim:(hq + hk) * dim], "v": qkv[:, (hq + hk) * dim:],
         "q_gamma": gamma(), "k_gamma": gamma(), "eps": 1e-6, "freq": freq, "factor": factor, "positions": pos,
         "slots": slots, "k_pool": k, "v_pool": v, "q_out": torch.zeros((rows, hq, dim), dtype=kv, device="cuda")}
    if own:             # the descriptors that a program keeps beside its pools
        import bit_spherical_vector_b200 as svq
        s["cache"], s["rope"] = svq.KvCache(k, v), svq.Rope(freq, interleaved=case["interleaved"], factor=factor)
    return s


def _prepare_attention(case, g):
    n, hq, hk, dim, page = case["requests"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    lens = _lengths(g, n, case["longest"], case["ragged"])
    idle = torch.rand(n, generator=g, device="cuda") < case["idle"]
    idle[0] = False
    if case["idle"] == 0 and case["ragged"] and n > 4:
        lens[n // 2] = 0                                            # an empty row in a padded batch
    width = (case["longest"] + page - 1) // page
    used = int(((lens + page - 1) // page).sum())
    deal = torch.randperm(used + 3, generator=g, device="cuda").to(torch.int32)
    held = (lens + page - 1) // page
    at = torch.arange(width, device="cuda", dtype=torch.int32)
    first = torch.cumsum(held, 0) - held
    table = torch.where(at[None, :] < held[:, None], deal[(first[:, None] + at[None, :]).clamp(max=used + 2)],
                        torch.full((), -1, dtype=torch.int32, device="cuda"))
    kv = _DT[case["kv"]]
    k, v = (_pool(used + 3, page, hk, dim, case["layout"], kv) for _ in range(2))
    where = at.repeat_interleave(page)[None, :] * page + torch.arange(page, device="cuda").repeat(width)[None, :]
    at_page, at_off = (where < lens[:, None]).nonzero(as_tuple=True)
    page_of, off_of = table[at_page, at_off // page].long(), at_off % page
    step = 1 << 17
    for i in range(0, page_of.numel(), step):                       # every key in use, a block at a time
        p, o = page_of[i:i + step], off_of[i:i + step]
        k[p, o] = torch.randn((p.numel(), hk, dim), generator=g, device="cuda").to(kv)
        v[p, o] = torch.randn((p.numel(), hk, dim), generator=g, device="cuda").to(kv)
    rows = torch.cat([torch.zeros(1, device="cuda"), torch.cumsum(~idle, 0)]).to(torch.int32)
    perm = torch.randperm(hq * dim, generator=g, device="cuda").to(torch.int32)
    order = None
    if case["stored"]:
        order = torch.empty_like(perm)
        order[perm.long()] = torch.arange(hq * dim, device="cuda", dtype=torch.int32)
    s = {"q": (1.5 * torch.randn((n, hq, dim), generator=g, device="cuda")).to(kv), "k_pool": k, "v_pool": v,
         "lens": lens, "table": table, "scale": 1.0 / math.sqrt(dim), "cu_rows": rows if case["idle"] else None,
         "order": order, "out": torch.zeros((n, hq * dim), dtype=_DT[case["out"]], device="cuda"),
         "lse": torch.zeros((n, hq), device="cuda") if case["lse"] else None,
         "workspace": torch.zeros(_WORKSPACE, dtype=torch.uint8, device="cuda")}
    if own:
        import bit_spherical_vector_b200 as svq
        s["cache"] = svq.KvCache(k, v)
    return s


def prepare(case, seed):
    g = _gen(seed)
    s = {"slots": _prepare_slots, "qk": _prepare_qk, "attention": _prepare_attention}[case["op"]](case, g)
    return dict(s, case=case)


# ------------------------------------------------------------------------------------------------ plain forms
def _plain_slots(s, page):
    lens, new, table, free, n_free = (s[k].long() for k in ("lens", "new", "table", "free", "n_free"))
    n, width = table.shape
    rows = s["slots"].numel()
    held = (lens + page - 1) // page
    add = new.clamp(min=0)
    need = (lens + add + page - 1) // page - held
    gone = torch.where(new < 0, held, torch.zeros_like(held))
    cu = torch.cat([torch.zeros_like(lens[:1]), torch.cumsum(add, 0)])
    first_new, first_gone = torch.cumsum(need, 0) - need, torch.cumsum(gone, 0) - gone
    # the stack: the free pages, then the released ones in request order
    at = torch.arange(free.numel(), device=free.device)
    back = (at - n_free).clamp(min=0)
    owner = (torch.searchsorted(torch.cumsum(gone, 0), back, right=True)).clamp(max=n - 1)
    page_back = table[owner, (back - first_gone[owner]).clamp(0, width - 1)]
    top = n_free + gone.sum()
    stack = torch.where(at < n_free, free, torch.where(at < top, page_back, free))
    left = top - need.sum()
    s["free"].copy_(torch.where((at >= n_free) & (at < left), stack, free))
    col = torch.arange(width, device=free.device)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    take = (top - 1 - (first_new[:, None] + col - held[:, None])).clamp(0, free.numel() - 1)
    full = torch.where(fresh, stack[take], table)
    s["table"].copy_(full)
    r = torch.arange(rows, device=free.device)
    b = torch.searchsorted(cu[1:], r, right=True).clamp(max=n - 1)
    pos = lens[b] + r - cu[b]
    slot = full[b, (pos // page).clamp(0, width - 1)] * page + pos % page
    live = r < cu[-1]
    gone_one = torch.full_like(r, -1)
    s["positions"].copy_(torch.where(live, pos, gone_one))
    s["slots"].copy_(torch.where(live, slot, gone_one))
    s["cu_rows"].copy_(cu)
    s["lens_out"].copy_(torch.where(new < 0, torch.zeros_like(lens), lens + add))
    s["n_free_out"].copy_(left)
    return s


def _plain_rotate(x, pos, freq, factor, interleaved):
    rot = 2 * freq.numel()
    a = pos.double()[:, None] * freq[None, :]
    cos, sin = ((f(a) * factor).float()[:, None, :] for f in (torch.cos, torch.sin))
    part, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        u, w = part[..., 0::2], part[..., 1::2]
        part = torch.stack([u * cos - w * sin, u * sin + w * cos], -1).flatten(-2)
    else:
        u, w = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([u * cos - w * sin, u * sin + w * cos], -1)
    return torch.cat([part, rest], -1)


def _plain_norm(x, gamma, eps):
    if gamma is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.float()


def _plain_qk(s, case):
    rows, hq, hk, dim, page = case["rows"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    live = s["slots"] >= 0
    turn = lambda x: _plain_rotate(x, s["positions"], s["freq"], s["factor"], case["interleaved"])
    q = turn(_plain_norm(s["q"].float().view(rows, hq, dim), s["q_gamma"], s["eps"])).to(s["q_out"].dtype)
    k = turn(_plain_norm(s["k"].float().view(rows, hk, dim), s["k_gamma"], s["eps"])).to(s["k_pool"].dtype)
    v = s["v"].reshape(rows, hk, dim).to(s["v_pool"].dtype)
    s["q_out"].copy_(torch.where(live[:, None, None], q, s["q_out"]))
    # padding rows write again what the last live slot of the table holds already
    at = s["slots"].long()
    last = live.long().cumsum(0).argmax()
    src = torch.where(live, torch.arange(rows, device=at.device), last)
    at = at[src]
    s["k_pool"][at // page, at % page] = k[src]
    s["v_pool"][at // page, at % page] = v[src]
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_attention(s, case):
    n, hq, hk, dim, page = case["requests"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    key = torch.arange(s["table"].shape[1] * page, device="cuda")
    live = key[None, :] < s["lens"][:, None]
    pages = s["table"].long().repeat_interleave(page, 1).clamp(min=0)
    k, v = (torch.where(live[:, :, None, None], s[w][pages, key % page].float(), torch.zeros((), device="cuda"))
            for w in ("k_pool", "v_pool"))
    row = torch.arange(n, device="cuda")
    if s["cu_rows"] is not None:
        row = s["cu_rows"][:-1].long().clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(n, hk, hq // hk, dim)
    score = torch.einsum("nhgd,nlhd->nhgl", q, k) * s["scale"]
    score = score.masked_fill(~live[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("nhgl,nlhd->nhgd", p, v) / torch.where(total == 0, torch.ones_like(total), total)
    o, lse = o.reshape(n, hq * dim), (torch.log(total) + top).view(n, hq)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    if s["cu_rows"] is not None:      # row r is that of the one request whose rows begin there and are not none
        r = torch.arange(n, device="cuda")
        who = torch.searchsorted(s["cu_rows"][1:].long(), r, right=True)
        keep, who = who < n, who.clamp(max=n - 1)
        o, lse = o[who], lse[who]
    if s["order"] is not None:
        o = torch.empty_like(o).index_copy_(1, s["order"].long(), o)
    s["out"].copy_(torch.where(keep[:, None], o, s["out"].float()))
    if s["lse"] is None:
        return {"out": s["out"]}
    s["lse"].copy_(torch.where(keep[:, None], lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    s, case = state, state["case"]
    if case["op"] == "slots":
        if own:
            import bit_spherical_vector_b200 as svq
            svq.svq_kv_assign(s["lens"], s["new"], case["page"], s["table"], s["free"], s["n_free"], s["lens_out"],
                              s["n_free_out"], s["cu_rows"], s["positions"], s["slots"])
        else:
            _plain_slots(s, case["page"])
        return {k: s[k] for k in ("table", "free", "lens_out", "n_free_out", "cu_rows", "positions", "slots")}
    if case["op"] == "qk":
        if own:
            import bit_spherical_vector_b200 as svq
            svq.svq_qk_norm_rope_cache(s["q"], s["k"], s["v"], s["q_gamma"], s["k_gamma"], s["eps"], s["rope"],
                                       s["positions"], s["slots"], s["cache"], s["q_out"])
            return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
        return _plain_qk(s, case)
    if own:
        import bit_spherical_vector_b200 as svq
        svq.svq_paged_attention(s["q"], s["cache"], s["lens"], s["table"], s["scale"], s["out"], s["workspace"],
                                cu_rows=s["cu_rows"], order=s["order"], lse=s["lse"])
        return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}
    return _plain_attention(s, case)


def work(case):
    if case["op"] == "slots":
        n, rows = case["requests"], case["rows"]
        fresh = rows / case["page"] if case["prompts"] else n / case["page"]
        return {"bytes": 4 * (2 * n + n + n + 1 + 2 * rows) + 8 * fresh + 8, "flops": 0}
    hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "qk":
        wide = 4 if case["x"] == "f32" else 2
        return {"bytes": case["rows"] * ((hq + 2 * hk) * dim * (wide + 2) + 8) + 4 * case["rot"] + (4 * dim if case["norm"] else 0),
                "flops": case["rows"] * (hq + hk) * (3 * case["rot"] + (4 * dim if case["norm"] else 0))}
    n = case["requests"] * (1 - case["idle"])
    keys = n * (case["longest"] / 2 if case["ragged"] else case["longest"])
    rows = n * hq * (4 * dim + (4 if case["lse"] else 0))
    return {"bytes": keys * (hk * dim * 4 + 4 / case["page"]) + rows, "flops": 4 * hq * dim * keys}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(s, case)
    return _exact_attention(s, case)


def _exact_qk(s, case):
    rows, dim, rot, page = case["rows"], case["dim"], case["rot"], case["page"]
    i = torch.arange(dim, device="cuda")
    half = rot // 2
    if case["interleaved"]:
        mate, pair, sign = i ^ 1, i // 2, torch.where(i % 2 == 0, -1.0, 1.0).double()
    else:
        mate, pair, sign = (i + half) % max(rot, 1), i % half, torch.where(i < half, -1.0, 1.0).double()
    turned = i < rot
    mate, pair = torch.where(turned, mate, i), torch.where(turned, pair, torch.zeros_like(i))
    angle = s["positions"].double()[:, None] * s["freq"][pair][None, :]
    c = torch.where(turned, torch.cos(angle) * s["factor"], torch.ones((), device="cuda", dtype=torch.float64))[:, None]
    w = torch.where(turned, sign * torch.sin(angle) * s["factor"], torch.zeros((), device="cuda", dtype=torch.float64))[:, None]

    def turn(x, heads, gamma):
        y = x.double().reshape(rows, heads, dim)
        if gamma is not None:
            y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / dim + s["eps"]) * gamma.double()
        return y * c + y[..., mate] * w

    q, k = turn(s["q"], case["q_heads"], s["q_gamma"]), turn(s["k"], case["kv_heads"], s["k_gamma"])
    v = s["v"].double().reshape(rows, case["kv_heads"], dim)
    live = (s["slots"] >= 0).nonzero()[:, 0]
    out = {"q": s["q_out"].double(), "k_pool": s["k_pool"].double(), "v_pool": s["v_pool"].double()}
    at = s["slots"][live].long()
    out["q"][live] = q[live]
    out["k_pool"][at // page, at % page] = k[live]
    out["v_pool"][at // page, at % page] = v[live]
    return out


def _exact_attention(s, case):
    hq, hk, dim, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    out, lse = s["out"].double(), torch.zeros((s["q"].shape[0], hq), device="cuda", dtype=torch.float64)
    lens = s["lens"].tolist()
    cu = s["cu_rows"].tolist() if s["cu_rows"] is not None else list(range(len(lens) + 1))
    for b, length in enumerate(lens):
        if cu[b] == cu[b + 1]:
            continue
        r = cu[b]
        if length == 0:
            out[r], lse[r] = 0.0, float("-inf")
            continue
        ps = s["table"][b, :(length + page - 1) // page].long()
        k, v = (s[w][ps].reshape(-1, hk, dim)[:length].double() for w in ("k_pool", "v_pool"))
        q = s["q"][r].double().view(hk, hq // hk, dim)
        score = torch.matmul(q, k.permute(1, 2, 0)) * s["scale"]
        lse[r] = torch.logsumexp(score, -1).reshape(hq)
        out[r] = torch.matmul(torch.softmax(score, -1), v.transpose(0, 1)).reshape(hq * dim)
    if s["order"] is not None:
        turned = torch.empty_like(out)
        turned[:, s["order"].long()] = out
        out = turned
    return {"out": out} if s["lse"] is None else {"out": out, "lse": lse}
