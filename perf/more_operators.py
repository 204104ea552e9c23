"""Cases and plain forms of the operators that serve a batch from one cache of pages.

Three operators that a serving loop calls around the decode step, in this order:

``tables``  block tables and slot maps from request lengths: pages of a free list are handed to
            the slots that grow or begin, those of slots that shrink or end are given back, and
            every new token gets its cache slot and position;
``norm``    norms of the query and key heads with the position rotation in the same pass, with the
            fused QKV bias, straight from the fused projection, into dense rows or, by the slot
            map, into the cache (rounded, or quantised with a scale per row);
``prefix``  the decode step of a batch whose slots share a long prefix: each slot attends to the
            first rows of the prefix and to its own rows, and the prefix is read once for all.

Where ``own`` is false ``run`` computes them with elementary torch operations in 32 bits;
where it is true it makes the library's calls.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
EB = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # every slot of a 70B-shaped batch has one more token: once per step, mostly no new page
        dict(name="tables_step", op="tables", kind="step", b=64, lmax=8192, page=256, lo=1, hi=8191),
        # prompts of a whole batch begin together
        dict(name="tables_admit", op="tables", kind="admit", b=256, lmax=8192, page=128, lo=1, hi=8191),
        # slots end, shrink, grow by one and begin in one call; most slots that a context holds
        dict(name="tables_churn", op="tables", kind="churn", b=1023, lmax=16384, page=256, lo=129, hi=16383),
        # a 7B-shaped step's eight tokens, dense: the smallest call, once per layer and step
        dict(name="norm_step_7b", op="norm", tokens=8, hq=32, hkv=32, d=128, dtype="f16", axes=1, rotary=128,
             pairing="halves", order="sections", fused=False, bias=False, fill="", page=0, far=4096),
        # a prompt of video patches and text for a 70B-shaped decoder, from the fused projection into pages, odd length
        dict(name="norm_video_fill", op="norm", tokens=16381, hq=64, hkv=8, d=128, dtype="bf16", axes=3, rotary=128,
             pairing="halves", order="sections", fused=True, bias=True, fill="bf16", page=256, far=100000),
        # prompts into an INT8 cache, partial rotation, adjacent pairs
        dict(name="norm_int8_fill", op="norm", tokens=4001, hq=32, hkv=32, d=128, dtype="f16", axes=1, rotary=64,
             pairing="adjacent", order="sections", fused=True, bias=False, fill="i8", page=0, far=32768),
        # a prompt in 32 bits, dense, heads of 64
        dict(name="norm_f32", op="norm", tokens=1001, hq=40, hkv=40, d=64, dtype="f32", axes=2, rotary=64,
             pairing="halves", order="interleaved", fused=True, bias=True, fill="", page=0, far=1000000),
        # a few chats behind one system prompt, 7B-shaped: the smallest call, once per layer and step
        dict(name="prefix_few_7b", op="prefix", b=4, t=1, hq=32, hkv=32, d=128, lmax=512, lo=17, hi=90, rows=777,
             seen="all", dtype="f16", cache="f16", out="f16", page=0, bias=False),
        # a 70B-shaped ragged batch behind a long prompt, all in one pool of pages, some slots without the prompt
        dict(name="prefix_70b", op="prefix", b=64, t=1, hq=64, hkv=8, d=128, lmax=2048, lo=1, hi=1023, rows=8191,
             seen="some", dtype="bf16", cache="bf16", out="bf16", page=256, bias=True),
        # many samples of one 7B-shaped question, fp32 output
        dict(name="prefix_samples_7b", op="prefix", b=100, t=1, hq=32, hkv=32, d=128, lmax=1024, lo=301, hi=500,
             rows=4000, seen="all", dtype="f16", cache="f16", out="f32", page=0, bias=False),
        # a long document read by many 70B-shaped slots, two new tokens per slot
        dict(name="prefix_document", op="prefix", b=64, t=2, hq=64, hkv=8, d=128, lmax=512, lo=33, hi=300, rows=32768,
             seen="all", dtype="bf16", cache="bf16", out="bf16", page=0, bias=False),
        # the INT8 cache's form, slots that share less and less of the prompt
        dict(name="prefix_int8", op="prefix", b=32, t=1, hq=64, hkv=8, d=128, lmax=512, lo=5, hi=400, rows=8000,
             seen="each", dtype="f16", cache="i8", out="f16", page=128, bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["tables", "norm", "prefix", "prefix"])
    if op == "tables":
        b = _log(rng, 1, 1024)
        page = rng.choice([128, 256, 512])
        hi = _log(rng, 2, min(16383, 1023 * 16383 // b))
        kind = rng.choice(["step", "admit", "churn", "churn"])
        return dict(op=op, kind=kind, b=b, lmax=-(-(hi + 1) // 16) * 16, page=rng.choice([0, page, page]), lo=rng.randint(1, hi),
                    hi=hi)
    d = rng.choice([64, 128, 128])
    if op == "norm":
        hq, hkv = rng.choice([(32, 32), (40, 40), (64, 8), (64, 1), (28, 4), (7, 1), (12, 3)])
        dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
        fill = rng.choice(["", dtype, dtype, rng.choice(["f32", "f16", "bf16", "i8", "i8"])])
        most = 16381 * 80 * 128 * 2 // ((hq + 2 * hkv) * d * EB[dtype])
        return dict(op=op, tokens=_log(rng, 1, min(most, 20000)), hq=hq, hkv=hkv, d=d, dtype=dtype,
                    axes=rng.choice([1, 1, 2, 3, 4]), rotary=rng.choice([d, d, d // 2, 2 * rng.randint(4, d // 2)]),
                    pairing=rng.choice(["halves", "halves", "adjacent"]), order=rng.choice(["sections", "interleaved"]),
                    fused=bool(fill) or rng.random() < 0.5, bias=rng.random() < 0.5, fill=fill,
                    page=rng.choice([0, 128, 256]), far=_log(rng, 1000, 1000000))
    cache = rng.choice(["f32", "f16", "bf16", "bf16", "i8"])
    dtype = "f16" if cache == "i8" else cache
    hq, hkv = rng.choice([(32, 32), (40, 40), (64, 8), (64, 8), (64, 1), (28, 4), (12, 3), (7, 1)])
    b, t = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 4])
    # products of a drawn case: no more than the largest listed one's, an eighth in 32 bits
    most = 64 * 2 * 64 * 32768 * 128 // (8 if cache == "f32" else 1)
    rows = _log(rng, 1, min(32768, most // (b * t * hq * d)))
    hi = _log(rng, 1, max(2, min(2000, 64 * 8 * 2048 // (b * hkv))))
    lo = rng.randint(0, hi)
    return dict(op=op, b=b, t=t, hq=hq, hkv=hkv, d=d, lmax=-(-(hi + t) // 16) * 16, lo=lo, hi=hi, rows=rows,
                seen=rng.choice(["all", "all", "some", "each"]), dtype=dtype, cache=cache,
                out=rng.choice([dtype, dtype, "f32"]), page=rng.choice([0, 0, 128, 256]), bias=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _normal(g, shape, dtype):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(generator=g)


def _spread(lo, hi, b):
    """b whole numbers spread evenly over lo .. hi."""
    return [round(x) for x in torch.linspace(lo, hi, b, dtype=torch.float64).tolist()]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _shuffled(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def _old_new(c):
    """Lengths before and after the call, slot by slot."""
    lens = _spread(c["lo"], c["hi"], c["b"])
    if c["kind"] == "step":
        return lens, [n + 1 for n in lens]
    if c["kind"] == "admit":
        return [0] * len(lens), lens
    # in turn: a slot ends, shrinks to half, grows by one, begins in a slot that was empty
    old = [n if i % 4 < 3 else -1 for i, n in enumerate(lens)]
    new = [(-1, n // 2, n + 1, n)[i % 4] for i, n in enumerate(lens)]
    return old, new


def _pages(n, page):
    return -(-max(n, 0) // page)


def _prefix_lens(c):
    """Rows of the prefix that each slot sees."""
    if c["seen"] == "each":
        return _spread(0, c["rows"], c["b"])
    return [0 if c["seen"] == "some" and i % 4 == 3 else c["rows"] for i in range(c["b"])]


def _sections(c):
    pairs, axes = c["rotary"] // 2, c["axes"]
    return [pairs * (a + 1) // axes - pairs * a // axes for a in range(axes)]


def _pair_axes(c):
    """Axis of each pair: whole sections one after the other, or round robin while a section lasts."""
    sec = _sections(c)
    if c["order"] == "sections":
        return [a for a, n in enumerate(sec) for _ in range(n)]
    return [a for k in range(max(sec)) for a, n in enumerate(sec) if k < n]


def _prepare_tables(c, g):
    old, new = _old_new(c)
    b, page = c["b"], c["page"]
    turn = _shuffled(g, b)
    s = {"c": c, "old": _ints(old)[turn].contiguous(), "new": _ints(new)[turn].contiguous(), "per": 0}
    total = sum(max(0, max(n, 0) - max(o, 0)) for o, n in zip(old, new))
    s["cap"] = -(-total // 64) * 64 + 64  # a token buffer of a fixed size, its end unused
    if page:
        s["per"] = -(-c["lmax"] // page)
        held = sum(_pages(n, page) for n in old)
        need = sum(max(0, _pages(n, page) - _pages(o, page)) for o, n in zip(old, new))
        s["pool"] = held + need + 7
        order = _shuffled(g, s["pool"]).to(torch.int32)
        # the slots hold the first pages of the order, the free list the others (then room for those that come back)
        count = (s["old"].clamp(min=0) + page - 1) // page
        first = torch.cumsum(count, 0) - count
        i = torch.arange(s["per"], device="cuda")
        at = (first.view(b, 1) + i).clamp(max=s["pool"] - 1)
        s["table"] = torch.where(i < count.view(b, 1), order[at], -1).to(torch.int32).contiguous()
        s["free"] = torch.full((s["pool"],), -1, dtype=torch.int32, device="cuda")
        s["free"][:s["pool"] - held] = order[held:]
        s["n_free"] = _ints([s["pool"] - held])
        s["n_free_out"] = torch.zeros_like(s["n_free"])
    s["served"], s["offsets"] = torch.zeros_like(s["old"]), _ints([0] * (b + 1))
    s["slots"], s["positions"] = _ints([0] * s["cap"]), _ints([0] * s["cap"])
    if own:
        import decode_step_masked_gb300 as ftd
        s["step"] = ftd.DecodeStep(b, 1, 1, 64, c["lmax"], "bf16", "bf16",
                                   **(dict(page_size=page, num_pages=s["pool"]) if page else {}))
    return s


def _prepare_norm(c, g):
    n, hq, hkv, d, dt, page = c["tokens"], c["hq"], c["hkv"], c["d"], DT[c["dtype"]], c["page"]
    s = {"c": c, "v": None, "slots": None, "scales": None}
    if c["fused"]:
        qkv = _normal(g, (n, (hq + 2 * hkv) * d), dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
    else:
        s["q"], s["k"] = _normal(g, (n, hq * d), dt), _normal(g, (n, hkv * d), dt)
    s["bias"] = _normal(g, ((hq + 2 * hkv) * d,), dt) * 0.1 if c["bias"] else None
    s["qw"], s["kw"] = 1.0 + 0.2 * _normal(g, (d,), dt), 1.0 + 0.2 * _normal(g, (d,), dt)
    start = torch.randint(0, c["far"], (1,), device="cuda", generator=g)
    i = torch.arange(n, device="cuda")
    steps = [i // 299, (i // 23) % 13, i % 23, i % 7] if c["axes"] > 1 else [i]  # frames of 13 x 23 patches
    s["pos"] = (torch.stack(steps[:c["axes"]]) + start).to(torch.int32).contiguous()
    s["axis_of"] = torch.tensor(_pair_axes(c), device="cuda")
    s["q_out"] = torch.empty((n, hq * d), dtype=dt, device="cuda")
    s["k_out"] = s["v_out"] = None
    lmax, opts = 16, {}
    if c["fill"]:
        # four sequences of the batch, or pages in any order; the batch's last tokens are padding
        if page:
            pages = -(-n // page)
            s["slots"] = _shuffled(g, pages)[i // page] * page + i % page
            lmax, shape, opts = pages * page, (pages, hkv, page, d), dict(page_size=page, num_pages=pages)
        else:
            lmax = -(-n // 4 // 16) * 16 + 16
            s["slots"], shape = i // (lmax - 3) * lmax + i % (lmax - 3), (4, hkv, lmax, d)
        s["slots"] = torch.where(i < n - n // 100, s["slots"], -1).to(torch.int32)
        s["k_cache"], s["v_cache"] = (torch.zeros(shape, dtype=DT[c["fill"]], device="cuda") for _ in range(2))
        if c["fill"] == "i8":
            s["scales"] = torch.zeros((2,) + shape[:-1], device="cuda")
            s["wide"] = [torch.empty(shape, dtype=torch.float16, device="cuda") for _ in range(2)]
    else:
        s["k_out"] = torch.empty((n, hkv * d), dtype=dt, device="cuda")
        s["v_out"] = torch.empty((n, hkv * d), dtype=dt, device="cuda") if c["fused"] else None
    if own:
        import decode_step_masked_gb300 as ftd
        s["step"] = ftd.DecodeStep(1 if page or not c["fill"] else 4, hq, hkv, d, lmax, c["dtype"], c["fill"] or c["dtype"],
                                   **opts)
        s["step"].set_rope(c["axes"], _sections(c), rotary_dim=c["rotary"], pairing=c["pairing"], order=c["order"])
    return s


def _prepare_prefix(c, g):
    b, t, hq, hkv, d, lmax, page = c["b"], c["t"], c["hq"], c["hkv"], c["d"], c["lmax"], c["page"]
    dt, ct = DT[c["dtype"]], DT[c["cache"]]
    s = {"c": c, "table": None, "prefix_table": None, "scales": None, "prefix_scales": None, "k_prefix": None, "v_prefix": None}
    s["lens"] = _ints([min(n, lmax - t) for n in _spread(c["lo"], c["hi"], b)])[_shuffled(g, b)].contiguous()
    s["prefix_lens"] = _ints(_prefix_lens(c))[_shuffled(g, b)].contiguous()
    s["n"] = min(c["hi"], lmax - t) + t

    def rows(shape):
        if c["cache"] == "i8":
            return (torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g) for _ in range(2))
        return (_normal(g, shape, ct) for _ in range(2))

    def scales(shape):
        return torch.rand((2,) + tuple(shape[:-1]), device="cuda", generator=g) * 0.02 + 0.005 if c["cache"] == "i8" else None

    opts = {}
    if page:
        per, first = -(-lmax // page), -(-c["rows"] // page)
        order = _shuffled(g, b * per + first).to(torch.int32)
        s["table"], s["prefix_table"] = order[first:].view(b, per).contiguous(), order[:first].contiguous()
        shape = (order.numel(), hkv, page, d)
        opts = dict(page_size=page, num_pages=order.numel())
    else:
        shape = (b, hkv, lmax, d)
        s["k_prefix"], s["v_prefix"] = rows((hkv, c["rows"], d))
        s["prefix_scales"] = scales((hkv, c["rows"], d))
    s["k"], s["v"] = rows(shape)
    s["scales"] = scales(shape)
    s["q"] = _normal(g, (b, t, hq, d), dt)
    s["k_new"], s["v_new"] = _normal(g, (b, t, hkv, d), dt), _normal(g, (b, t, hkv, d), dt)
    s["bias"] = _normal(g, ((hq + 2 * hkv) * d,), dt) * 0.1 if c["bias"] else None
    s["out"] = torch.empty((b, t, hq, d), dtype=DT[c["out"]], device="cuda")
    if own:
        import decode_step_masked_gb300 as ftd
        s["step"] = ftd.DecodeStep(b, hq, hkv, d, lmax, c["dtype"], c["cache"], out_dtype=c["out"], q_len=t, **opts)
        s["step"].enable_prefix()
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "tables":
        return _prepare_tables(case, g)
    return _prepare_norm(case, g) if case["op"] == "norm" else _prepare_prefix(case, g)


# ------------------------------------------------------------ plain forms
def _tables_plain(s):
    c, per = s["c"], s["per"]
    b, page = c["b"], c["page"]
    old, new = s["old"].clamp(min=0).long(), s["new"].clamp(min=0).long()
    served = torch.ones_like(old, dtype=torch.bool)
    if page:
        pool, n_free = s["pool"], s["n_free"].long()
        held, want = (old + page - 1) // page, (new + page - 1) // page
        grow, back = (want - held).clamp(min=0), (held - want).clamp(min=0)
        freed = back.sum()
        served = (grow == 0) | (torch.cumsum(grow, 0) <= n_free + freed)
        grow = grow * served
        i = torch.arange(per, device="cuda")
        # the pages that come back, slot by slot
        at = (torch.cumsum(back, 0) - back).view(b, 1) + i - want.view(b, 1)
        coming = (i >= want.view(b, 1)) & (i < held.view(b, 1))
        stack = torch.zeros(pool + 1, dtype=torch.int64, device="cuda")
        stack.scatter_(0, torch.where(coming, at, pool).view(-1), s["table"].long().view(-1))
        # they lie on top of the free list, and the slots that grow take from the top
        k = torch.cumsum(grow, 0).view(b, 1) - grow.view(b, 1) + i - held.view(b, 1)
        taken = (i >= held.view(b, 1)) & (i < (held + grow).view(b, 1))
        top = torch.where(k < freed, stack[(freed - 1 - k).clamp(0, pool)],
                          s["free"].long()[(n_free - 1 - (k - freed)).clamp(0, pool - 1)])
        s["table"].copy_(torch.where(taken, top, s["table"].long()))
        j = torch.arange(pool, device="cuda") - n_free
        s["free"].copy_(torch.where((j >= 0) & (j < freed - grow.sum()), stack[j.clamp(0, pool)], s["free"].long()))
        s["n_free_out"].copy_(n_free + freed - grow.sum())
    s["served"].copy_(torch.where(served, s["new"], s["old"]))
    count = torch.where(served, (new - old).clamp(min=0), 0)
    ends = torch.cumsum(count, 0)
    s["offsets"][1:].copy_(ends)
    tok = torch.arange(s["cap"], device="cuda")
    slot = torch.searchsorted(ends, tok, right=True).clamp(max=b - 1)
    pos = old[slot] + tok - (ends - count)[slot]
    live = tok < ends[-1]
    pos = torch.where(live, pos, 0)
    if page:
        place = s["table"].long()[slot, pos // page] * page + pos % page
    else:
        place = slot * c["lmax"] + pos
    s["slots"].copy_(torch.where(live, place, -1))
    s["positions"].copy_(torch.where(live, pos, 0))


def _turned(c, x, cos, sin):
    """Heads x [n][heads][D] turned by the pairs' angles."""
    r = c["rotary"]
    if c["pairing"] == "halves":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., r:]], -1)


def _put(s, cache, x, plane):
    """Rows x [n][Hkv][D] into the cache at their slots (INT8: codes, and their scales into a plane)."""
    page, hkv, lmax = cache.shape[2], cache.shape[1], cache.shape[2]
    keep = s["slots"] >= 0
    at, x = s["slots"][keep].long(), x[keep]
    if cache.dtype == torch.int8:
        top = x.abs().amax(-1)
        sc = torch.where(top == 0, torch.ones_like(top), top / 127.0)
        s["scales"][plane][at // page, :, at % page] = sc
        x = torch.round(x / sc.unsqueeze(-1)).clamp(-127, 127)
    cache[at // lmax, :, at % lmax] = x.to(cache.dtype)


def _norm_plain(s):
    c = s["c"]
    n, hq, hkv, d, r = c["tokens"], c["hq"], c["hkv"], c["d"], c["rotary"]
    # angles in 64 bits: far positions times small steps
    inv = torch.pow(10000.0, -torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    ang = s["pos"].double()[s["axis_of"]].T * inv  # [n][r / 2]
    cos, sin = torch.cos(ang).float().unsqueeze(1), torch.sin(ang).float().unsqueeze(1)

    def wide(x, first, heads):
        x = x.float()
        if s["bias"] is not None:
            x = x + s["bias"][first * d:(first + heads) * d].float()
        return x.view(n, heads, d)

    def head(x, w):
        return _turned(c, x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float(), cos, sin)

    s["q_out"].copy_(head(wide(s["q"], 0, hq), s["qw"]).view(n, hq * d))
    k = head(wide(s["k"], hq, hkv), s["kw"])
    v = None if s["v"] is None else wide(s["v"], hq + hkv, hkv)
    if c["fill"]:
        _put(s, s["k_cache"], k, 0)
        _put(s, s["v_cache"], v, 1)
        return
    s["k_out"].copy_(k.view(n, hkv * d))
    if v is not None:
        s["v_out"].copy_(v.view(n, hkv * d))


def _rows(c, x, table, n):
    """The first n rows of every slot as [B][Hkv][n]..., through its table where there is one."""
    if table is None:
        return x[:, :, :n]
    y = x[table[:, :-(-n // c["page"])].long()].transpose(1, 2)  # [B][Hkv][per][page]...
    return y.reshape(y.shape[:2] + (-1,) + y.shape[4:])[:, :, :n]


def _append(s, cache, new, first, plane):
    """The step's new rows into the cache (INT8: and their scales)."""
    c = s["c"]
    b, t, hkv, d = c["b"], c["t"], c["hkv"], c["d"]
    x = new.float()
    if s["bias"] is not None:
        x = x + s["bias"][first * d:(first + hkv) * d].float().view(hkv, d)
    at = s["lens"].long().view(b, 1) + torch.arange(t, device="cuda")
    if s["table"] is None:
        i, j = torch.arange(b, device="cuda").view(b, 1).expand(b, t), at
    else:
        i, j = s["table"].long().gather(1, at // c["page"]), at % c["page"]
    if s["scales"] is not None:
        top = x.abs().amax(-1)
        sc = torch.where(top == 0, torch.ones_like(top), top / 127.0)
        s["scales"][plane][i, :, j] = sc
        x = torch.round(x / sc.unsqueeze(-1)).clamp(-127, 127)
    cache[i, :, j] = x.to(cache.dtype)


def _prefix_plain(s):
    c = s["c"]
    b, t, hq, hkv, d, n, p = c["b"], c["t"], c["hq"], c["hkv"], c["d"], s["n"], c["rows"]
    _append(s, s["k"], s["k_new"], hq, 0)
    _append(s, s["v"], s["v_new"], hq + hkv, 1)
    at, L = torch.arange(n, device="cuda"), s["lens"].view(b, 1, 1)
    live = (at < L + t).view(b, 1, n, 1)

    def private(cache, plane):
        x = _rows(c, cache, s["table"], n).float()
        if s["scales"] is not None:
            x = x * _rows(c, s["scales"][plane], s["table"], n).unsqueeze(-1)
        return torch.where(live, x, 0.0)

    def shared(cache, prefix, plane):
        paged = prefix is None
        x = (_rows(c, cache, s["prefix_table"].view(1, -1), p)[0] if paged else prefix).float()
        if s["scales"] is not None:
            x = x * (_rows(c, s["scales"][plane], s["prefix_table"].view(1, -1), p)[0] if paged
                     else s["prefix_scales"][plane]).unsqueeze(-1)
        return x

    q = s["q"].float()
    if s["bias"] is not None:
        q = q + s["bias"][:hq * d].float().view(hq, d)
    g = hq // hkv
    q = (q * (1.0 / math.sqrt(d))).view(b, t, hkv, g, d).permute(2, 0, 1, 3, 4)  # [Hkv][B][T][group][D]
    # the prefix's scores, all slots' rows in one product; then each slot's own
    far = torch.matmul(q.reshape(hkv, b * t * g, d), shared(s["k"], s["k_prefix"], 0).transpose(1, 2)).view(hkv, b, t * g, p)
    far.masked_fill_(torch.arange(p, device="cuda") >= s["prefix_lens"].view(1, b, 1, 1), float("-inf"))
    near = torch.matmul(q.transpose(0, 1).reshape(b, hkv, t * g, d), private(s["k"], 0).transpose(2, 3)).view(b, hkv, t, g, n)
    seen = at <= L + torch.arange(t, device="cuda").view(1, t, 1)
    near = near.masked_fill(~seen.view(b, 1, t, 1, n), float("-inf")).view(b, hkv, t * g, n).transpose(0, 1)
    top = torch.maximum(far.amax(-1, keepdim=True), near.amax(-1, keepdim=True))
    far.sub_(top).exp_()
    near = torch.exp(near - top)
    total = far.sum(-1, keepdim=True) + near.sum(-1, keepdim=True)
    o = torch.matmul(far.view(hkv, b * t * g, p), shared(s["v"], s["v_prefix"], 1)).view(hkv, b, t * g, d)
    o = (o + torch.matmul(near.transpose(0, 1), private(s["v"], 1)).transpose(0, 1)) / total
    s["out"].copy_(o.view(hkv, b, t, g, d).permute(1, 2, 0, 3, 4).reshape(b, t, hq, d))


def _values(s):
    """An INT8 cache's rows as the values they stand for (rows of no token are zero)."""
    return [torch.mul(s[x], s["scales"][i].unsqueeze(-1), out=s["wide"][i]) for i, x in enumerate(("k_cache", "v_cache"))]


def run(state):
    s, c = state, state["c"]
    if c["op"] == "tables":
        if own:
            s["step"].tables(s["old"], s["new"], s["served"], block_table=s.get("table"), free_pages=s.get("free"),
                             n_free=s.get("n_free"), n_free_out=s.get("n_free_out"), offsets=s["offsets"], slots=s["slots"],
                             positions=s["positions"])
        else:
            _tables_plain(s)
        return [s[x] for x in ("served", "offsets", "slots", "positions", "table", "free", "n_free_out") if x in s]
    if c["op"] == "norm":
        if own:
            s["step"].norm_rope(s["q"], s["k"], s["v"], s["pos"], s["q_out"], s["k_out"], s["v_out"], bias=s["bias"],
                                q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, slots=s["slots"], k_cache=s.get("k_cache"),
                                v_cache=s.get("v_cache"), scales=s["scales"])
        else:
            _norm_plain(s)
        if c["fill"] == "i8":
            return [s["q_out"]] + _values(s)
        return [s[x] for x in ("q_out", "k_out", "v_out", "k_cache", "v_cache") if s.get(x) is not None]
    if own:
        s["step"].prefix(s["q"], s["k_new"], s["v_new"], s["lens"], s["prefix_lens"], s["out"], k_prefix=s["k_prefix"],
                         v_prefix=s["v_prefix"], prefix_scales=s["prefix_scales"], prefix_table=s["prefix_table"],
                         bias=s["bias"], k_cache=s["k"], v_cache=s["v"], scales=s["scales"], block_table=s["table"])
    else:
        _prefix_plain(s)
    return [s[x] for x in ("out", "k", "v", "scales") if s[x] is not None]


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "tables":
        old, new = _old_new(c)
        tokens = sum(max(0, max(n, 0) - max(o, 0)) for o, n in zip(old, new))
        moved = sum(abs(_pages(n, c["page"]) - _pages(o, c["page"])) for o, n in zip(old, new)) if c["page"] else 0
        # both lengths, the length served and an offset per slot; an entry read and written per page; two numbers per token
        return {"bytes": 16 * c["b"] + 8 * moved + 8 * tokens, "flops": float(tokens + c["b"])}
    d = c["d"]
    if c["op"] == "norm":
        n, hq, hkv, e = c["tokens"], c["hq"], c["hkv"], EB[c["dtype"]]
        heads = hq + hkv * (2 if c["fused"] else 1)
        kv = heads - hq
        kept = n - n // 100 if c["fill"] else n
        row = d * EB[c["fill"] or c["dtype"]] + (4 if c["fill"] == "i8" else 0)  # a key or value head as written
        small = ((hq + 2 * hkv) * d * e if c["bias"] else 0) + 2 * d * e + n * 4 * (c["axes"] + bool(c["fill"]))
        return {"bytes": n * hq * d * 2 * e + (n if not c["fill"] else kept) * kv * (d * e + row) + small,
                "flops": n * (hq + hkv) * (4 * d + 3 * c["rotary"]) + (n * heads * d if c["bias"] else 0)}
    b, t, hq, hkv = c["b"], c["t"], c["hq"], c["hkv"]
    row = 2 * d * EB[c["cache"]] + (8 if c["cache"] == "i8" else 0)  # a position's K and V (and scales) in one kv head
    lens = [min(n, c["lmax"] - t) for n in _spread(c["lo"], c["hi"], b)]
    seen = _prefix_lens(c)
    io = b * t * hq * d * (EB[c["dtype"]] + EB[c["out"]]) + b * t * hkv * (2 * d * EB[c["dtype"]] + row)
    return {"bytes": hkv * row * (max(seen) + sum(lens)) + io,
            "flops": 4.0 * t * hq * d * (sum(seen) + sum(n + t for n in lens))}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits, head by head and slot by slot; the tables hold whole numbers only."""
    c = case
    if c["op"] == "tables":
        return None
    s = prepare(case, seed)
    d, hq, hkv = c["d"], c["hq"], c["hkv"]
    if c["op"] == "norm":
        n, r, axis = c["tokens"], c["rotary"], _pair_axes(c)
        outs = []
        for x, w, heads, first in ((s["q"], s["qw"], hq, 0), (s["k"], s["kw"], hkv, hq), (s["v"], None, hkv, hq + hkv)):
            if x is None:
                continue
            y = x.double().clone()
            if s["bias"] is not None:
                y += s["bias"].double()[first * d:(first + heads) * d]
            y = y.view(n, heads, d)
            if w is not None:
                y = y / torch.sqrt(torch.sum(y ** 2, -1, keepdim=True) / d + 1e-6) * w.double()
                z = y.clone()
                for i in range(r // 2):
                    a, b = (i, i + r // 2) if c["pairing"] == "halves" else (2 * i, 2 * i + 1)
                    turn = s["pos"][axis[i]].double() * 10000.0 ** (-2.0 * i / r)
                    co, si = torch.cos(turn).view(n, 1), torch.sin(turn).view(n, 1)
                    z[..., a] = y[..., a] * co - y[..., b] * si
                    z[..., b] = y[..., a] * si + y[..., b] * co
                y = z
            if first and c["fill"]:
                kept = s["slots"] >= 0
                at, y = s["slots"][kept].long(), y[kept]
                if c["fill"] == "i8":
                    step = y.abs().amax(-1, keepdim=True) / 127.0
                    y = torch.round(y / step) * step
                full = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda")
                full[at // full.shape[2], :, at % full.shape[2]] = y
                outs.append(full)
            else:
                outs.append(y.reshape(n, heads * d))
        return outs
    if 4.0 * c["b"] * c["t"] * hq * d * c["rows"] > 4e11:
        return None
    b, t, g, p = c["b"], c["t"], hq // hkv, c["rows"]
    bias = s["bias"].double() if s["bias"] is not None else torch.zeros(((hq + 2 * hkv) * d,), dtype=torch.float64, device="cuda")
    page, i8 = c["page"], c["cache"] == "i8"

    def history(x, sc, table, n):
        """n rows of one slot (or of the prefix) as [Hkv][n][D]."""
        if table is not None:
            x = x[table].transpose(0, 1).reshape(hkv, -1, d)
            sc = None if sc is None else sc[table].transpose(0, 1).reshape(hkv, -1)
        x = x[:, :n].double()
        return x if sc is None else x * sc[:, :n].double().unsqueeze(-1)

    if page:
        pt = s["prefix_table"].long()
        kp, vp = (history(s[x], s["scales"][i] if i8 else None, pt, p) for i, x in enumerate(("k", "v")))
    else:
        kp, vp = (history(s[x + "_prefix"], s["prefix_scales"][i] if i8 else None, None, p) for i, x in enumerate(("k", "v")))
    lens, seen = s["lens"].tolist(), s["prefix_lens"].tolist()
    out = torch.zeros((b, t, hq, d), dtype=torch.float64, device="cuda")
    for i in range(b):
        keys, values = [], []
        for x, new, o, to, plane in ((s["k"], s["k_new"], hq, keys, 0), (s["v"], s["v_new"], hq + hkv, values, 1)):
            sc = s["scales"][plane] if i8 else None
            if page:
                old = history(x, sc, s["table"][i].long(), lens[i])
            else:
                old = history(x[i], None if sc is None else sc[i], None, lens[i])
            # the appended rows as the cache holds them: the bias is added and the sum rounded in 32 bits
            y = (new[i].float() + bias.float()[o * d:(o + hkv) * d].view(hkv, d)).transpose(0, 1)
            if i8:
                top = y.abs().amax(-1, keepdim=True)
                step = torch.where(top == 0, torch.ones_like(top), top / 127.0)
                y = torch.round(y / step).clamp(-127, 127).double() * step.double()
            else:
                y = y.to(x.dtype).double()
            to += [(kp if plane == 0 else vp)[:, :seen[i]], old, y]
        k, v = torch.cat(keys, 1), torch.cat(values, 1)
        q = s["q"][i].double() + bias[:hq * d].view(hq, d)
        for j in range(t):
            m = seen[i] + lens[i] + j + 1
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", q[j].view(hkv, g, d), k[:, :m]) / math.sqrt(d), -1)
            out[i, j] = torch.einsum("hgn,hnd->hgd", w, v[:, :m]).reshape(hq, d)
    return [out] + [None] * (2 + i8)
