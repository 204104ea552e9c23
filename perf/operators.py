"""Cases and plain forms of the operators around the decode step's cache.

Four operators that a decoder with a bounded cache calls next to the decode step itself:

``rope``    rotary positions with one to four axes (time, height, width, ...) applied to the
            query and key heads of the step's or a prompt's tokens, with the fused QKV bias,
            straight from the fused projection output when it is given as one;
``scored``  the decode step that also adds each cached position's attention weight, summed
            over the query rows of its kv head, to a running plane;
``evict``   eviction by that plane: each kv head keeps its sinks, its newest tokens and the
            heaviest others, and the kept rows behind the budget move into the holes before it;
``cross``   cross attention of a step's tokens (or beams) to an encoder's states, with
            lengths of their own.

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
        # a 7B-shaped step's eight tokens, one text axis: the smallest call, once per layer and step
        dict(name="rope_step_7b", op="rope", tokens=8, hq=32, hkv=32, d=128, dtype="f16", axes=1, rotary=128,
             pairing="halves", order="sections", fused=False, bias=False, far=4096),
        # a prompt of video patches and text for a 70B-shaped decoder, from the fused projection, odd length
        dict(name="rope_video_prompt", op="rope", tokens=16381, hq=64, hkv=8, d=128, dtype="bf16", axes=3, rotary=128,
             pairing="halves", order="sections", fused=True, bias=True, far=100000),
        # a prompt in 32 bits with partial rotation, adjacent pairs and interleaved axes
        dict(name="rope_partial_f32", op="rope", tokens=1001, hq=40, hkv=40, d=128, dtype="f32", axes=2, rotary=64,
             pairing="adjacent", order="interleaved", fused=True, bias=True, far=1000000),
        # a 7B-shaped step with accumulated weights
        dict(name="scored_7b", op="scored", b=8, t=1, hq=32, hkv=32, d=128, lmax=4096, lo=2047, hi=2047, dtype="f16",
             cache="f16", page=0, bias=True),
        # a 70B-shaped grouped-query step at a context of 8192
        dict(name="scored_70b", op="scored", b=16, t=1, hq=64, hkv=8, d=128, lmax=8192, lo=8191, hi=8191, dtype="bf16",
             cache="bf16", page=0, bias=False),
        # a ragged continuous batch on an INT8 cache in pages of 256
        dict(name="scored_int8_ragged", op="scored", b=64, t=1, hq=32, hkv=32, d=128, lmax=2048, lo=511, hi=2047,
             dtype="f16", cache="i8", page=256, bias=False),
        # one token too many in each 7B-shaped slot: eviction on every step
        dict(name="evict_one_7b", op="evict", b=8, hkv=32, d=128, lmax=4096, lo=2049, hi=2049, budget=2048, recent=512,
             sinks=4, cache="f16", page=0),
        # a 13B-shaped ragged batch cut to half of its longest contexts, some slots below the budget
        dict(name="evict_half_13b", op="evict", b=32, hkv=40, d=128, lmax=4096, lo=129, hi=4096, budget=2048,
             recent=1024, sinks=4, cache="bf16", page=0),
        # few kv heads, a long context in INT8 pages cut to an eighth
        dict(name="evict_long_int8", op="evict", b=4, hkv=8, d=128, lmax=65536, lo=65001, hi=65536, budget=8192,
             recent=2048, sinks=16, cache="i8", page=256),
        # one sequence's step over the 1500 states of a half-minute of speech
        dict(name="cross_speech_1", op="cross", b=1, t=1, hq=16, hkv=16, d=64, lmax=1504, lo=1500, hi=1500,
             dtype="f16", cache="f16", bias=True),
        # four beams of each of 16 ragged sources, which read the same states
        dict(name="cross_beams", op="cross", b=16, t=4, hq=32, hkv=32, d=128, lmax=2048, lo=33, hi=2047, dtype="bf16",
             cache="bf16", bias=True),
        # a 70B-shaped decoder over the states of long documents
        dict(name="cross_70b", op="cross", b=16, t=1, hq=64, hkv=8, d=128, lmax=8192, lo=8001, hi=8192, dtype="bf16",
             cache="bf16", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["rope", "scored", "evict", "cross"])
    d = rng.choice([64, 128, 128])
    if op == "rope":
        hq, hkv = rng.choice([(32, 32), (40, 40), (64, 8), (64, 1), (28, 4), (7, 1), (12, 3)])
        dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
        fused = rng.random() < 0.5
        most = 16381 * 80 * 128 * 2 // ((hq + 2 * hkv) * d * EB[dtype])
        rotary = rng.choice([d, d, d // 2, 2 * rng.randint(4, d // 2)])
        return dict(op=op, tokens=_log(rng, 1, min(most, 20000)), hq=hq, hkv=hkv, d=d, dtype=dtype,
                    axes=rng.choice([1, 2, 3, 3, 4]), rotary=rotary, pairing=rng.choice(["halves", "halves", "adjacent"]),
                    order=rng.choice(["sections", "interleaved"]), fused=fused, bias=rng.random() < 0.5,
                    far=_log(rng, 1000, 1000000))
    cache = rng.choice(["f32", "f16", "bf16", "bf16", "i8"])
    dtype = "f16" if cache == "i8" else cache
    budget_bytes = 16 * 8 * 8192 * 128 * 2
    if op == "evict":
        hkv = rng.choice([1, 4, 8, 32, 40])
        b = _log(rng, 1, 64)
        most = budget_bytes // (b * hkv * d * EB[cache])
        hi = _log(rng, min(200, most), min(most, 40000))
        lo = rng.randint(max(1, hi // 4), hi)
        budget = rng.randint(max(1, hi // 8), hi)
        sinks = min(rng.choice([0, 4, 16]), budget)
        recent = rng.randint(0, budget - sinks)
        return dict(op=op, b=b, hkv=hkv, d=d, lmax=-(-hi // 16) * 16, lo=lo, hi=hi, budget=budget, recent=recent,
                    sinks=sinks, cache=cache, page=rng.choice([0, 0, 128, 256]))
    hq, hkv = rng.choice([(32, 32), (40, 40), (64, 8), (64, 1), (28, 4), (12, 3), (16, 4)])
    b, t = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 4, 8])
    most = min(budget_bytes // (b * hkv * d * EB[cache]), 200000000 // (b * hq * t))
    hi = _log(rng, 20, min(most, 32000))
    lo = rng.randint(0 if op == "cross" else t - 1, hi) if rng.random() < 0.7 else hi
    c = dict(op=op, b=b, t=t, hq=hq, hkv=hkv, d=d, lmax=-(-(hi + t) // 16) * 16, lo=lo, hi=hi, dtype=dtype, cache=cache,
             bias=rng.random() < 0.5)
    if op == "scored":
        c["page"] = rng.choice([0, 0, 128, 256])
    return c


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _lens(c, g):
    """b lengths spread evenly over lo .. hi, shuffled: their sum is the case's alone."""
    n = torch.linspace(c["lo"], c["hi"], c["b"], dtype=torch.float64).round().to(torch.int32).cuda()
    return n[torch.randperm(c["b"], generator=g, device="cuda")].contiguous()


def _normal(g, shape, dtype):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(generator=g)


def _cache(c, g, shape):
    """K and V rows (INT8: codes, and their scales in two planes) of a cache."""
    if c["cache"] != "i8":
        return _normal(g, shape, DT[c["cache"]]), _normal(g, shape, DT[c["cache"]]), None
    k = torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g)
    v = torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g)
    s = torch.rand((2,) + tuple(shape[:-1]), device="cuda", generator=g) * 0.02 + 0.005
    return k, v, s


def _rope_sections(c):
    pairs, axes = c["rotary"] // 2, c["axes"]
    return [pairs * (a + 1) // axes - pairs * a // axes for a in range(axes)]


def _pair_axes(c):
    """Axis of each pair: whole sections one after the other, or round robin while a section lasts."""
    sec = _rope_sections(c)
    if c["order"] == "sections":
        return [a for a, n in enumerate(sec) for _ in range(n)]
    left, out = list(sec), []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _page_table(c, g, rows):
    """A shuffled page for every page_size positions of every slot, or None."""
    if not c.get("page"):
        return None
    per = -(-rows // c["page"])
    return torch.randperm(c["b"] * per, generator=g, device="cuda").to(torch.int32).view(c["b"], per)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    if c["op"] == "rope":
        n, hq, hkv, d, dt = c["tokens"], c["hq"], c["hkv"], c["d"], DT[c["dtype"]]
        if c["fused"]:
            qkv = _normal(g, (n, (hq + 2 * hkv) * d), dt)
            s["q"], s["k"], s["v"] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
        else:
            s["q"], s["k"], s["v"] = _normal(g, (n, hq * d), dt), _normal(g, (n, hkv * d), dt), None
        s["bias"] = _normal(g, ((hq + 2 * hkv) * d,), dt) * 0.1 if c["bias"] else None
        start = torch.randint(0, c["far"], (1,), device="cuda", generator=g)
        i = torch.arange(n, device="cuda")
        steps = [i // 299, (i // 23) % 13, i % 23, i % 7] if c["axes"] > 1 else [i]  # frames of 13 x 23 patches
        s["pos"] = (torch.stack(steps[:c["axes"]]) + start).to(torch.int32).contiguous()
        s["axis_of"] = torch.tensor(_pair_axes(c), device="cuda")
        s["out"] = [torch.empty((n, h * d), dtype=dt, device="cuda") for h in ((hq, hkv, hkv) if c["fused"] else (hq, hkv))]
        if own:
            import decode_step_masked_gb300 as ftd
            s["step"] = ftd.DecodeStep(1, hq, hkv, d, 16, c["dtype"], c["dtype"])
            s["step"].set_rope(c["axes"], _rope_sections(c), rotary_dim=c["rotary"], pairing=c["pairing"],
                               order=c["order"])
        return s
    b, hkv, d, lmax = c["b"], c["hkv"], c["d"], c["lmax"]
    s["lens"] = _lens(c, g)
    s["nmax"] = c["hi"]
    table = _page_table(c, g, lmax)
    shape = (b, hkv, lmax, d) if table is None else (table.numel(), hkv, c["page"], d)
    s["table"] = table
    s["k"], s["v"], s["scales"] = _cache(c, g, shape)
    if c["op"] != "cross":
        # weights gathered so far: a few heavy positions, many light ones
        s["acc"] = torch.exp(2.0 * torch.randn(shape[:-1], device="cuda", generator=g))
        s["acc_out"] = torch.zeros_like(s["acc"])
    paged = dict(page_size=c["page"], num_pages=table.numel()) if table is not None else {}
    if c["op"] == "evict":
        # rows hold positions out of order, as earlier evictions leave them; the newest are the last
        rows = torch.rand((b, hkv, lmax), device="cuda", generator=g)
        old = torch.arange(lmax, device="cuda") < (s["lens"] - c["recent"]).view(b, 1, 1)
        rows = torch.where(old, rows, 2.0 + torch.arange(lmax, device="cuda") / lmax)
        pos = torch.argsort(torch.argsort(rows, dim=-1), dim=-1).to(torch.int32)
        s["next_pos"] = s["lens"].clone()
        s["pos"] = pos.contiguous() if table is None else _to_pages(pos, table, c["page"])
        s["pos_out"] = torch.zeros_like(s["pos"])
        s["new_lens"] = torch.zeros_like(s["lens"])
        if own:
            import decode_step_masked_gb300 as ftd
            s["step"] = ftd.DecodeStep(b, hkv, hkv, d, lmax, "f16" if c["cache"] == "i8" else c["cache"], c["cache"],
                                       scored=True, **paged)
        return s
    t, hq, dt = c["t"], c["hq"], DT[c["dtype"]]
    s["q"] = _normal(g, (b, t, hq, d), dt)
    s["out"] = torch.empty((b, t, hq, d), dtype=dt, device="cuda")
    opts = dict(q_len=t, out_dtype=c["dtype"], **paged)
    if c["op"] == "scored":
        s["lens"].clamp_(max=lmax - t)
        s["k_new"], s["v_new"] = _normal(g, (b, t, hkv, d), dt), _normal(g, (b, t, hkv, d), dt)
        s["bias"] = _normal(g, ((hq + 2 * hkv) * d,), dt) * 0.1 if c["bias"] else None
        s["next_pos"] = s["lens"] + 5  # five tokens were evicted before
        s["pos"] = torch.zeros(shape[:-1], dtype=torch.int32, device="cuda")
        opts["scored"] = True
    else:
        s["bias"] = _normal(g, (hq * d,), dt) * 0.1 if c["bias"] else None
    if own:
        import decode_step_masked_gb300 as ftd
        s["step"] = ftd.DecodeStep(b, hq, hkv, d, lmax, c["dtype"], c["cache"], **opts)
    return s


# ------------------------------------------------------------ plain forms
def _to_pages(x, table, page):
    """[B][Hkv][L]... as pages [P][Hkv][page]..., positions past L zero."""
    b, hkv, n = x.shape[:3]
    per = table.shape[1]
    full = torch.zeros((b, hkv, per * page) + x.shape[3:], dtype=x.dtype, device=x.device)
    full[:, :, :n] = x
    out = torch.empty((table.numel(), hkv, page) + x.shape[3:], dtype=x.dtype, device=x.device)
    out[table.long().view(-1)] = full.view((b, hkv, per, page) + x.shape[3:]).transpose(1, 2).reshape(
        (b * per, hkv, page) + x.shape[3:])
    return out


def _rows(s, x, n):
    """The first n positions of a cache or plane as [B][Hkv][n]..."""
    if s["table"] is None:
        return x[:, :, :n]
    page = s["c"]["page"]
    per = -(-n // page)
    y = x[s["table"][:, :per].long()].transpose(1, 2)  # [B][Hkv][per][page]...
    return y.reshape(y.shape[:2] + (per * page,) + y.shape[4:])[:, :, :n]


def _put_rows(s, x, rows, seen):
    """Write rows [B][Hkv][n]... back to the first n positions where seen [B][n]."""
    c, n = s["c"], rows.shape[2]
    b, hkv = rows.shape[:2]
    bb = torch.arange(b, device="cuda").view(b, 1, 1).expand(b, hkv, n)
    hh = torch.arange(hkv, device="cuda").view(1, hkv, 1).expand(b, hkv, n)
    tt = torch.arange(n, device="cuda").view(1, 1, n).expand(b, hkv, n)
    m = seen.view(b, 1, n).expand(b, hkv, n)
    bb, hh, tt = bb[m], hh[m], tt[m]
    if s["table"] is None:
        x[bb, hh, tt] = rows[m]
    else:
        x[s["table"][bb, tt // c["page"]].long(), hh, tt % c["page"]] = rows[m]


def _rope_plain(s):
    c = s["c"]
    n, hq, hkv, d, r = c["tokens"], c["hq"], c["hkv"], c["d"], c["rotary"]
    # angles in 64 bits: far positions times small steps
    inv = torch.pow(10000.0, -torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    ang = s["pos"].double()[s["axis_of"]].T * inv  # [n][r / 2]
    cos, sin = torch.cos(ang).float().unsqueeze(1), torch.sin(ang).float().unsqueeze(1)

    def turn(x, first, heads):
        x = x.float()
        if s["bias"] is not None:
            x = x + s["bias"][first * d:(first + heads) * d].float()
        x = x.view(n, heads, d)
        if c["pairing"] == "halves":
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
        else:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., r:]], -1)
        return y.view(n, heads * d)

    s["out"][0].copy_(turn(s["q"], 0, hq))
    s["out"][1].copy_(turn(s["k"], hq, hkv))
    if s["v"] is not None:
        v = s["v"].float()
        s["out"][2].copy_(v if s["bias"] is None else v + s["bias"][(hq + hkv) * d:].float())
    return s["out"]


def _attend_plain(s, k, v, q, seen):
    """q [B][T][Hq][D] over rows [B][Hkv][n][D] (32 bits), seen [B][T][n]; a row that sees
    nothing gives zero.  Returns the output and the weights [B][Hkv][group][T][n]."""
    c = s["c"]
    b, t, hq, hkv, d, n = c["b"], c["t"], c["hq"], c["hkv"], c["d"], k.shape[2]
    q = q.float()
    if s["bias"] is not None:
        q = q + s["bias"][:hq * d].float().view(hq, d)
    q = q.view(b, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)  # rows: group, token
    sc = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    sc = sc.view(b, hkv, hq // hkv, t, n)
    m = seen.view(b, 1, 1, t, n)
    sc = sc.masked_fill(~m, float("-inf"))
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.view(b, hkv, -1, n), v).view(b, hkv, hq // hkv, t, d)
    return o.permute(0, 3, 1, 2, 4).reshape(b, t, hq, d), p


def _wide(x, scales):
    return x.float() if scales is None else x.float() * scales.unsqueeze(-1)


def _scored_plain(s):
    c = s["c"]
    b, t, hq, hkv, d = c["b"], c["t"], c["hq"], c["hkv"], c["d"]
    n = min(s["nmax"] + t, c["lmax"])
    at = torch.arange(n, device="cuda")
    L = s["lens"].view(b, 1)
    new = (at >= L) & (at < L + t)  # [B][n]
    tok = (at - L).clamp(0, t - 1)
    for name, cache, plane in (("k", s["k"], 0), ("v", s["v"], 1)):
        x = s[name + "_new"].float()
        if s["bias"] is not None:
            o = (hq + plane * hkv) * d
            x = x + s["bias"][o:o + hkv * d].float().view(hkv, d)
        if s["scales"] is not None:
            top = x.abs().amax(-1)
            sc = torch.where(top == 0, torch.ones_like(top), top / 127.0)
            _put_rows(s, s["scales"][plane], _spread(sc, tok), new)
            x = torch.round(x / sc.unsqueeze(-1)).clamp(-127, 127)
        _put_rows(s, cache, _spread(x, tok).to(cache.dtype), new)
    _put_rows(s, s["pos"], (s["next_pos"].view(b, 1) + tok).to(torch.int32).view(b, 1, n).expand(b, hkv, n), new)
    ks, vs = (None, None) if s["scales"] is None else (_rows(s, s["scales"][0], n), _rows(s, s["scales"][1], n))
    seen = at.view(1, 1, n) <= (L.view(b, 1, 1) + torch.arange(t, device="cuda").view(1, t, 1))
    live = (at < L + t).view(b, 1, n, 1)
    k = torch.where(live, _wide(_rows(s, s["k"], n), ks), 0.0)
    v = torch.where(live, _wide(_rows(s, s["v"], n), vs), 0.0)
    o, p = _attend_plain(s, k, v, s["q"], seen)
    s["out"].copy_(o)
    acc = torch.where((at < L).view(b, 1, n), _rows(s, s["acc"], n), 0.0) + p.sum((2, 3))
    _put_rows(s, s["acc_out"], acc, at < L + t)
    return s


def _spread(x, tok):
    """The new tokens' rows [B][T][Hkv]... at the positions of tok [B][n]: [B][Hkv][n]..."""
    b, n = tok.shape
    return x[torch.arange(b, device="cuda").view(b, 1), tok].transpose(1, 2)


def _evict_plain(s):
    c = s["c"]
    b, hkv, n, keep = c["b"], c["hkv"], s["nmax"], c["budget"]
    at = torch.arange(n, device="cuda")
    L = s["lens"].view(b, 1, 1)
    acc, pos = _rows(s, s["acc"], n), _rows(s, s["pos"], n)
    safe = (pos < c["sinks"]) | (pos >= s["next_pos"].view(b, 1, 1) - c["recent"])
    key = torch.where(safe, torch.full_like(acc, float("inf")), acc)
    key = torch.where(at < L, key, torch.full_like(acc, float("-inf")))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order).contiguous())
    kept = (rank < keep) & (at < L)
    m = min(keep, n)
    # the j-th kept row behind the budget goes to the j-th hole before it
    behind = kept & (at >= keep)
    which = torch.cumsum(behind, -1) - 1
    movers = torch.zeros((b, hkv, n + 1), dtype=torch.int64, device="cuda")
    movers.scatter_(-1, torch.where(behind, which, n), at.expand(b, hkv, n).contiguous())
    hole = ~kept[..., :m] & (at[:m] < L)
    src = torch.where(hole, movers.gather(-1, (torch.cumsum(hole, -1) - 1).clamp(min=0)), at[:m])
    s["new_lens"].copy_(s["lens"].clamp(max=keep))
    live = at[:m] < s["new_lens"].view(b, 1)
    for x, out in ((s["k"], s["k"]), (s["v"], s["v"])):
        _put_rows(s, out, _rows(s, x, n).gather(2, src.unsqueeze(-1).expand(b, hkv, m, c["d"])), live)
    planes = [(s["acc"], s["acc_out"]), (s["pos"], s["pos_out"])]
    if s["scales"] is not None:
        planes += [(s["scales"][0], s["scales"][0]), (s["scales"][1], s["scales"][1])]
    for x, out in planes:
        _put_rows(s, out, _rows(s, x, n).gather(2, src), live)


def _cross_plain(s):
    c = s["c"]
    b, t, n = c["b"], c["t"], s["nmax"]
    ks, vs = (None, None) if s["scales"] is None else (s["scales"][0][:, :, :n], s["scales"][1][:, :, :n])
    seen = torch.arange(n, device="cuda").view(1, 1, n) < s["lens"].view(b, 1, 1)
    o, _ = _attend_plain(s, _wide(s["k"][:, :, :n], ks), _wide(s["v"][:, :, :n], vs), s["q"], seen.expand(b, t, n))
    s["out"].copy_(o)


def run(state):
    s, op = state, state["c"]["op"]
    if op == "rope":
        if own:
            s["step"].rope(s["q"], s["k"], s["v"], s["pos"], *s["out"], bias=s["bias"])
            return s["out"]
        return _rope_plain(s)
    if op == "scored":
        if own:
            s["step"].scored(s["q"], s["k_new"], s["v_new"], s["lens"], s["next_pos"], s["acc"], s["pos"], s["out"],
                             acc_out=s["acc_out"], bias=s["bias"], k_cache=s["k"], v_cache=s["v"], scales=s["scales"],
                             block_table=s["table"])
        else:
            _scored_plain(s)
        return [s[x] for x in ("out", "acc_out", "pos", "k", "v", "scales") if s[x] is not None]
    if op == "evict":
        if own:
            c = s["c"]
            s["step"].evict(s["acc"], s["pos"], s["lens"], s["next_pos"], s["new_lens"], c["budget"], recent=c["recent"],
                            sinks=c["sinks"], acc_out=s["acc_out"], positions_out=s["pos_out"], k_cache=s["k"],
                            v_cache=s["v"], scales=s["scales"], block_table=s["table"])
        else:
            _evict_plain(s)
        return [s[x] for x in ("new_lens", "acc_out", "pos_out", "k", "v", "scales") if s[x] is not None]
    if own:
        s["step"].cross(s["q"], s["lens"], s["out"], q_bias=s["bias"], k_mem=s["k"], v_mem=s["v"], scales=s["scales"])
    else:
        _cross_plain(s)
    return s["out"]


# ------------------------------------------------------------------- work
def work(case):
    c = case
    d = c["d"]
    if c["op"] == "rope":
        heads = c["hq"] + c["hkv"] * (2 if c["fused"] else 1)
        n = c["tokens"]
        bias = (c["hq"] + 2 * c["hkv"]) * d * EB[c["dtype"]] if c["bias"] else 0
        return {"bytes": 2 * n * heads * d * EB[c["dtype"]] + n * c["axes"] * 4 + bias,
                "flops": n * (c["hq"] + c["hkv"]) * c["rotary"] // 2 * 6 + (n * heads * d if c["bias"] else 0)}
    lens = [round(x) for x in torch.linspace(c["lo"], c["hi"], c["b"], dtype=torch.float64).tolist()]
    row = 2 * d * EB[c["cache"]] + (8 if c["cache"] == "i8" else 0)  # a position's K and V (and scales) in one kv head
    if c["op"] == "evict":
        nbytes = 0.0
        for n in lens:
            keep = min(n, c["budget"])
            behind = max(0, n - c["budget"])
            fresh = min(behind, c["recent"])  # the newest rows are the last ones
            loose = n - c["recent"] - c["sinks"]
            share = max(0, keep - c["recent"] - c["sinks"]) / loose if loose > 0 else 0.0
            moved = min(keep, fresh + (behind - fresh) * share)
            # every weight and position of a slot over the budget is read, the kept ones are written, moved rows are read and written
            nbytes += c["hkv"] * (8 * (n if behind else keep) + 8 * keep + 2 * moved * row)
        return {"bytes": nbytes, "flops": float(c["hkv"] * sum(lens))}
    t, rows = c["t"], c["hq"] * c["t"]
    io = c["b"] * 2 * rows * d * EB[c["dtype"]]
    if c["op"] == "cross":
        return {"bytes": c["hkv"] * sum(lens) * row + io, "flops": 4.0 * rows * d * sum(lens)}
    new = c["b"] * t * c["hkv"] * (2 * d * EB[c["dtype"]] + row)
    return {"bytes": c["hkv"] * sum(lens) * (row + 8) + io + new,
            "flops": 4.0 * rows * d * sum(n + t for n in lens)}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits, one slot at a time; eviction computes no numbers."""
    c = case
    if c["op"] == "evict":
        return None
    s = prepare(case, seed)
    d = c["d"]
    if c["op"] == "rope":
        r, n = c["rotary"], c["tokens"]
        axis = _pair_axes(c)
        outs = []
        first = 0
        for x, heads, turns in ((s["q"], c["hq"], True), (s["k"], c["hkv"], True), (s["v"], c["hkv"], False)):
            if x is not None:
                y = x.double().clone()
                if s["bias"] is not None:
                    y += s["bias"].double()[first:first + heads * d]
                y = y.view(n, heads, d)
                if turns:
                    z = y.clone()
                    for i in range(r // 2):
                        a, b = (i, i + r // 2) if c["pairing"] == "halves" else (2 * i, 2 * i + 1)
                        w = s["pos"][axis[i]].double() * 10000.0 ** (-2.0 * i / r)
                        co, si = torch.cos(w).view(n, 1), torch.sin(w).view(n, 1)
                        z[..., a] = y[..., a] * co - y[..., b] * si
                        z[..., b] = y[..., a] * si + y[..., b] * co
                    y = z
                outs.append(y.view(n, heads * d))
            first += heads * d
        return outs
    b, t, hq, hkv = c["b"], c["t"], c["hq"], c["hkv"]
    grp = hq // hkv
    scored = c["op"] == "scored"
    out = torch.zeros((b, t, hq, d), dtype=torch.float64, device="cuda")
    acc_out = s["acc_out"].double() if scored else None
    bias = s["bias"].double() if s["bias"] is not None else torch.zeros(((hq + 2 * hkv) * d,), dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for i in range(b):
        n = lens[i]
        if s["table"] is None:
            k, v = s["k"][i, :, :n].double(), s["v"][i, :, :n].double()
            sc = s["scales"][:, i, :, :n].double() if s["scales"] is not None else None
        else:
            pg = s["table"][i].long()
            k, v = (x[pg].transpose(0, 1).reshape(hkv, -1, d)[:, :n].double() for x in (s["k"], s["v"]))
            sc = s["scales"][:, pg].transpose(1, 2).reshape(2, hkv, -1)[:, :, :n].double() if s["scales"] is not None else None
        if sc is not None:
            k, v = k * sc[0].unsqueeze(-1), v * sc[1].unsqueeze(-1)
        if scored:
            # the appended rows as the cache holds them: the bias is added and the sum rounded in 32 bits
            for name, o in (("k", hq), ("v", hq + hkv)):
                x = (s[name + "_new"][i].float() + bias.float()[o * d:(o + hkv) * d].view(hkv, d)).transpose(0, 1)
                if sc is not None:
                    top = x.abs().amax(-1, keepdim=True)
                    step = torch.where(top == 0, torch.ones_like(top), top / 127.0)
                    x = torch.round(x / step).clamp(-127, 127).double() * step.double()
                else:
                    x = x.to(s["k"].dtype).double()
                if name == "k":
                    k = torch.cat([k, x], 1)
                else:
                    v = torch.cat([v, x], 1)
        elif n == 0:
            continue
        q = s["q"][i].double() + bias[:hq * d].view(hq, d)  # [T][Hq][D]
        for j in range(t):
            m = n + j + 1 if scored else n
            w = torch.einsum("hgd,hnd->hgn", q[j].view(hkv, grp, d), k[:, :m]) / math.sqrt(d)
            w = torch.softmax(w, -1)
            out[i, j] = torch.einsum("hgn,hnd->hgd", w, v[:, :m]).reshape(hq, d)
            if scored:
                add = torch.zeros((hkv, n + t), dtype=torch.float64, device="cuda")
                add[:, :m] = w.sum(1)
                if j == 0:
                    total = add
                else:
                    total = total + add
        if scored:
            at = torch.arange(n + t, device="cuda")
            if s["table"] is None:
                total[:, :n] += s["acc"][i, :, :n].double()
                acc_out[i, :, :n + t] = total
            else:
                pg, off = s["table"][i].long()[at // c["page"]], at % c["page"]
                total[:, :n] += s["acc"][pg, :, off].T[:, :n].double()
                acc_out[pg, :, off] = total.T
    if not scored:
        return out
    return [out, acc_out] + [None] * (3 + (s["scales"] is not None))
