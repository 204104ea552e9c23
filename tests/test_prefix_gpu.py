"""ftd_decode_mha_prefix against attention over prefix and own rows in 64 bits: every cache type and kernel, grouped heads,
several new tokens, prefixes from no row to thousands, slots that see all, part or none of it, inactive and overflowing
slots, pages, everything that no slot sees poisoned, graphs, streams, and the refusals."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from tests import operators_ref as ref
from tests.gpu_util import TORCH_OUT, assert_same_bytes, dev, from_pages, host, make_step, page_layout, to_pages, valid_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


def case(cache, qkv, B, Hq, Hkv, D, Lmax, lens, P, seen, T=1, seed=61, bias=0.1, heavy=0.0):
    """Inputs of the step, and a prefix of P rows whose rows from the longest that is seen on are poison.  heavy: the
    prefix's keys grow along it, so that running references move again and again."""
    w, inp = ref.step_case(cache, qkv, B, Hq, Hkv, D, Lmax, lens, T=T, seed=seed, bias=bias)
    live = [s for s, L in zip(seen, lens) if 0 <= L <= Lmax - T]
    most = min(max(live + [0]), P)
    pw = w.with_(B=1, Lmax=-(-max(P, 1) // 16) * 16, q_len=1)
    from synthetic import gen_all, to_storage
    pre = gen_all(pw, seed=seed + 1, seq_lens=np.array([most], np.int32), fill_beyond="nan")
    k = pre["k_cache"][0, :, :P]
    if heavy and cache == "i8":
        pre["scales"][0] *= (1.0 + heavy * np.arange(pre["scales"].shape[-1]) / P).astype(np.float32)
    elif heavy:
        x = ref.widen(k, cache) * (1.0 + heavy * np.arange(P) / P)[None, :, None]
        k = np.where(np.isnan(x), k, to_storage(x.astype(np.float32), cache)) if cache != "bf16" else \
            np.where(np.isnan(x), k, to_storage(np.nan_to_num(x).astype(np.float32), cache))
    inp["k_prefix"], inp["v_prefix"] = np.ascontiguousarray(k), np.ascontiguousarray(pre["v_cache"][0, :, :P])
    if pre.get("scales") is not None:
        inp["prefix_scales"] = np.ascontiguousarray(pre["scales"][:, 0, :, :P])
    inp["prefix_lens"] = np.array(seen, np.int32)
    return w, inp


PAIR = {"f32": 2.0 ** -22, "f16": 2.0 ** -21, "bf16": 2.0 ** -16, "i8": 2.0 ** -16}


def expect(w, inp, k_after, v_after, scales_after, single):
    """Outputs [B][T][Hq][D] in 64 bits and the bound of the kernels' error of each.

    A score is a dot product of D products in fp32 (accumulated in any order: D + 8 half steps of the sum of
    magnitudes); q as a pair of 16-bit numbers keeps 2^-16 of it with bf16, 2^-21 with f16, two INT8 levels of a row
    2^-15 of its largest magnitude.  A weight's relative error is its score's error, once more for the sum it is
    divided by, and its own rounding: a half step of the 16-bit type where it is kept as one number, else the
    pair's.  The sum over n rows adds n + 32 half steps; f16 weights below its normal range are off by 2^-25 of
    the largest weight each."""
    out, tol = np.zeros((w.B, w.q_len, w.Hq, w.D)), np.zeros((w.B, w.q_len, w.Hq, w.D))
    g, P = w.Hq // w.Hkv, inp["k_prefix"].shape[1]
    ps = inp.get("prefix_scales")
    i8 = w.cache_dtype == "i8"
    rp = ref.HALF_STEP.get(w.cache_dtype, 2.0 ** -8) if single else PAIR[w.cache_dtype]
    for b in range(w.B):
        L = int(inp["seq_lens"][b])
        if not 0 <= L <= w.Lmax - w.q_len:
            continue
        n = max(0, min(int(inp["prefix_lens"][b]), P))
        rows = []
        for pre, after, plane in ((inp["k_prefix"], k_after, 0), (inp["v_prefix"], v_after, 1)):
            x = ref.widen(pre[:, :n], w.cache_dtype)
            if i8:
                x = x * ps[plane, :, :n, None].astype(np.float64)
            rows.append(np.concatenate([x, ref.cache_rows(w, after, scales_after, plane, b, L + w.q_len)], axis=1))
        q = ref.queries(w, inp, b)
        k, v = (np.repeat(x, g, axis=0) for x in rows)
        for j in range(w.q_len):
            m = n + L + j + 1
            s = np.einsum("hd,hnd->hn", q[j], k[:, :m]) / np.sqrt(w.D)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            mass = np.einsum("hd,hnd->hn", np.abs(q[j]), np.abs(k[:, :m])).max(1) / np.sqrt(w.D)
            if i8:
                mass8 = np.abs(q[j]).max(1) * np.abs(k[:, :m]).sum(2).max(1) / np.sqrt(w.D)
            e = mass * ((w.D + 8) * 2.0 ** -24 + PAIR[w.cache_dtype]) + (mass8 * 2.0 ** -15 if i8 else 0.0)
            out[b, j] = np.einsum("hn,hnd->hd", p, v[:, :m])
            av = np.einsum("hn,hnd->hd", p, np.abs(v[:, :m]))
            tol[b, j] = av * (2 * e + rp + (m + 32) * 2.0 ** -24)[:, None] + m * 2.0 ** -25 * np.abs(v[:, :m]).max(1)
    return out, tol


def run(w, inp, out_dtype="f32", page=0, cuda_core=False, bias=True, step=None, status=ftd.FTD_OK, calls=1, values=True):
    import torch
    T, lens, P = w.q_len, inp["seq_lens"], inp["k_prefix"].shape[1]
    arrs = {"k": inp["k_cache"], "v": inp["v_cache"]}
    sc, psc = inp.get("scales"), inp.get("prefix_scales")
    opts, kw, table = {}, {}, None
    if page:
        table, own_pages, _ = page_layout(w, lens, page, 2, seed=7, q_len=T)
        first = -(-P // page)
        opts = dict(page_size=page, num_pages=own_pages + first)
        where = own_pages + np.random.default_rng(3).permutation(first)
        pages = {}
        for x in ("k", "v"):
            a = np.zeros((own_pages + first, w.Hkv, page, w.D), arrs[x].dtype)
            a[:own_pages] = to_pages(w, arrs[x], table, own_pages, page, 0)
            a[own_pages:] = inp["k_cache"].dtype.type(0)
            for i in range(first):
                n = min(page, P - i * page)
                a[where[i], :, :n] = inp[x + "_prefix"][:, i * page:i * page + n]
            pages[x] = a
        arrs = pages
        if sc is not None:
            s = np.ones((2, own_pages + first, w.Hkv, page), np.float32)
            for pl in range(2):
                s[pl, :own_pages] = to_pages(w, sc[pl], table, own_pages, page, 1.0)
                for i in range(first):
                    n = min(page, P - i * page)
                    s[pl, where[i], :, :n] = psc[pl, :, i * page:i * page + n]
            sc = s
        kw = dict(block_table=dev(table), prefix_table=dev(where.astype(np.int32)))
    else:
        kw = dict(k_prefix=dev(inp["k_prefix"]), v_prefix=dev(inp["v_prefix"]), prefix_scales=dev(psc) if psc is not None else None)
    own = step is None
    if own:
        step = make_step(w, force_cuda_core=cuda_core, out_dtype=out_dtype, q_len=T, **opts)
        step.enable_prefix()
    q, kn, vn, sl, pl = (dev(inp[x]) for x in ("q", "k_new", "v_new", "seq_lens", "prefix_lens"))
    kc, vc = dev(arrs["k"]), dev(arrs["v"])
    t_sc = dev(sc) if sc is not None else None
    use = bias and inp.get("bias") is not None
    out = torch.full((w.B, T, w.Hq, w.D), float("nan"), dtype=getattr(torch, TORCH_OUT[out_dtype]), device="cuda")
    before = ftd.ftd_kernel_launches()
    for _ in range(calls):
        step.prefix(q, kn, vn, sl, pl, out, bias=dev(inp["bias"]) if use else None, k_cache=kc, v_cache=vc, scales=t_sc, **kw)
    torch.cuda.synchronize()
    assert ftd.ftd_kernel_launches() in (before + 2 * calls, before + 3 * calls)
    assert step.get_error() == status
    if not values:
        return
    got = out.double().cpu().numpy()
    ka, va = host(kc, arrs["k"]), host(vc, arrs["v"])
    sa = None if t_sc is None else t_sc.cpu().numpy()
    if page:
        ka, va = (from_pages(w, a[:own_pages], table, page, lens, T) for a in (ka, va))
        if sa is not None:
            sa = np.stack([from_pages(w, sa[i][:own_pages], table, page, lens, T) for i in range(2)])
    if own:
        step.close()
    inp = inp if use else dict(inp, bias=None)
    # weights of one 16-bit number (INT8's are of bf16: two for fp16 out)
    single = out_dtype != "f32" and not cuda_core and w.cache_dtype != "f32" and (w.cache_dtype, out_dtype) != ("i8", "f16")
    want, tol = expect(w, inp, ka, va, sa, single)
    if out_dtype != "f32":
        tol = tol + np.abs(want) * ref.HALF_STEP[out_dtype] * (1 + 2.0 ** -7) + (2.0 ** -25 if out_dtype == "f16" else 0.0)
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    worst = float((err / np.maximum(tol, 1e-30)).max())
    assert np.all(err <= tol), worst
    return got, (ka, va, sa)


SHAPES = {
    "mha_f32": ("f32", "f32", 4, 4, 128, False),
    "mha_f32_d64": ("f32", "f32", 6, 2, 64, False),
    "mha_bf16": ("bf16", "bf16", 4, 4, 128, False),
    "mha_f16_d64": ("f16", "f16", 4, 4, 64, False),
    "gqa8_bf16": ("bf16", "bf16", 16, 2, 128, False),
    "gqa8_f16": ("f16", "f16", 16, 2, 128, False),
    "gqa7_d64": ("bf16", "bf16", 7, 1, 64, False),
    "gqa3_cc": ("f16", "f16", 6, 2, 128, True),
    "gqa8_cc_bf16_d64": ("bf16", "bf16", 8, 1, 64, True),
    "mqa64": ("bf16", "bf16", 64, 1, 128, False),
    "mqa32_f16": ("f16", "f16", 32, 1, 128, False),
    "f32_on_bf16": ("bf16", "f32", 8, 2, 128, False),
    "bf16_on_f16": ("f16", "bf16", 8, 2, 64, False),
    "mha_i8": ("i8", "f16", 4, 4, 128, False),
    "gqa8_i8": ("i8", "bf16", 16, 2, 128, False),
    "gqa4_i8_d64": ("i8", "f16", 8, 2, 64, False),
    "gqa8_cc_i8": ("i8", "f16", 16, 2, 128, True),
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("page", [0, 128])
def test_shapes(shape, page):
    """A ragged batch behind one prefix, in fp32 out with a bias and in 16 bits without."""
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    lens, seen = [0, 5, 130, -1, 61, 200], [300, 300, 300, 300, 0, 177]
    w, inp = case(cache, qkv, 6, Hq, Hkv, D, 256, lens, 300, seen)
    run(w, inp, page=page, cuda_core=cc)
    run(w, inp, out_dtype="f32" if qkv == "f32" else qkv, page=page, cuda_core=cc, bias=False)


@pytest.mark.parametrize("P", [1, 2, 15, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 4097])
@pytest.mark.parametrize("cache,D", [("f32", 128), ("bf16", 128), ("f16", 64), ("i8", 128)])
def test_prefix_lengths(P, cache, D):
    qkv = "f16" if cache == "i8" else cache
    w, inp = case(cache, qkv, 3, 8, 2, D, 64, [0, 17, 40], P, [P, P, P // 2], seed=P)
    run(w, inp)
    run(w, inp, out_dtype=qkv, bias=False)


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 8, 1), (2, 3, 5, 1), (33, 1, 2, 2), (16, 1, 8, 1), (9, 1, 16, 1), (43, 1, 6, 2),
                                        (65, 2, 2, 1), (64, 1, 8, 2), (257, 1, 1, 1), (40, 4, 8, 1), (1024, 1, 2, 1)])
@pytest.mark.parametrize("cache,D", [("f32", 64), ("bf16", 128), ("f16", 64), ("i8", 64)])
def test_query_rows(B, T, Hq, Hkv, cache, D):
    """Blocks of query rows that are full, ragged, held twice, and many."""
    qkv = "bf16" if cache == "i8" else cache
    rng = np.random.default_rng(B + T)
    lens = rng.integers(0, 29, B)
    w, inp = case(cache, qkv, B, Hq, Hkv, D, 32, lens, 333, rng.choice([333, 333, 333, 120, 0], B), T=T, seed=B)
    run(w, inp)
    run(w, inp, out_dtype=qkv, bias=False)


@pytest.mark.parametrize("cache", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("seen", ["none", "first", "last", "one", "each", "negative"])
def test_who_sees_what(cache, seen):
    B, P = 40, 700
    s = dict(none=[0] * B, first=[P] + [0] * (B - 1), last=[0] * (B - 1) + [P], one=[1] * B, each=[P * i // (B - 1) for i in range(B)],
             negative=[-5 if i % 2 else P for i in range(B)])[seen]
    w, inp = case(cache, "f16" if cache == "i8" else cache, B, 16, 2, 128, 32, [i % 30 for i in range(B)], P, s)
    run(w, inp)


@pytest.mark.parametrize("cache,out", [("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"), ("bf16", "f32"), ("i8", "f16"), ("i8", "f32")])
@pytest.mark.parametrize("heavy", [4.0, 30.0])
def test_rising_scores(cache, out, heavy):
    """Keys that grow along the prefix: the running maxima move far, and more than once."""
    w, inp = case(cache, "f16" if cache == "i8" else cache, 5, 16, 2, 128, 32, [0, 3, 9, 20, 31], 1500, [1500, 1500, 800, 0, 1500], heavy=heavy)
    run(w, inp, out_dtype=out, bias=out == "f32")


@pytest.mark.parametrize("cache", ["f32", "f16", "i8"])
def test_slots_without_work(cache):
    """Inactive and overflowing slots: zeros, and the longest prefix among them poisons nothing."""
    w, inp = case(cache, "f16" if cache == "i8" else cache, 5, 8, 2, 64, 48, [-1, 48, 5, 47, 100], 400, [400, 400, 200, 100, 400])
    got, _ = run(w, inp, status=ftd.FTD_ERR_SEQ_OVERFLOW)
    assert not got[[0, 1, 4]].any() and got[[2, 3]].any()


@pytest.mark.parametrize("cache,qkv,out,D,bias", [("i8", "f16", "f16", 128, None), ("i8", "bf16", "bf16", 64, 0.1), ("i8", "f16", "f32", 128, 0.1),
                                                  ("i8", "bf16", "f32", 64, None), ("f16", "f16", "f16", 128, None), ("bf16", "bf16", "f32", 128, 0.1),
                                                  ("f32", "f32", "f32", 64, None)])
@pytest.mark.parametrize("B", [3, 40])
def test_many_tiles_a_block(cache, qkv, out, D, bias, B):
    """Every block goes through its buffers many times, over pieces of several kv heads: few rows (each tile is one stream's)
    and, with more heads of a kv head, two row blocks."""
    g, P = (1, 4110) if B == 3 else (5, 4110)
    hkv = 40 if B == 3 else 12
    w, inp = case(cache, qkv, B, hkv * g, hkv, D, 32, [b % 30 for b in range(B)], P, [P - 7 * b for b in range(B)], bias=bias)
    run(w, inp, out_dtype=out, bias=bias is not None)


def test_prefix_lens_too_long():
    w, inp = case("bf16", "bf16", 3, 8, 2, 128, 48, [1, 2, 3], 200, [200, 201, 1 << 30])
    run(w, inp, status=ftd.FTD_ERR_SEQ_OVERFLOW)


def test_same_result_every_time():
    """No atomics decide an output: calls on the same inputs give the same bits, and appended rows are the step's."""
    import torch
    w, inp = case("bf16", "bf16", 20, 16, 2, 128, 64, list(range(20)), 900, [900] * 20)
    a, (ka, va, _) = run(w, inp, calls=3)
    b, (kb, vb, _) = run(w, inp)
    assert np.array_equal(a, b)
    step = make_step(w)
    kc, vc = dev(inp["k_cache"]), dev(inp["v_cache"])
    out = torch.empty((w.B, 1, w.Hq, w.D), device="cuda")
    step(dev(inp["q"]), dev(inp["k_new"]), dev(inp["v_new"]), dev(inp["seq_lens"]), out, bias=dev(inp["bias"]), k_cache=kc, v_cache=vc)
    torch.cuda.synchronize()
    assert_same_bytes(host(kc, ka), ka, "K")
    assert_same_bytes(host(vc, va), va, "V")
    step.close()


@pytest.mark.parametrize("cache", ["f32", "bf16"])
def test_lengths_that_change_between_calls(cache):
    """One context's calls on lengths that cross tiles: no part of an earlier call is joined."""
    step = None
    for lens in ([0, 1, 127, 128, 140, 300], [1, 2, 128, 129, 141, 301], [300, 0, 0, 511, 5, 129], [-1, 511, 256, 255, 257, 1], [64] * 6):
        w, inp = case(cache, cache, 6, 8, 2, 64, 512, lens, 200, [200, 150, 200, 0, 200, 129], seed=sum(lens))
        if step is None:
            step = make_step(w)
            step.enable_prefix()
        run(w, inp, step=step)
    step.close()


@pytest.mark.parametrize("cache", ["f32", "bf16"])
def test_empty_prefix(cache):
    """No rows, or rows that nobody sees: the step's own result."""
    import torch
    w, inp = case(cache, cache, 4, 8, 2, 128, 64, [0, 5, 30, 63], 100, [0] * 4)
    step = make_step(w)
    step.enable_prefix()
    args = [dev(inp[x]) for x in ("q", "k_new", "v_new", "seq_lens")]
    kc, vc, bias = dev(inp["k_cache"]), dev(inp["v_cache"]), dev(inp["bias"])
    outs = [torch.full((w.B, 1, w.Hq, w.D), float("nan"), device="cuda") for _ in range(3)]
    kw = dict(bias=bias, k_cache=kc, v_cache=vc)
    step(*args, outs[0], **kw)
    n = ftd.ftd_kernel_launches()
    step.prefix(*args, dev(inp["prefix_lens"]), outs[1], **kw)
    assert ftd.ftd_kernel_launches() == n + 1
    step.prefix(*args, dev(inp["prefix_lens"]), outs[2], k_prefix=dev(inp["k_prefix"]), v_prefix=dev(inp["v_prefix"]), **kw)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    # beside a prefix the own rows' tiles are cut differently, so their sums are taken in another order than the
    # step's: within the bounds of any call
    run(w, inp)
    assert step.get_error() == ftd.FTD_OK
    step.close()


def test_graphs_and_streams():
    """Captured with changing lengths, two graphs of one context in turn, an eager call on another stream between."""
    import torch
    w, inp = case("bf16", "bf16", 8, 16, 2, 128, 64, [3] * 8, 500, [500] * 8, bias=None)
    step = make_step(w, out_dtype="bf16")
    step.enable_prefix()
    q, kn, vn = (dev(inp[x]) for x in ("q", "k_new", "v_new"))
    kc, vc = dev(np.nan_to_num(inp["k_cache"])), dev(np.nan_to_num(inp["v_cache"]))
    kp, vp = dev(inp["k_prefix"]), dev(inp["v_prefix"])
    lens, seen = dev(inp["seq_lens"]), dev(inp["prefix_lens"])
    outs = [torch.zeros((8, 1, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    side, graphs = torch.cuda.Stream(), []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step.prefix(q, kn, vn, lens, seen, outs[k], k_prefix=kp, v_prefix=vp, k_cache=kc, v_cache=vc)
            lens.add_(1)
        graphs.append(g)
    rng = np.random.default_rng(5)
    for i in range(12):
        seen.copy_(dev(rng.choice([500, 300, 0], 8).astype(np.int32)))
        at = lens.clone()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step.prefix(q, kn, vn, at, seen, outs[2], k_prefix=kp, v_prefix=vp, k_cache=kc, v_cache=vc)
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], outs[2])
    assert int(lens[0]) == 15 and step.get_error() == ftd.FTD_OK
    step.close()


def test_bad_prefix_page():
    """A page outside the pool: the error, and a result from within the pool's memory."""
    import torch
    for cache in ("f32", "bf16", "i8"):
        step = ftd.DecodeStep(2, 8, 2, 128, 256, "bf16", cache, page_size=128, num_pages=6)
        step.enable_prefix()
        z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        out = torch.full((2, 8, 128), float("nan"), device="cuda")
        for bad in (6, -1, 1 << 30):
            step.prefix(z(2, 8, 128), z(2, 2, 128), z(2, 2, 128), dev(np.array([3, 130], np.int32)), dev(np.array([300, 300], np.int32)),
                        out, block_table=dev(np.array([[0, -1], [1, 2]], np.int32)), prefix_table=dev(np.array([3, bad, 5], np.int32)))
            torch.cuda.synchronize()
            assert step.get_error() == ftd.FTD_ERR_BAD_PAGE
        step.close()


def test_refusals():
    import torch
    h = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    flat, paged = ftd.DecodeStep(2, 4, 2, 64, 32, "f16", "f16"), ftd.DecodeStep(2, 4, 2, 64, 256, "f16", "f16", page_size=128, num_pages=4)
    ok = dict(q=h(2, 4, 64), k_new=h(2, 2, 64), v_new=h(2, 2, 64), seq_lens=i(2), prefix_lens=i(2), out=torch.zeros((2, 4, 64), device="cuda"))
    n = ftd.ftd_kernel_launches()
    with pytest.raises(ftd.FtdError, match="enable_prefix"):
        flat.prefix(**ok)
    windowed = ftd.DecodeStep(2, 4, 2, 64, 32, "f16", "f16", window=8)
    with pytest.raises(ftd.FtdError, match="window"):
        windowed.enable_prefix()
    many = ftd.DecodeStep(1024, 64, 1, 64, 16, "f16", "f16", q_len=2)
    with pytest.raises(ftd.FtdError, match="query rows"):
        many.enable_prefix()
    for s in (flat, paged):
        s.enable_prefix()
        s.enable_prefix()
    k, v = h(2, 70, 64), h(2, 70, 64)
    for kw in (dict(k_prefix=k), dict(k_prefix=k, v_prefix=h(2, 71, 64)), dict(k_prefix=k, v_prefix=v, prefix_table=i(1)),
               dict(k_prefix=k.float(), v_prefix=v.float()), dict(k_prefix=k, v_prefix=v, seq_lens=i(2).long()),
               dict(k_prefix=k, v_prefix=v, prefix_lens=i(1)), dict(k_prefix=k, v_prefix=v, block_table=i(2, 2)),
               dict(k_prefix=h(2, 71, 64).view(-1)[4:4 + 2 * 70 * 64].view(2, 70, 64), v_prefix=v),
               dict(k_prefix=k.transpose(0, 1), v_prefix=v.transpose(0, 1))):
        with pytest.raises((ftd.FtdError, ValueError)):
            flat.prefix(**dict(ok, **kw))
    for kw in (dict(), dict(block_table=i(2, 2), k_prefix=k, v_prefix=v), dict(block_table=i(2, 2), prefix_table=i(2).long())):
        with pytest.raises((ftd.FtdError, ValueError)):
            paged.prefix(**dict(ok, **kw))
    a = [ok[x].data_ptr() for x in ("q", "k_new", "v_new", "seq_lens", "prefix_lens", "out")]
    for rows in (-1, 1 << 30, 1 << 31, 1 << 62, (1 << 63) - 1):  # (times two heads)
        assert ftd.ftd_decode_mha_prefix(flat.ctx, a[0], a[1], a[2], 0, 0, 0, 0, a[3], 0, k.data_ptr(), v.data_ptr(), 0, 0, rows,
                                         a[4], a[5], 0) == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_kernel_launches() == n
    for s in (flat, paged, windowed, many):
        s.close()


@pytest.mark.parametrize("cache,out", [("bf16", "bf16"), ("bf16", "f32"), ("i8", "f16")])
def test_waits_that_run_out(cache, out):
    """A withheld copy: the bounded waits give up, the error is reported, and the next call is right."""
    qkv = "f16" if cache == "i8" else cache
    w, inp = case(cache, qkv, 4, 16, 2, 128, 64, [3, 9, 0, 30], 700, [700] * 4, bias=None)
    step = make_step(w, out_dtype=out, wait_limit_us=2000)
    step.enable_prefix()
    run(w, inp, out_dtype=out, step=step)
    assert ftd.ftd_debug_stall_next(step.ctx, 1) == ftd.FTD_OK
    run(w, inp, out_dtype=out, step=step, status=ftd.FTD_ERR_DEVICE_TIMEOUT, values=False)
    run(w, inp, out_dtype=out, step=step)
    step.close()
