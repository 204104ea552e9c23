"""The operators around the step at the ends of their documented ranges: up to 64 new tokens, windows
shorter than a step, other softmax scales, 1024 slots, caches whose offsets pass 32 bits, the
smallest caches, thousands of heads, and a score workspace that does not fit the device."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
import oracle
from tests import operators_ref as ref
from tests import test_cross_gpu as cross
from tests import test_rope_gpu as rope
from tests import test_scored_gpu as scored
from tests.gpu_util import TOL_MAXABS, TOL_MAXABS_I8, assert_close, make_step
from tests.test_evict_gpu import check as check_evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


SHAPES = {"mha_bf16": ("bf16", "bf16", 2, 2, 128), "mha_f16_d64": ("f16", "f16", 2, 2, 64), "gqa7_f32": ("f32", "f32", 7, 1, 64),
          "gqa3": ("f16", "f16", 3, 1, 128), "gqa8": ("bf16", "bf16", 8, 1, 128), "mha_i8": ("i8", "f16", 2, 2, 128),
          "gqa4_i8_d64": ("i8", "bf16", 4, 1, 64), "gqa8_i8": ("i8", "f16", 8, 1, 128)}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("T", [17, 64])
def test_many_new_tokens(shape, T):
    """New rows that span two tiles, more tokens than a block of rows, slots with nothing cached."""
    cache, qkv, Hq, Hkv, D = SHAPES[shape]
    Lmax = 400
    w, inp = ref.step_case(cache, qkv, 6, Hq, Hkv, D, Lmax, [0, 100, 127, Lmax - T, Lmax - T + 1, -1], T=T)
    scored.check(w, inp)
    w, inp = cross.case(cache, qkv, 5, Hq, Hkv, D, Lmax, [0, 1, 129, Lmax, -5], T=T)
    got, status = cross.run(w, inp)
    assert status == ftd.FTD_OK
    assert_close(got, cross.expect(w, inp), i8=cache == "i8", what=shape)


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("T,window", [(5, 3), (5, 1), (64, 10), (20, 140)])
@pytest.mark.parametrize("apart", [False, True])
def test_windows_shorter_than_a_step(shape, T, window, apart):
    cache, qkv, Hq, Hkv, D = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, 4, Hq, Hkv, D, 400, [0, 120, 250, 400 - T], T=T)
    scored.check(w, inp, window=window, apart=apart)


@pytest.mark.parametrize("shape", ["mha_bf16", "gqa3", "gqa8", "mha_i8", "gqa8_i8"])
@pytest.mark.parametrize("T", [9, 64])
def test_many_new_tokens_in_pages(shape, T):
    cache, qkv, Hq, Hkv, D = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, 5, Hq, Hkv, D, 512, [0, 125, 250, 512 - T, -1], T=T)
    scored.check(w, inp, page=128)


@pytest.mark.parametrize("shape", ["mha_bf16", "mha_f16_d64", "gqa7_f32", "gqa8", "mha_i8", "gqa8_i8"])
@pytest.mark.parametrize("scale", [0.01, 0.125, 0.37, 0.6931472])
def test_softmax_scales(shape, scale):
    """The scored step keeps a power of two of the scale in q and the rest beside it: both exactly a power, in the
    log2 domain, just below one and far from one."""
    import torch
    cache, qkv, Hq, Hkv, D = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, 3, Hq, Hkv, D, 256, [200, 3, 0], bias=None)
    r = oracle.load().decode_step(w, inp, nthreads=4, softmax_scale=scale)
    step = make_step(w, softmax_scale=scale, scored=True)
    d = {x: scored.dev(inp[x]) for x in ("q", "k_new", "v_new", "k_cache", "v_cache", "seq_lens")}
    sc = scored.dev(inp["scales"]) if cache == "i8" else None
    acc, out = torch.zeros((3, Hkv, 256), device="cuda"), torch.empty((3, Hq, D), device="cuda")
    step.scored(d["q"], d["k_new"], d["v_new"], d["seq_lens"], None, acc, None, out, k_cache=d["k_cache"],
                v_cache=d["v_cache"], scales=sc)
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    assert_close(out.double().cpu().numpy(), r["out"], i8=cache == "i8", what=f"scale {scale}")
    kh = scored.host(d["k_cache"], inp["k_cache"])
    scg = sc.cpu().numpy() if sc is not None else None
    g = Hq // Hkv
    for b, L in enumerate(inp["seq_lens"]):
        k = ref.cache_rows(w, kh, scg, 0, b, L + 1)
        q = ref.queries(w, inp, b)[0]
        s = scale * np.einsum("hd,hnd->hn", q, np.repeat(k, g, axis=0))
        p = np.exp(s - s.max(axis=1, keepdims=True))
        want = (p / p.sum(axis=1, keepdims=True)).reshape(Hkv, g, -1).sum(axis=1)
        mass = scale * np.einsum("hd,hnd->hn", np.abs(q), np.abs(np.repeat(k, g, axis=0))).max()
        got = acc[b, :, :L + 1].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= want * (ref.weight_tolerance(w, mass, False) + 2.0 ** -23) + 1e-30)
    # cross attention over the same rows as a memory
    lens = d["seq_lens"] + 1
    cr = torch.empty_like(out)
    step.cross(d["q"], lens, cr, k_mem=d["k_cache"], v_mem=d["v_cache"], scales=sc)
    torch.cuda.synchronize()
    assert np.abs(cr.double().cpu().numpy() - r["out"]).max() <= (TOL_MAXABS_I8 if cache == "i8" else TOL_MAXABS)
    step.close()


@pytest.mark.parametrize("cache,Hq,Hkv", [("bf16", 1, 1), ("f16", 16, 1), ("i8", 2, 1), ("f32", 3, 3)])
@pytest.mark.parametrize("page", [0, 128])
def test_1024_slots(cache, Hq, Hkv, page):
    rng = np.random.default_rng(7)
    lens = rng.integers(-1, 32, 1024)
    w, inp = ref.step_case(cache, "f16" if cache == "i8" else cache, 1024, Hq, Hkv, 64, 32, lens)
    scored.check(w, inp, page=page)
    check_evict(cache, 1024, Hkv, 64, 32, lens, 9, recent=3, sinks=1, page=page, apart=page == 0)


@pytest.mark.parametrize("L", [0, 1, 2, 15, 16])
@pytest.mark.parametrize("budget", [1, 15, 16])
def test_smallest_caches(L, budget):
    check_evict("f16", 2, 1, 64, 16, [L, 16], budget)
    if L < 16:
        w, inp = ref.step_case("f16", "f16", 2, 4, 1, 64, 16, [L, 15])
        scored.check(w, inp)


@pytest.mark.parametrize("Hq,Hkv", [(5000, 1), (4097, 4097), (9000, 3000)])
def test_thousands_of_heads(Hq, Hkv):
    rope.check(Hq, Hkv, 64, "f16", 3, axes=2)


def test_rows_far_apart():
    """Rows of a projection whose element offsets pass 32 bits."""
    import torch
    stride, Hq, Hkv, D, n = (1 << 30) + 8, 4, 2, 64, 5
    buf = torch.empty(4 * stride + 4096, dtype=torch.float16, device="cuda")
    x = torch.as_strided(buf, (n, (Hq + 2 * Hkv) * D), (stride, 1))
    x.normal_()
    pos = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    step = ftd.DecodeStep(1, Hq, Hkv, D, 16, "f16", "f16")
    step.set_rope()
    outs = [[torch.empty((n, h * D), dtype=torch.float16, device="cuda") for h in (Hq, Hkv, Hkv)] for _ in range(2)]
    for y, o in ((x, outs[0]), (x.contiguous(), outs[1])):
        step.rope(y[:, :Hq * D], y[:, Hq * D:(Hq + Hkv) * D], y[:, (Hq + Hkv) * D:], pos, *o)
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    step.close()


@pytest.mark.parametrize("cache,Hq,page", [("bf16", 20, 0), ("bf16", 160, 0), ("f16", 20, 128), ("i8", 160, 0)])
def test_offsets_past_32_bits(cache, Hq, page):
    """The last kv head's rows lie more than 2^31 elements into the cache: scored step, eviction and cross attention
    there give what they give on a small cache with the same rows."""
    import torch
    Hkv, D, B, n, budget = 20, 128, 1, 700, 300
    td = {"bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}[cache]
    qd = torch.bfloat16 if cache == "bf16" else torch.float16
    g = torch.Generator(device="cuda").manual_seed(11)
    res = []
    q = torch.randn((B, Hq, D), device="cuda", generator=g).to(qd)
    kn, vn = (torch.randn((B, Hkv, D), device="cuda", generator=g).to(qd) for _ in range(2))
    rows = [torch.randint(-127, 128, (B, Hkv, n, D), device="cuda", generator=g).to(torch.int8) if cache == "i8" else
            torch.randn((B, Hkv, n, D), device="cuda", generator=g).to(td) for _ in range(2)]
    scl = torch.rand((2, B, Hkv, n), device="cuda", generator=g) * 0.02
    acc_rows = torch.rand((B, Hkv, n), device="cuda", generator=g)
    for Lmax in (1024, 1 << 20):
        opts, table, shape = {}, None, (B, Hkv, Lmax)
        if page:  # 8 pages of 1024 positions, or the last ones of many
            pages = 8 if Lmax == 1024 else (1 << 20) // page
            opts, shape = dict(page_size=page, num_pages=pages), (pages, Hkv, page)
            table = torch.arange(pages - 1, pages - 9, -1, dtype=torch.int32, device="cuda").view(1, 8).contiguous()
        step = ftd.DecodeStep(B, Hq, Hkv, D, 1024 if page else Lmax, "bf16" if cache == "bf16" else "f16", cache, scored=True, **opts)
        k, v = (torch.empty(shape + (D,), dtype=td, device="cuda") for _ in range(2))
        sc = torch.empty((2,) + shape, device="cuda") if cache == "i8" else None
        acc, pos = torch.empty(shape, device="cuda"), torch.empty(shape, dtype=torch.int32, device="cuda")

        def put(x, r):
            if not page:
                x[:, :, :n] = r
            else:
                for i in range(-(-n // page)):
                    m = min(page, n - i * page)
                    x[int(table[0, i])][:, :m] = r[0, :, i * page:i * page + m]

        def get(x, m):
            if not page:
                return x[:, :, :m].clone()
            return torch.cat([x[int(table[0, i])] for i in range(8)], 1)[None, :, :m].clone()
        put(k, rows[0]), put(v, rows[1]), put(acc, acc_rows)
        put(pos, torch.arange(n, dtype=torch.int32, device="cuda").expand(B, Hkv, n))
        if sc is not None:
            put(sc[0], scl[0]), put(sc[1], scl[1])
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        out, cr = torch.empty((B, Hq, D), device="cuda"), torch.zeros((B, Hq, D), device="cuda")
        kw = dict(scales=sc, block_table=table)
        step.scored(q, kn, vn, lens, lens, acc, pos, out, k_cache=k, v_cache=v, **kw)
        lens += 1
        got = [out.clone(), get(acc, n + 1), get(pos, n + 1)] + [get(x, n + 1) for x in (k, v)]
        step.evict(acc, pos, lens, lens, lens, budget, recent=20, sinks=4, k_cache=k, v_cache=v, **kw)
        if not page:
            step.cross(q, lens, cr, k_mem=k, v_mem=v, scales=sc)
        torch.cuda.synchronize()
        assert step.get_error() == ftd.FTD_OK and lens.item() == budget
        # (the kernel, and so the last bits of weights and outputs, may differ between the two sizes; the eviction's
        # order is taken from weights that differ by far more)
        res.append(got + [get(pos, budget)] + [get(x, budget) for x in (k, v)] + [cr.clone()])
        step.close()
        del k, v, sc, acc, pos, step
        torch.cuda.empty_cache()
    small, large = res
    for i in (0, 8):
        assert_close(large[i].double().cpu().numpy(), small[i].double().cpu().numpy(), i8=cache == "i8")
    assert torch.allclose(large[1], small[1], rtol=2.0 ** -16, atol=0)
    for i in (2, 3, 4, 5, 6, 7):
        assert torch.equal(large[i], small[i]), i


def test_score_workspace_that_does_not_fit():
    """FTD_ERR_OOM, and the context goes on without scores."""
    import torch
    B, Hq, Hkv, D, Lmax, T = 8, 64, 1, 64, 1 << 22, 64
    step = ftd.DecodeStep(B, Hq, Hkv, D, Lmax, "f16", "i8", q_len=T)
    with pytest.raises(ftd.FtdError) as e:
        step.enable_scores()
    assert e.value.status == ftd.FTD_ERR_OOM
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, out = torch.zeros((B, T, Hq, D), dtype=torch.float16, device="cuda"), torch.empty((B, T, Hq, D), device="cuda")
    step.cross(q, lens, out)
    torch.cuda.synchronize()
    assert not out.any() and step.get_error() == ftd.FTD_OK
    a = torch.zeros(16, device="cuda")
    assert ftd.ftd_decode_mha_scored(step.ctx, q.data_ptr(), q.data_ptr(), q.data_ptr(), 0, 0, 0, 0, lens.data_ptr(), 0, 0,
                                     a.data_ptr(), 0, 0, out.data_ptr(), 0) == ftd.FTD_ERR_INVALID_ARG
    step.close()
