"""The planes of ftd_decode_mha_scored: calls back to back in place, calls that fail part-way, and caches
whose rows end inside the last block of positions."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from tests import operators_ref as ref
from tests.gpu_util import dev, make_step, page_layout, to_pages
from tests.test_scored_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


@pytest.mark.parametrize("cache,Hq,Hkv,T,page", [("bf16", 32, 32, 1, 0), ("f16", 16, 2, 1, 128), ("bf16", 32, 2, 1, 0),
                                                 ("i8", 8, 8, 1, 256), ("f32", 4, 4, 2, 0)])
@pytest.mark.parametrize("captured", [False, True])
def test_back_to_back_in_place(cache, Hq, Hkv, T, page, captured):
    """Scored step, lengths, eviction, scored step, ... in place and without the host waiting in between give
    the bytes of the same calls with a wait after each: what a call reads is what the one before it left."""
    import torch
    B, D, Lmax, budget, steps = 6, 128, 512, 300, 24
    qkv = "f16" if cache == "i8" else cache
    lens0 = [400, 301, 300, 299, 40, 0]
    w, inp = ref.step_case(cache, qkv, B, Hq, Hkv, D, Lmax, lens0, T=T)
    opts, table, shape = {}, None, (B, Hkv, Lmax)
    arrs = {n: inp[n] for n in ("k_cache", "v_cache")}
    sc0 = inp.get("scales")
    if page:
        # (every page of every slot: the lengths grow)
        per = Lmax // page
        table = np.random.default_rng(2).permutation(B * per).reshape(B, per).astype(np.int32)
        opts, shape = dict(page_size=page, num_pages=B * per), (B * per, Hkv, page)
        arrs = {n: to_pages(w, a, table, B * per, page, np.zeros((), a.dtype)) for n, a in arrs.items()}
        if sc0 is not None:
            sc0 = np.stack([to_pages(w, x, table, B * per, page, np.float32(0)) for x in sc0])
    q, kn, vn, bias = (dev(inp[x]) for x in ("q", "k_new", "v_new", "bias"))
    tb = dev(table) if page else None
    g0 = torch.Generator(device="cuda").manual_seed(4)
    acc0 = torch.rand(shape, device="cuda", generator=g0)
    results = []
    for wait in (True, False):
        step = make_step(w, scored=True, q_len=T, **opts)
        k, v = dev(arrs["k_cache"]), dev(arrs["v_cache"])
        sc = dev(sc0) if sc0 is not None else None
        lens, npos = torch.tensor(lens0, dtype=torch.int32, device="cuda"), torch.tensor(lens0, dtype=torch.int32, device="cuda")
        acc, pos = acc0.clone(), torch.arange(shape[2], dtype=torch.int32, device="cuda").expand(shape).contiguous()
        out = torch.empty((steps, B, T, Hq, D), device="cuda")
        pause = torch.cuda.synchronize if wait else (lambda: None)
        torch.cuda.synchronize()

        def run(pause):
            for i in range(steps):
                step.scored(q, kn, vn, lens, npos, acc, pos, out[i], bias=bias, k_cache=k, v_cache=v, scales=sc, block_table=tb)
                pause()
                lens.add_(T)
                npos.add_(T)
                pause()
                if i % 3 == 2:
                    step.evict(acc, pos, lens, npos, lens, budget, recent=20, sinks=2, k_cache=k, v_cache=v, scales=sc,
                               block_table=tb)
                    pause()
        if captured and not wait:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                run(pause)
            g.replay()
        else:
            run(pause)
        torch.cuda.synchronize()
        assert step.get_error() == ftd.FTD_OK
        step.close()
        results.append([t.clone() for t in (lens, out, acc, pos)] + [t.view(torch.uint8).clone() for t in (k, v)])
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("cache,Hq,Hkv,D", [("bf16", 16, 1, 128), ("f16", 24, 1, 64), ("i8", 32, 2, 128), ("f32", 14, 1, 64),
                                            ("bf16", 13, 1, 128)])
@pytest.mark.parametrize("Lmax", [16, 144, 272, 400])
def test_many_rows_with_a_ragged_end(cache, Hq, Hkv, D, Lmax):
    """More than twelve query rows per kv head, cache rows that end 16 positions into a block of 128: nothing
    past a row's end counts, whatever the next row's scores are."""
    lens = [Lmax - 1, Lmax, 0, Lmax - 5, Lmax - 1]
    w, inp = ref.step_case(cache, "f16" if cache == "i8" else cache, len(lens), Hq, Hkv, D, Lmax, lens)
    check(w, inp)


SHAPES = {"mha_bf16": ("bf16", "bf16", 8, 8), "gqa8_tc": ("bf16", "bf16", 16, 2), "gqa16_tc": ("f16", "f16", 32, 2),
          "mha_i8": ("i8", "f16", 4, 4)}


@pytest.mark.parametrize("shape", list(SHAPES))
def test_a_call_that_gave_up_leaves_the_planes(shape):
    """A withheld copy: the weights gathered so far and the positions are kept, and the same call made again
    gives what it gives on a fresh context."""
    import torch
    cache, qkv, Hq, Hkv = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, 2, Hq, Hkv, 128, 512, [500, 130])
    rng = np.random.default_rng(6)
    acc0 = dev(rng.random((2, Hkv, 512)).astype(np.float32))
    pos0 = dev(rng.integers(0, 999, (2, Hkv, 512)).astype(np.int32))
    after = []
    for stall in (0, 1):
        step = make_step(w, scored=True, wait_limit_us=2000)
        q, kn, vn, b, sl, kc, vc = (dev(inp[x]) for x in ("q", "k_new", "v_new", "bias", "seq_lens", "k_cache", "v_cache"))
        sc = dev(inp["scales"]) if inp.get("scales") is not None else None
        acc, pos, out = acc0.clone(), pos0.clone(), torch.empty((2, Hq, 128), device="cuda")
        call = lambda: step.scored(q, kn, vn, sl, sl, acc, pos, out, bias=b, k_cache=kc, v_cache=vc, scales=sc)  # noqa: E731
        if stall:
            assert ftd.ftd_debug_stall_next(step.ctx, 1) == ftd.FTD_OK
            call()
            torch.cuda.synchronize()
            assert step.get_error() == ftd.FTD_ERR_DEVICE_TIMEOUT
            assert torch.equal(acc, acc0) and torch.equal(pos, pos0)
        call()
        torch.cuda.synchronize()
        assert step.get_error() == ftd.FTD_OK
        assert not torch.equal(acc, acc0)
        after.append((acc.clone(), pos.clone(), out.clone()))
        step.close()
    for a, b in zip(*after):
        assert torch.equal(a, b)


@pytest.mark.parametrize("Hq,Hkv,T,window", [(8, 8, 1, 0), (16, 2, 1, 0), (32, 1, 1, 0), (16, 2, 2, 0), (8, 8, 1, 100)])
@pytest.mark.parametrize("apart", [False, True])
def test_a_bad_page_leaves_its_slot_in_the_planes(Hq, Hkv, T, window, apart):
    """The slot behind a bad table entry keeps its weights and positions, the others' are those of a sound call;
    entries behind a window are not looked at."""
    import torch
    lens = [300, 200, 250]
    w, inp = ref.step_case("bf16", "bf16", 3, Hq, Hkv, 128, 512, lens, T=T)
    table, num_pages, _ = page_layout(w, lens, 128, 2, seed=3, q_len=T)
    bad = table.copy()
    bad[0, 1] = num_pages  # positions 128 .. 255: visible in slot 0, with the window too
    if window:
        bad[2, 0] = -7  # positions 0 .. 127: slot 2 sees 151 .. 250
    k0, v0 = (to_pages(w, inp[n], table, num_pages, 128, np.zeros((), inp[n].dtype)) for n in ("k_cache", "v_cache"))
    rng = np.random.default_rng(8)
    acc0 = dev(rng.random((num_pages, Hkv, 128)).astype(np.float32))
    pos0 = dev(rng.integers(0, 999, (num_pages, Hkv, 128)).astype(np.int32))
    res = []
    for tb in (table, bad):
        step = make_step(w, scored=True, page_size=128, num_pages=num_pages, q_len=T, window=window)
        acc, pos = acc0.clone(), pos0.clone()
        acc_out = acc0.clone() if apart else None
        out = torch.empty((3, T, Hq, 128), device="cuda")
        sl = dev(inp["seq_lens"])
        step.scored(dev(inp["q"]), dev(inp["k_new"]), dev(inp["v_new"]), sl, sl, acc, pos, out, acc_out=acc_out,
                    bias=dev(inp["bias"]), k_cache=dev(k0), v_cache=dev(v0), block_table=dev(tb))
        torch.cuda.synchronize()
        assert step.get_error() == (ftd.FTD_OK if tb is table else ftd.FTD_ERR_BAD_PAGE)
        res.append(((acc_out if apart else acc).clone(), pos.clone()))
        step.close()
    mine = {b: [int(x) for x in table[b] if 0 <= x < num_pages] for b in range(3)}
    for i, first in ((0, acc0), (1, pos0)):
        assert torch.equal(res[1][i][mine[0]], first[mine[0]])
        assert torch.equal(res[1][i][mine[1]], res[0][i][mine[1]])
        assert not torch.equal(res[0][i][mine[0]], first[mine[0]])
        assert torch.equal(res[1][i][mine[2]], res[0][i][mine[2]])
