"""ftd_decode_mha_scored: the step's output and appended rows against the oracle, the
accumulated weights against attention in 64 bits, the positions plane exactly; every
cache type and kernel, several new tokens, windows, pages, ragged and empty slots, with
everything outside a slot's rows poisoned and left as it was."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
import oracle
from tests import operators_ref as ref
from tests.gpu_util import (assert_close, assert_same_bytes, dev, from_pages, host, make_step, page_layout, rising_scores, scale_q,
                            to_pages, valid_rows)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


SHAPES = {
    "mha_bf16": ("bf16", "bf16", 8, 8, 128, False),
    "mha_f16_d64": ("f16", "f16", 4, 4, 64, False),
    "mha_f32": ("f32", "f32", 4, 4, 128, False),
    "odd_group": ("f32", "f32", 6, 2, 64, False),
    "mha_i8": ("i8", "f16", 8, 8, 128, False),
    "gqa4_i8_d64": ("i8", "f16", 8, 2, 64, False),
    "gqa4_tc": ("bf16", "bf16", 16, 4, 128, False),
    "gqa8_tc": ("bf16", "bf16", 16, 2, 128, False),
    "gqa8_tc_f16": ("f16", "f16", 16, 2, 128, False),
    "gqa16_tc": ("bf16", "bf16", 32, 2, 128, False),
    "gqa48_tc": ("f16", "f16", 48, 1, 128, False),
    "gqa8_tc_i8": ("i8", "f16", 16, 2, 128, False),
    "gqa8_cc": ("bf16", "bf16", 16, 2, 128, True),
    "gqa8_cc_i8": ("i8", "f16", 16, 2, 128, True),
    "wide32": ("bf16", "bf16", 32, 1, 128, False),
    "wide64": ("f16", "f16", 64, 1, 128, False),
    "two_wide": ("bf16", "bf16", 128, 1, 128, False),
    # rows that fill no block of 4: padded tensor-core blocks, and 17, which no block divides
    # head_dim 64 on the tensor cores
    "gqa8_d64": ("bf16", "bf16", 16, 2, 64, False),
    "gqa16_d64": ("f16", "f16", 16, 1, 64, False),
    "gqa32_d64": ("bf16", "bf16", 64, 2, 64, False),
    "gqa7_d64": ("f16", "f32", 14, 2, 64, False),
    "gqa8_i8_d64": ("i8", "bf16", 16, 2, 64, False),
    "gqa6_i8_d64": ("i8", "f16", 12, 2, 64, False),
    "gqa7": ("bf16", "bf16", 14, 2, 128, False),
    "gqa3": ("f16", "f16", 6, 2, 128, False),
    "gqa20": ("bf16", "bf16", 20, 1, 128, False),
    "gqa17": ("f16", "f16", 17, 1, 128, False),
    "gqa7_i8": ("i8", "f16", 14, 2, 128, False),
    "gqa12_i8": ("i8", "f16", 24, 2, 128, False),
}


def run(w, inp, window=0, cc=False, page=0, apart=True, step=None, bias=True, next_pos=None, seed=51):
    """One call on poisoned planes; checks everything but out's values, which it returns with the status."""
    import torch
    T, lens = w.q_len, inp["seq_lens"]
    ok = [0 <= L <= w.Lmax - T for L in lens]
    rng = np.random.default_rng(seed)
    acc = np.full((w.B, w.Hkv, w.Lmax), np.nan, np.float32)
    pos = np.full((w.B, w.Hkv, w.Lmax), -77, np.int32)
    for b, L in enumerate(lens):
        if ok[b]:
            acc[b, :, :L] = rng.random((w.Hkv, L)).astype(np.float32)
            pos[b, :, :L] = np.arange(L)
    next_pos = np.asarray(lens, np.int32) + 9 if next_pos is None else next_pos
    opts = {}
    arrs = dict(k=inp["k_cache"], v=inp["v_cache"], acc=acc, pos=pos)
    sc = inp.get("scales")
    table = None
    if page:
        table, num_pages, _ = page_layout(w, lens, page, 2, seed=7, q_len=T)
        opts = dict(page_size=page, num_pages=num_pages)
        arrs = {n: to_pages(w, a, table, num_pages, page, np.zeros((), a.dtype)) for n, a in arrs.items()}
        if sc is not None:
            sc = np.stack([to_pages(w, sc[i], table, num_pages, page, np.float32(0)) for i in range(2)])
    own = step is None
    if own:
        step = make_step(w, force_cuda_core=cc, window=window, q_len=T, scored=True, **opts)
    d = {n: dev(a) for n, a in arrs.items()}
    scd = dev(sc) if sc is not None else None
    out = torch.full((w.B, T, w.Hq, w.D), float("nan"), device="cuda")
    acc_out = torch.full_like(d["acc"], -5.0) if apart else d["acc"]
    q, kn, vn, sl = (dev(inp[x]) for x in ("q", "k_new", "v_new", "seq_lens"))
    before = ftd.ftd_kernel_launches()
    step.scored(q, kn, vn, sl, dev(next_pos), d["acc"], d["pos"], out, acc_out=acc_out if apart else None,
                bias=dev(inp["bias"]) if bias else None, k_cache=d["k"], v_cache=d["v"], scales=scd,
                block_table=dev(table) if page else None)
    torch.cuda.synchronize()
    assert ftd.ftd_kernel_launches() == before + 2
    status = step.get_error()
    got = {n: t.cpu().numpy() for n, t in (("acc", acc_out), ("pos", d["pos"]))}
    kv = {n: host(d[n], arrs[n]) for n in ("k", "v")}
    scg = scd.cpu().numpy() if scd is not None else None
    if apart:
        a0 = d["acc"].cpu().numpy()
        assert_same_bytes(a0, arrs["acc"], "acc is only read")
    if page:
        got = {n: from_pages(w, a, table, page, lens, q_len=T) for n, a in got.items()}
        kv = {n: from_pages(w, a, table, page, lens, q_len=T) for n, a in kv.items()}
        if scg is not None:
            scg = np.stack([from_pages(w, scg[i], table, page, lens, q_len=T) for i in range(2)])
    inp_b = inp if bias else dict(inp, bias=None)
    worst = 0.0
    for b, L in enumerate(lens):
        end = L + T if ok[b] else 0
        if not page:  # outside the slot's rows nothing is written
            rest = got["acc"][b, :, end:]
            assert np.all(rest == -5.0) if apart else np.all(np.isnan(rest)), b
            assert_same_bytes(got["pos"][b, :, end:], pos[b, :, end:], "positions past the end")
        if not ok[b]:
            continue
        add, mass = ref.added_weights(w, inp_b, kv["k"], scg, b, window)
        want = add.copy()
        want[:, :L] += acc[b, :, :L].astype(np.float64)
        tol = add * ref.weight_tolerance(w, mass, bias) + 2 * want * 2.0 ** -24 + 1e-30
        err = np.abs(got["acc"][b, :, :end].astype(np.float64) - want)
        worst = max(worst, float((err / tol).max()))
        assert np.all(err <= tol), (b, L, float((err / tol).max()))
        assert np.array_equal(got["pos"][b, :, :L], pos[b, :, :L])
        for j in range(T):
            assert np.all(got["pos"][b, :, L + j] == next_pos[b] + j)
    if own:
        step.close()
    return out, kv, scg, status


def check(w, inp, window=0, cc=False, page=0, **kw):
    r = oracle.load().decode_step(w, inp, nthreads=8, window=window)
    out, kv, scg, status = run(w, inp, window=window, cc=cc, page=page, **kw)
    assert status == (ftd.FTD_ERR_SEQ_OVERFLOW if r["overflow"] else ftd.FTD_OK)
    want = dict(k=r["k_cache"].copy(), v=r["v_cache"].copy())
    if w.cache_dtype == "i8":  # this step's row scale is its own
        scales = inp["scales"].copy()
        for b, L in enumerate(inp["seq_lens"]):
            if 0 <= L <= w.Lmax - w.q_len:
                for i, n in enumerate("kv"):
                    want[n][b, :, L:L + w.q_len], scales[i, b, :, L:L + w.q_len] = ref.appended_i8(w, inp, b, n)
                    assert_same_bytes(scg[i, b, :, :L + w.q_len], scales[i, b, :, :L + w.q_len], f"{n} scales after append")
    if page:
        want = {n: valid_rows(w, a, inp["seq_lens"], q_len=w.q_len) for n, a in want.items()}
    for n in "kv":
        assert_same_bytes(kv[n], want[n], f"{n} after append")
    assert_close(out.double().cpu().numpy().reshape(r["out"].shape), r["out"], i8=w.cache_dtype == "i8")


LENS = [0, 1, 63, 127, 128, 300, -1, 511, 512]


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("T", [1, 3])
def test_shapes(shape, T):
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, len(LENS), Hq, Hkv, D, 512, LENS, T=T)
    check(w, inp, cc=cc, apart=T == 1)


@pytest.mark.parametrize("Hq,Hkv,T", [(64, 1, 1), (32, 1, 1), (64, 2, 1), (32, 1, 3), (128, 1, 1)])
def test_wide_and_narrow_blocks(Hq, Hkv, T):
    """Multiples of 32 query rows, with more tiles than SMs (64- or 32-row blocks) and with fewer (16-row ones)."""
    for B, Lmax in ((3, 512), (40, 1024)):
        lens = np.random.default_rng(B).integers(0, Lmax - T, B)
        if B == 40:
            lens = lens // 4
        w, inp = ref.step_case("bf16", "bf16", B, Hq, Hkv, 128, Lmax, lens, T=T)
        check(w, inp)


@pytest.mark.parametrize("shape", ["mha_bf16", "mha_f32", "mha_i8", "gqa8_tc", "gqa8_tc_i8", "wide32", "wide64", "gqa8_d64",
                                   "gqa8_i8_d64"])
@pytest.mark.parametrize("T,window", [(1, 1), (1, 100), (2, 130), (4, 400)])
@pytest.mark.parametrize("apart", [False, True])
def test_windows(shape, T, window, apart):
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, 5, Hq, Hkv, D, 768, [0, 99, 130, 500, 764], T=T)
    check(w, inp, cc=cc, window=window, apart=apart)


@pytest.mark.parametrize("shape", ["mha_bf16", "mha_i8", "gqa8_tc", "gqa8_tc_i8", "wide64", "gqa8_d64", "gqa8_i8_d64"])
@pytest.mark.parametrize("page", [128, 256])
def test_pages(shape, page):
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, 6, Hq, Hkv, D, 720, [0, 127, 128, 500, -1, 718], T=2)
    check(w, inp, cc=cc, page=page)


@pytest.mark.parametrize("shape", ["mha_bf16", "mha_f32", "gqa8_tc", "wide32", "gqa8_tc_i8", "mha_i8", "gqa16_d64",
                                   "gqa8_i8_d64"])
def test_long_context_split_over_blocks(shape):
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, 2, Hq, Hkv, D, 8192, [8190, 40], T=2)
    check(w, inp, cc=cc)


@pytest.mark.parametrize("shape", ["wide32", "wide64", "two_wide"])
@pytest.mark.parametrize("T,window,page", [(1, 0, 0), (3, 0, 0), (1, 100, 0), (2, 130, 0), (2, 0, 256)])
def test_wide_options(shape, T, window, page):
    """Edge lengths, windows and pages on the wide kernel (caches long enough for its blocks)."""
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    if Hq * T > 200:
        T = 1
    w, inp = ref.step_case(cache, qkv, 6, Hq, Hkv, D, 4096, [0, 99, 127, 128, 1500, -1], T=T)
    check(w, inp, window=window, page=page, apart=window == 0)


@pytest.mark.parametrize("shape,B,Lmax", [("gqa8_tc", 12, 32768), ("mha_bf16", 20, 32800), ("wide32", 8, 20000),
                                          ("wide64", 4, 20016), ("gqa8_tc_i8", 12, 32768)])
def test_scores_dropped_from_l2(shape, B, Lmax):
    """Score workspaces past 16 MB, whose lines are dropped after their reading (and, with 20016 positions a
    row, are not): two calls in a row, the second on other lengths, with many query rows and with few."""
    import torch
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    rng = np.random.default_rng(B)
    w = ref.Workload("drop", B=B, Hq=Hq, Hkv=Hkv, D=D, Lmax=Lmax, qkv_dtype=qkv, cache_dtype=cache)
    assert B * Hq * Lmax * 4 >= 16 << 20
    step = make_step(w, scored=True)
    td = {"bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
    g = torch.Generator(device="cuda").manual_seed(3)
    shp = (B, Hkv, Lmax, D)
    if cache == "i8":
        k, v = (torch.randint(-127, 128, shp, dtype=torch.int8, device="cuda", generator=g) for _ in range(2))
        sc = torch.rand((2,) + shp[:3], device="cuda", generator=g) * 0.02
    else:
        k, v = (torch.randn(shp, device="cuda", generator=g, dtype=td[cache]) for _ in range(2))
        sc = None
    q = torch.randn((B, Hq, D), device="cuda", generator=g, dtype=td[qkv])
    kn, vn = (torch.randn((B, Hkv, D), device="cuda", generator=g, dtype=td[qkv]) for _ in range(2))
    out = torch.empty((B, Hq, D), device="cuda")
    acc, acc_out = torch.zeros(shp[:3], device="cuda"), torch.empty(shp[:3], device="cuda")
    for _ in range(3):
        lens = torch.from_numpy(rng.integers(0, Lmax, B).astype(np.int32)).cuda()
        acc_out.fill_(-1.0)
        step.scored(q, kn, vn, lens, lens, acc, None, out, acc_out=acc_out, k_cache=k, v_cache=v, scales=sc)
        torch.cuda.synchronize()
        for b in {0, B // 2, B - 1}:
            n = int(lens[b]) + 1
            kk = k[b, :, :n].double() * (sc[0, b, :, :n, None].double() if sc is not None else 1.0)
            s = torch.einsum("hgd,hnd->hgn", q[b].double().view(Hkv, Hq // Hkv, D), kk) / np.sqrt(D)
            want = torch.softmax(s, -1).sum(1)
            got = acc_out[b, :, :n].double()
            mass = float((q[b].double().abs().view(Hkv, -1, D).amax(1)[:, None] * kk.abs()).sum(-1).max()) / np.sqrt(D)
            assert torch.all((got - want).abs() <= want * ref.weight_tolerance(w, mass, False) + 1e-30)
            assert torch.all(acc_out[b, :, n:] == -1.0)
    assert step.get_error() == ftd.FTD_OK
    step.close()


@pytest.mark.parametrize("shape", ["mha_bf16", "gqa8_tc", "wide64"])
def test_rising_scores(shape):
    """The running reference moves all along the context, so early weights come out near zero."""
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, 2, Hq, Hkv, D, 2048, [2000, 700])
    check(w, rising_scores(w, inp))


@pytest.mark.parametrize("shape", ["mha_bf16", "gqa8_tc", "gqa8_tc_f16", "mha_i8", "gqa8_tc_i8", "wide32"])
def test_weights_without_bias(shape):
    """A 16-bit query without a bias is held exactly, so the fp32 weights keep fp32 accuracy."""
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = ref.step_case(cache, qkv, 3, Hq, Hkv, D, 512, [500, 200, 7])
    run(w, inp, bias=False)


@pytest.mark.parametrize("cache,qkv", [("f16", "f32"), ("i8", "bf16")])
def test_large_queries(cache, qkv):
    """Queries past fp16's range whose scaled values are within it, as the plain step takes them."""
    w, inp = ref.step_case(cache, qkv, 2, 16, 2, 128, 256, [200, 5], bias=None)
    inp = scale_q(w, inp, 30000.0)
    inp["k_cache"] = (inp["k_cache"].astype(np.float32) * 1e-4).astype(np.float16) if cache == "f16" else inp["k_cache"]
    if cache == "i8":
        inp["scales"][0] *= np.float32(1e-4)
    inp["k_new"] = ref.store(ref.widen(inp["k_new"], qkv) * 1e-4, qkv)
    assert np.abs(ref.widen(inp["q"], qkv)).max() > 65504
    out, *_ = run(w, inp, bias=False)
    r = oracle.load().decode_step(w, inp, nthreads=8)
    assert_close(out.double().cpu().numpy().reshape(r["out"].shape), r["out"], i8=cache == "i8")


def test_weights_sum_to_the_rows():
    """Over the positions, a kv head's added weights are its query rows' count, step after step."""
    import torch
    w, inp = ref.step_case("bf16", "bf16", 2, 16, 2, 128, 256, [100, 3])
    step = make_step(w, scored=True)
    kc, vc, b = dev(inp["k_cache"]), dev(inp["v_cache"]), dev(inp["bias"])
    acc = torch.zeros((2, 2, 256), device="cuda")
    pos = torch.zeros((2, 2, 256), dtype=torch.int32, device="cuda")
    out = torch.empty((2, 16, 128), device="cuda")
    lens = torch.tensor([100, 3], dtype=torch.int32, device="cuda")
    for i in range(5):
        step.scored(dev(inp["q"]), dev(inp["k_new"]), dev(inp["v_new"]), lens, lens, acc, pos, out, bias=b, k_cache=kc,
                    v_cache=vc)
        lens += 1
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    # five rows of eight weights that sum to 1, each weight off by under 2^-20 of itself
    assert np.all(np.abs(acc.double().sum(-1).cpu().numpy() - 40.0) <= 40.0 * 2.0 ** -18)
    assert pos[0, 0, 100:105].tolist() == [100, 101, 102, 103, 104] and pos[1, 1, 3:8].tolist() == [3, 4, 5, 6, 7]
    step.close()


def test_without_positions_and_same_step_output():
    """positions may be absent; the output is the plain step's within the bars, and a plain step on
    the same context afterwards gives its own bytes."""
    import torch
    w, inp = ref.step_case("f16", "f16", 3, 8, 8, 128, 256, [200, 3, 0])
    step = make_step(w, scored=True)
    q, kn, vn, b, sl = (dev(inp[x]) for x in ("q", "k_new", "v_new", "bias", "seq_lens"))
    acc = torch.zeros((3, 8, 256), device="cuda")
    outs = [torch.empty((3, 8, 128), device="cuda") for _ in range(3)]
    for i, o in enumerate(outs):
        kc, vc = dev(inp["k_cache"]), dev(inp["v_cache"])
        if i == 1:
            step.scored(q, kn, vn, sl, None, acc, None, o, bias=b, k_cache=kc, v_cache=vc)
        else:
            step(q, kn, vn, sl, o, bias=b, k_cache=kc, v_cache=vc)
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    assert torch.equal(outs[0], outs[2])
    assert_close(outs[1].double().cpu().numpy(), outs[0].double().cpu().numpy())
    step.close()


def test_graph_replay_and_late_lengths():
    import torch
    w, inp = ref.step_case("bf16", "bf16", 3, 16, 2, 128, 512, [400, 40, 4])
    step = make_step(w, scored=True)
    q, kn, vn, b = (dev(inp[x]) for x in ("q", "k_new", "v_new", "bias"))
    kc, vc = dev(inp["k_cache"]), dev(inp["v_cache"])
    lens = torch.tensor([400, 40, 4], dtype=torch.int32, device="cuda")
    acc = torch.zeros((3, 2, 512), device="cuda")
    acc_out, pos = torch.zeros_like(acc), torch.zeros((3, 2, 512), dtype=torch.int32, device="cuda")
    out = torch.empty((3, 16, 128), device="cuda")

    def call():
        step.scored(q, kn, vn, lens, lens, acc, pos, out, acc_out=acc_out, bias=b, k_cache=kc, v_cache=vc)
    call()
    torch.cuda.synchronize()
    want = acc_out.clone(), out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    acc_out.zero_(), out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(acc_out, want[0]) and torch.equal(out, want[1])
    src = lens.clone()
    lens.copy_(torch.tensor([2, 500, 300], dtype=torch.int32))
    acc_out.zero_(), out.zero_()
    s = torch.cuda.current_stream().cuda_stream
    assert ftd.ftd_debug_late_lengths(src.data_ptr(), lens.data_ptr(), 3, 300, s) == ftd.FTD_OK
    call()
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    tol = dict(rtol=2.0 ** -16, atol=1e-7)  # the same sums, cut into pieces elsewhere
    assert torch.allclose(acc_out, want[0], **tol) and torch.allclose(out, want[1], rtol=1e-3, atol=1e-4)
    step.close()


def test_bad_page_is_reported_and_nothing_is_written_through_it():
    import torch
    w, inp = ref.step_case("bf16", "bf16", 2, 16, 2, 128, 512, [300, 200])
    table, num_pages, _ = page_layout(w, inp["seq_lens"], 128, 2, seed=3)
    bad = table.copy()
    bad[0, 1] = num_pages
    bad[0, 2] = -1
    step = make_step(w, scored=True, page_size=128, num_pages=num_pages)
    d = {n: dev(to_pages(w, inp[n], table, num_pages, 128, np.zeros((), inp[n].dtype))) for n in ("k_cache", "v_cache")}
    acc = torch.zeros((num_pages, 2, 128), device="cuda")
    pos = torch.full((num_pages, 2, 128), -1, dtype=torch.int32, device="cuda")
    out = torch.empty((2, 16, 128), device="cuda")
    sl = dev(inp["seq_lens"])
    step.scored(dev(inp["q"]), dev(inp["k_new"]), dev(inp["v_new"]), sl, sl, acc, pos, out, bias=dev(inp["bias"]),
                k_cache=d["k_cache"], v_cache=d["v_cache"], block_table=dev(bad))
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_ERR_BAD_PAGE
    used = set(table[0, :1]) | set(table[1, :2])
    for pg in range(num_pages):
        if pg not in used:
            assert not acc[pg].any() and (pos[pg] == -1).all(), pg
    step.close()


@pytest.mark.parametrize("shape", ["mha_bf16", "mha_i8", "gqa8_tc", "gqa8_tc_i8", "gqa8_d64", "wide32", "wide64"])
def test_withheld_copy_times_out_and_the_next_call_is_right(shape):
    import torch
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    Lmax = 12288 if shape.startswith("wide") else 512  # (long enough for the wide kernel's blocks)
    w, inp = ref.step_case(cache, qkv, 2, Hq, Hkv, D, Lmax, [500, 130])
    step = make_step(w, scored=True, wait_limit_us=2000)
    q, kn, vn, b, sl, kc, vc = (dev(inp[x]) for x in ("q", "k_new", "v_new", "bias", "seq_lens", "k_cache", "v_cache"))
    sc = dev(inp["scales"]) if inp.get("scales") is not None else None
    acc, out = torch.zeros((2, Hkv, Lmax), device="cuda"), torch.empty((2, Hq, D), device="cuda")
    acc_out = torch.zeros_like(acc)
    call = lambda: step.scored(q, kn, vn, sl, sl, acc, None, out, acc_out=acc_out, bias=b, k_cache=kc, v_cache=vc, scales=sc)  # noqa: E731
    assert ftd.ftd_debug_stall_next(step.ctx, 1) == ftd.FTD_OK
    call()
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_ERR_DEVICE_TIMEOUT
    r = oracle.load().decode_step(w, inp, nthreads=8)
    for _ in range(2):
        call()
        torch.cuda.synchronize()
        assert step.get_error() == ftd.FTD_OK
        assert_close(out.double().cpu().numpy(), r["out"], i8=cache == "i8", what=shape)
        n = Hq // Hkv  # each query row's weights sum to 1
        assert np.all(np.abs(acc_out.double().sum(-1).cpu().numpy() - n) <= n * 2.0 ** -16)
    step.close()


def test_refusals():
    import torch
    w, _ = ref.step_case("bf16", "bf16", 2, 8, 8, 128, 256, [1, 1])
    n = ftd.ftd_kernel_launches()
    a = torch.zeros((2, 8, 256), device="cuda")

    def call(step, **kw):
        x = dict(q=256, k=256, v=256, bias=0, kc=0, vc=0, table=0, lens=256, scales=0, next_pos=256, acc=a.data_ptr(),
                 acc_out=0, pos=256, out=256)
        x.update(kw)
        return ftd.ftd_decode_mha_scored(step.ctx, x["q"], x["k"], x["v"], x["bias"], x["kc"], x["vc"], x["table"],
                                         x["lens"], x["scales"], x["next_pos"], x["acc"], x["acc_out"], x["pos"],
                                         x["out"], 0)
    step = make_step(w)
    assert call(step) == ftd.FTD_ERR_INVALID_ARG and "ftd_enable_scores" in ftd.ftd_last_error()
    step.enable_scores()
    step.enable_scores()  # a second call does nothing
    for kw in (dict(acc=0), dict(acc=a.data_ptr() + 4), dict(acc_out=a.data_ptr() + 16), dict(acc_out=a.data_ptr() + 4),
               dict(next_pos=0), dict(next_pos=258), dict(pos=258), dict(table=256), dict(q=0), dict(k=0), dict(lens=0),
               dict(out=0), dict(out=264), dict(kc=264), dict(lens=257)):
        assert call(step, **kw) == ftd.FTD_ERR_INVALID_ARG, kw
        assert ftd.ftd_last_error() != ""
    step.close()
    step = make_step(w, scored=True, page_size=128, num_pages=4)
    assert call(step) == ftd.FTD_ERR_INVALID_ARG and "block table" in ftd.ftd_last_error()
    step.close()
    assert ftd.ftd_kernel_launches() == n
