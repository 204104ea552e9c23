"""ftd_cache_evict against a plain restatement, byte for byte: which rows stay, where the moved
ones go, and that nothing else changes; ties, special weights, protected rows, ragged and
inactive slots, every cache type, pages, planes in place and apart, long caches, and a
decoder's loop of rotary positions, scored steps, evictions and cross attention."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
import oracle
from synthetic import Workload, to_storage
from tests import operators_ref as ref
from tests.gpu_util import assert_close, assert_same_bytes, dev, from_pages, host, make_step, page_layout, to_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


def rows_of(w, rng):
    shape = (w.B, w.Hkv, w.Lmax, w.D)
    if w.cache_dtype == "i8":
        return [rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2)], rng.random((2,) + shape[:3]).astype(np.float32)
    return [to_storage(rng.standard_normal(shape).astype(np.float32), w.cache_dtype) for _ in range(2)], None


def positions_of(w, lens, next_pos, rng):
    """Distinct positions below next_pos, shuffled; next_pos is at least the slot's rows."""
    pos = np.full((w.B, w.Hkv, w.Lmax), -9, np.int32)
    for b, L in enumerate(lens):
        for h in range(w.Hkv if L > 0 else 0):
            pos[b, h, :min(L, w.Lmax)] = rng.permutation(int(next_pos[b]))[:min(L, w.Lmax)]
    return pos


def check(cache, B, Hkv, D, Lmax, lens, budget, recent=0, sinks=0, page=0, apart=True, alias=False, acc=None, seed=61):
    import torch
    w = Workload("evict", B=B, Hq=Hkv, Hkv=Hkv, D=D, Lmax=Lmax, qkv_dtype="f16" if cache == "i8" else cache,
                 cache_dtype=cache)
    rng = np.random.default_rng(seed)
    (k, v), sc = rows_of(w, rng)
    lens = np.asarray(lens, np.int32)
    next_pos = (np.clip(lens, 0, Lmax) + rng.integers(0, 50, B)).astype(np.int32)
    pos = positions_of(w, lens, next_pos, rng)
    if acc is None:
        acc = np.exp(2 * rng.standard_normal((B, Hkv, Lmax))).astype(np.float32)
    arrs = dict(k=k, v=v, acc=acc, pos=pos)
    if sc is not None:
        arrs.update(ks=sc[0], vs=sc[1])
    opts, table = {}, None
    dlens = lens if not page else np.where((lens >= 0) & (lens <= Lmax), lens, -1)
    if page:
        table, num_pages, _ = page_layout(w, dlens, page, 2, seed=8, q_len=0)
        opts = dict(page_size=page, num_pages=num_pages)
        dv = {n: to_pages(w, a, table, num_pages, page, np.zeros((), a.dtype)) for n, a in arrs.items()}
    else:
        dv = arrs
    d = {n: dev(a) for n, a in dv.items() if n not in ("ks", "vs")}
    scd = dev(np.stack([dv["ks"], dv["vs"]])) if sc is not None else None
    step = make_step(w, scored=True, **opts)
    acc_out = torch.full_like(d["acc"], -5.0) if apart else None
    pos_out = torch.full_like(d["pos"], -5) if apart else None
    sl = dev(lens)
    new = sl if alias else torch.full_like(sl, 12345)
    before = ftd.ftd_kernel_launches()
    for _ in range(2 if apart and not alias else 1):  # a second call on the same planes finds the same rows
        step.evict(d["acc"], d["pos"], sl, dev(next_pos), new, budget, recent=recent, sinks=sinks, acc_out=acc_out,
                   positions_out=pos_out, k_cache=d["k"], v_cache=d["v"], scales=scd,
                   block_table=dev(table) if page else None)
    torch.cuda.synchronize()
    assert ftd.ftd_kernel_launches() in (before + 2, before + 4)
    status = step.get_error()
    step.close()
    over = bool(np.any(lens > Lmax))
    assert status == (ftd.FTD_ERR_SEQ_OVERFLOW if over else ftd.FTD_OK)
    want = {n: a.copy() for n, a in arrs.items()}
    new_want = ref.evict(list(want.values()), arrs["acc"], arrs["pos"], lens, next_pos, budget, recent, sinks)
    assert np.array_equal(new.cpu().numpy(), new_want)
    got = dict(k=host(d["k"], k), v=host(d["v"], v), acc=(acc_out if apart else d["acc"]).cpu().numpy(),
               pos=(pos_out if apart else d["pos"]).cpu().numpy())
    if sc is not None:
        s = scd.cpu().numpy()
        got.update(ks=s[0], vs=s[1])
    if page:
        got = {n: from_pages(w, a, table, page, dlens, q_len=0) for n, a in got.items()}
        z = lambda a: np.zeros_like(a)  # noqa: E731
        keep = [n if 0 <= n <= Lmax else 0 for n in lens]
        want = {n: np.stack([np.concatenate([a[b][:, :keep[b]], z(a[b][:, keep[b]:])], axis=1) for b in range(B)])
                for n, a in want.items()}
    for n, a in got.items():
        for b, L in enumerate(lens):
            if n in ("acc", "pos") and apart:
                end = int(new_want[b]) if 0 <= L <= Lmax else 0
                assert_same_bytes(a[b, :, :end], want[n][b, :, :end], f"{n} of slot {b}")
                if not page:
                    assert np.all(a[b, :, end:] == -5), f"{n} of slot {b} past its rows"
            else:
                assert_same_bytes(a[b], want[n][b], f"{n} of slot {b}")


LENS = [0, 1, 99, 100, 101, 150, 256, -1]


@pytest.mark.parametrize("cache,D", [("bf16", 128), ("f16", 64), ("f32", 128), ("f32", 64), ("i8", 128), ("i8", 64)])
@pytest.mark.parametrize("apart", [False, True])
def test_cache_types(cache, D, apart):
    check(cache, len(LENS), 3, D, 256, LENS, 100, recent=20, sinks=4, apart=apart)


@pytest.mark.parametrize("cache", ["bf16", "i8"])
@pytest.mark.parametrize("page", [128, 256])
@pytest.mark.parametrize("apart", [False, True])
def test_pages(cache, page, apart):
    check(cache, 5, 2, 128, 400, [400, 130, 128, -1, 131], 129, recent=60, sinks=2, page=page, apart=apart)


@pytest.mark.parametrize("budget,recent,sinks", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (255, 255, 0), (255, 0, 255),
                                                 (128, 64, 64), (100, 0, 0), (256, 10, 10)])
def test_budgets(budget, recent, sinks):
    check("f16", 3, 2, 64, 256, [256, 200, 255], budget, recent, sinks)


@pytest.mark.parametrize("alias", [False, True])
def test_lengths_in_place(alias):
    check("bf16", 40, 5, 64, 128, list(range(89, 129)), 100, recent=9, alias=alias, apart=False)


def test_overflowing_slot_is_skipped():
    check("bf16", 4, 2, 64, 128, [128, 129, 2 ** 31 - 1, -2 ** 31], 50, apart=True)


@pytest.mark.parametrize("kind", ["equal", "few", "special", "descending", "ascending"])
def test_ties_and_special_weights(kind):
    rng = np.random.default_rng(5)
    shape = (3, 2, 640)
    acc = {"equal": np.full(shape, 0.25), "few": rng.integers(0, 3, shape),
           "special": rng.choice([0.0, -0.0, -1.0, 1e-45, 3e38, np.inf, -np.inf, np.nan, 1.0, -1e-40], shape),
           "descending": np.broadcast_to(-np.arange(640.0), shape),
           "ascending": np.broadcast_to(np.arange(640.0), shape)}[kind].astype(np.float32)
    if kind == "special":
        acc[acc == 0] = 0.0  # +0 only: the two zeros are separate keys below
    check("f16", 3, 2, 64, 640, [640, 401, 500], 400, recent=30, sinks=3, acc=acc)


@pytest.mark.parametrize("Lmax,L,budget", [(8192, 8190, 1000), (8192, 8192, 8191), (40000, 39999, 20000),
                                           (65536, 65530, 5000), (65536, 60000, 59999), (450000, 449999, 200000)])
def test_long_caches(Lmax, L, budget):
    """Past the keys that fit shared memory they are kept in the workspace."""
    check("i8", 1, 2, 64, Lmax, [L], budget, recent=500, sinks=16)


def test_more_protected_rows_than_the_budget():
    """Positions that repeat can protect more rows than recent: the lower rows stay."""
    import torch
    w = Workload("evict", B=1, Hq=1, Hkv=1, D=64, Lmax=64, qkv_dtype="f16", cache_dtype="f16")
    step = make_step(w, scored=True)
    k = torch.arange(64, device="cuda").view(1, 1, 64, 1).expand(1, 1, 64, 64).to(torch.float16).contiguous()
    v = -k
    acc = torch.rand((1, 1, 64), device="cuda")
    pos = torch.full((1, 1, 64), 63, dtype=torch.int32, device="cuda")
    sl = torch.tensor([64], dtype=torch.int32, device="cuda")
    step.evict(acc, pos, sl, sl, sl, 10, recent=5, k_cache=k, v_cache=v)
    torch.cuda.synchronize()
    assert sl.item() == 10 and k[0, 0, :, 0].tolist() == [float(i) for i in range(64)]
    step.close()


def test_bad_page_is_reported_and_the_slot_is_left():
    import torch
    w = Workload("evict", B=2, Hq=2, Hkv=2, D=64, Lmax=512, qkv_dtype="f16", cache_dtype="f16")
    rng = np.random.default_rng(9)
    lens = np.array([400, 300], np.int32)
    table, num_pages, _ = page_layout(w, lens, 128, 1, seed=4, q_len=0)
    bad = table.copy()
    bad[0, 2] = num_pages
    step = make_step(w, scored=True, page_size=128, num_pages=num_pages)
    k = torch.randn((num_pages, 2, 128, 64), device="cuda").half()
    v, k0 = k.clone(), k.clone()
    acc = torch.rand((num_pages, 2, 128), device="cuda")
    pos = dev(to_pages(w, positions_of(w, lens, lens, rng), table, num_pages, 128, np.int32(0)))
    sl = dev(lens)
    new = torch.zeros_like(sl)
    step.evict(acc, pos, sl, sl, new, 100, k_cache=k, v_cache=v, block_table=dev(bad))
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_ERR_BAD_PAGE
    for pg in range(num_pages):
        if pg not in set(table[1, :3]):
            assert torch.equal(k[pg], k0[pg])
    assert not torch.equal(k, k0) and new[1].item() == 100
    step.evict(acc, pos, sl, sl, new, 100, k_cache=k, v_cache=v, block_table=dev(table))  # the next call starts clean
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    step.close()


def test_graph_replay_from_other_lengths():
    """A captured eviction follows the lengths it finds."""
    import torch
    w = Workload("evict", B=2, Hq=2, Hkv=2, D=64, Lmax=256, qkv_dtype="f16", cache_dtype="f16")
    step = make_step(w, scored=True)
    rng = np.random.default_rng(10)
    sl = torch.zeros(2, dtype=torch.int32, device="cuda")
    npos = torch.full((2,), 256, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((2, 2, 256, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    acc, pos = torch.zeros((2, 2, 256), device="cuda"), torch.zeros((2, 2, 256), dtype=torch.int32, device="cuda")
    call = lambda: step.evict(acc, pos, sl, npos, sl, 64, recent=8, k_cache=k, v_cache=v)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([256, 64], [65, 200], [0, 100]):
        (k0, v0), _ = rows_of(w, rng)
        p0 = np.broadcast_to(np.arange(256, dtype=np.int32), (2, 2, 256)).copy()
        a0 = rng.random((2, 2, 256)).astype(np.float32)
        for t, a in ((k, k0), (v, v0), (acc, a0), (pos, p0), (sl, np.array(lens, np.int32))):
            t.copy_(torch.from_numpy(a))
        g.replay()
        torch.cuda.synchronize()
        want = [k0.copy(), v0.copy(), a0.copy(), p0.copy()]
        new = ref.evict(want, a0, p0, np.array(lens), [256, 256], 64, 8, 0)
        assert sl.tolist() == new.tolist()
        for t, a in zip((k, v, acc, pos), want):
            assert_same_bytes(t.cpu().numpy(), a, str(lens))
    assert step.get_error() == ftd.FTD_OK
    step.close()


def test_two_contexts_on_two_streams():
    """Each context has its own workspace: two decoders interleaved on two streams, not the current one,
    give what each gives alone."""
    import torch
    rng = np.random.default_rng(14)
    cases = [ref.step_case("bf16", "bf16", 3, 16, 2, 128, 512, [500, 300, 2], seed=s) for s in (1, 2)]
    pos0 = torch.arange(512, dtype=torch.int32, device="cuda").expand(3, 2, 512).contiguous()
    acc0 = [torch.from_numpy(rng.random((3, 2, 512)).astype(np.float32)).cuda() for _ in cases]
    results = []
    for together in (False, True):
        state = []
        for (w, inp), a in zip(cases, acc0):
            d = {x: dev(inp[x]) for x in ("q", "k_new", "v_new", "bias", "k_cache", "v_cache", "seq_lens")}
            st = dict(d, step=make_step(w, scored=True), acc=a.clone(), pos=pos0.clone(), s=torch.cuda.Stream(),
                      out=torch.empty((3, 16, 128), device="cuda"), cross=torch.empty((3, 16, 128), device="cuda"))
            st["step"].set_rope()
            state.append(st)
        torch.cuda.synchronize()
        for _ in range(6):
            for st in state:
                with torch.cuda.stream(st["s"]):
                    n = st["seq_lens"]
                    bf = lambda x: st[x].view(torch.bfloat16)  # noqa: E731
                    q, k = torch.empty_like(bf("q")), torch.empty_like(bf("k_new"))
                    st["step"].rope(bf("q"), bf("k_new"), None, n.view(1, 3), q, k)
                    st["step"].scored(q, k, st["v_new"], n, n, st["acc"], st["pos"], st["out"], k_cache=st["k_cache"],
                                      v_cache=st["v_cache"])
                    n += 1
                    st["step"].evict(st["acc"], st["pos"], n, n, n, 280, recent=20, k_cache=st["k_cache"],
                                     v_cache=st["v_cache"])
                    st["step"].cross(q, n, st["cross"], k_mem=st["k_cache"], v_mem=st["v_cache"])
                    if not together:
                        st["s"].synchronize()
        torch.cuda.synchronize()
        for st in state:
            assert st["step"].get_error() == ftd.FTD_OK
            st["step"].close()
        results.append([[st[x].clone() for x in ("out", "cross", "acc", "pos", "seq_lens", "k_cache", "v_cache")] for st in state])
    for a, b in zip(*results):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("cache", ["bf16", "i8"])
def test_pool_caches(cache):
    """The scored step and the eviction on the context's own caches give what they give on the caller's."""
    import torch
    from tests.gpu_util import device_view
    w, inp = ref.step_case(cache, "f16" if cache == "i8" else cache, 2, 8, 2, 128, 128, [100, 77])
    np_dt = {"bf16": np.int16, "i8": np.int8}[cache]
    res = []
    for own in (True, False):
        step = make_step(w, scored=True)
        kc, vc = dev(inp["k_cache"]), dev(inp["v_cache"])
        sc = dev(inp["scales"]) if cache == "i8" else None
        if own:
            kp, vp, sp = step.cache_ptrs()
            pk, pv = (device_view(p, inp["k_cache"].shape, np_dt) for p in (kp, vp))
            pk.copy_(kc), pv.copy_(vc)
            if sc is not None:
                ps = device_view(sp, inp["scales"].shape, np.float32)
                ps.copy_(sc)
                sc = ps
            kc, vc = pk, pv
        lens = dev(inp["seq_lens"])
        acc = torch.zeros((2, 2, 128), device="cuda")
        pos = torch.arange(128, dtype=torch.int32, device="cuda").expand(2, 2, 128).contiguous()
        out = torch.empty((2, 8, 128), device="cuda")
        kw = {} if own else dict(k_cache=kc, v_cache=vc, scales=sc)
        step.scored(dev(inp["q"]), dev(inp["k_new"]), dev(inp["v_new"]), lens, lens, acc, pos, out, bias=dev(inp["bias"]), **kw)
        lens += 1
        step.evict(acc, pos, lens, lens, lens, np.int64(50), recent=np.int64(10), **kw)
        torch.cuda.synchronize()
        assert step.get_error() == ftd.FTD_OK
        res.append([t.clone() for t in (out, acc, pos, lens, kc[:, :, :50], vc[:, :, :50])] + ([sc[:, :, :, :50].clone()] if sc is not None else []))
        step.close()
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_refusals():
    import torch
    w = Workload("evict", B=2, Hq=2, Hkv=2, D=64, Lmax=256, qkv_dtype="f16", cache_dtype="f16")
    a = torch.zeros((2, 2, 256), device="cuda")
    p = a.data_ptr()
    n = ftd.ftd_kernel_launches()

    def call(step, **kw):
        x = dict(k=0, v=0, scales=0, table=0, lens=256, next_pos=256, acc=p, acc_out=0, pos=p, pos_out=0, new=256,
                 budget=100, recent=10, sinks=4)
        x.update(kw)
        return ftd.ftd_cache_evict(step.ctx, x["k"], x["v"], x["scales"], x["table"], x["lens"], x["next_pos"], x["acc"],
                                   x["acc_out"], x["pos"], x["pos_out"], x["new"], x["budget"], x["recent"], x["sinks"], 0)
    step = make_step(w)
    assert call(step) == ftd.FTD_ERR_INVALID_ARG and "ftd_enable_scores" in ftd.ftd_last_error()
    step.enable_scores()
    for kw in (dict(lens=0), dict(next_pos=0), dict(acc=0), dict(pos=0), dict(new=0), dict(lens=258), dict(acc=p + 2),
               dict(pos=p + 1), dict(new=257), dict(next_pos=257), dict(budget=0), dict(budget=-1), dict(budget=257),
               dict(recent=-1), dict(sinks=-1), dict(recent=97), dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(k=264),
               dict(v=264), dict(table=256), dict(acc_out=p + 4), dict(pos_out=p + 4), dict(acc_out=p + 2),
               dict(new=260), dict(new=252)):
        assert call(step, **kw) == ftd.FTD_ERR_INVALID_ARG, kw
        assert ftd.ftd_last_error() != ""
    step.close()
    for opts in (dict(window=32), dict(page_size=128, num_pages=4)):
        step = make_step(w, scored=True, **opts)
        assert call(step) == ftd.FTD_ERR_INVALID_ARG, opts
        step.close()
    assert ftd.ftd_kernel_launches() == n


# ------------------------------------------------------------ together
@pytest.mark.parametrize("cache,Hq,Hkv,page", [("bf16", 8, 2, 0), ("f16", 4, 4, 128), ("i8", 16, 2, 128), ("f32", 2, 2, 0)])
def test_decoder_loop(cache, Hq, Hkv, page):
    """A decoder with a bounded cache: every step turns its query and key to the token's position,
    runs the scored step, attends to an encoder's states, and evicts when the cache is full.  The
    cache's rows, planes and positions are followed in numpy from the device's own planes, so a wrong
    row anywhere shows as a wrong output later."""
    import torch
    B, D, Lmax, budget, recent, sinks, M = 2, 128, 128 if not page else 256, 40, 8, 2, 70
    qkv = "f16" if cache == "i8" else cache
    td = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[qkv]
    w = Workload("loop", B=B, Hq=Hq, Hkv=Hkv, D=D, Lmax=Lmax, qkv_dtype=qkv, cache_dtype=cache)
    rng = np.random.default_rng(12)
    opts, table = {}, None
    if page:
        per = -(-Lmax // page)
        table = rng.permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
        opts = dict(page_size=page, num_pages=B * per + 1)
    step = make_step(w, scored=True, **opts)
    step.set_rope(2, [24, 40])
    wm = w.with_(Lmax=80)
    (km, vm), scm = rows_of(wm, rng)
    if scm is not None:
        scm *= 0.02
    mem = make_step(wm)
    shape = (B, Hkv, Lmax, D) if not page else (B * per + 1, Hkv, page, D)
    kc, vc = (torch.zeros(shape, dtype=torch.int8 if cache == "i8" else td, device="cuda") for _ in range(2))
    sc = torch.ones((2,) + shape[:3], device="cuda") if cache == "i8" else None
    acc, pos = torch.zeros(shape[:3], device="cuda"), torch.zeros(shape[:3], dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    npos = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    mlens = torch.tensor([M, 3], dtype=torch.int32, device="cuda")
    tb = dev(table) if page else None
    kmd, vmd, scd = dev(km), dev(vm), (dev(scm) if scm is not None else None)

    def plane(t):
        a = t.cpu().numpy() if t.dtype != torch.bfloat16 else t.view(torch.int16).cpu().numpy().view(np.uint16)
        return a if not page else from_pages(w, a, table, page, [Lmax] * B, q_len=0)

    def store(x):
        return dev(to_storage(x.astype(np.float32), qkv)).view(td) if qkv == "bf16" else dev(to_storage(x.astype(np.float32), qkv))
    evictions = 0
    for it in range(100):
        qkv_t = store(rng.standard_normal((B, (Hq + 2 * Hkv) * D)))
        bias = store(0.1 * rng.standard_normal((Hq + 2 * Hkv) * D))
        q, k, v = torch.empty((B, Hq, D), dtype=td, device="cuda"), *(torch.empty((B, Hkv, D), dtype=td, device="cuda") for _ in range(2))
        step.rope(qkv_t[:, :Hq * D], qkv_t[:, Hq * D:(Hq + Hkv) * D], qkv_t[:, (Hq + Hkv) * D:],
                  torch.stack([npos, npos // 2]).contiguous(), q, k, v, bias=bias)
        before = [plane(x) for x in (acc, pos)]
        L0, n0 = lens.tolist(), npos.tolist()
        out, cr = torch.empty((B, Hq, D), device="cuda"), torch.empty((B, Hq, D), device="cuda")
        step.scored(q, k, v, lens, npos, acc, pos, out, k_cache=kc, v_cache=vc, scales=sc, block_table=tb)
        mem.cross(q, mlens, cr, k_mem=kmd, v_mem=vmd, scales=scd)
        torch.cuda.synchronize()
        if it % 9 == 0 or it > 90:
            kh, vh = plane(kc), plane(vc)
            sh = np.stack([plane(sc[0]), plane(sc[1])]) if sc is not None else None
            qh = q.cpu().view(torch.int16).numpy().view(np.uint16) if qkv == "bf16" else q.cpu().numpy()
            inp = dict(q=qh, bias=None, seq_lens=np.array(L0))
            ah, ph = plane(acc), plane(pos)
            for b in range(B):
                n = L0[b] + 1
                add, mass = ref.added_weights(w, inp, kh, sh, b)
                want = add.copy()
                want[:, :L0[b]] += before[0][b, :, :L0[b]]
                assert np.all(np.abs(ah[b, :, :n] - want) <= add * ref.weight_tolerance(w, mass, False) + want * 2.0 ** -23)
                assert np.all(ph[b, :, L0[b]] == n0[b])
                p, _ = ref.weights(w, ref.queries(w, inp, b)[0], ref.cache_rows(w, kh, sh, 0, b, n), 0, n)
                vv = np.repeat(ref.cache_rows(w, vh, sh, 1, b, n), Hq // Hkv, axis=0)
                assert_close(out[b].double().cpu().numpy(), np.einsum("hn,hnd->hd", p, vv), i8=cache == "i8")
            assert_close(cr.double().cpu().numpy(), ref.cross(wm, qh[:, None], None, km, vm, scm, [M, 3])[:, 0], i8=cache == "i8")
        lens += 1
        npos += 1
        if int(lens.max()) == 60:  # full: every head down to the budget
            evictions += 1
            planes = [plane(x) for x in (kc, vc, acc, pos)] + ([plane(sc[0]), plane(sc[1])] if sc is not None else [])
            new = ref.evict(planes, planes[2].copy(), planes[3].copy(), lens.cpu().numpy(), npos.cpu().numpy(), budget, recent, sinks)
            step.evict(acc, pos, lens, npos, lens, budget, recent=recent, sinks=sinks, k_cache=kc, v_cache=vc, scales=sc,
                       block_table=tb)
            torch.cuda.synchronize()
            assert lens.tolist() == new.tolist() == [budget] * B
            now = [plane(x) for x in (kc, vc, acc, pos)] + ([plane(sc[0]), plane(sc[1])] if sc is not None else [])
            for a, b in zip(now, planes):
                assert_same_bytes(a[:, :, :60], b[:, :, :60], "after eviction")
    assert evictions == 3
    assert step.get_error() == ftd.FTD_OK and mem.get_error() == ftd.FTD_OK
    step.close()
    mem.close()
