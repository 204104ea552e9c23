"""ftd_cross_mha against attention in 64 bits: every cache type and kernel, grouped heads,
beams, memory lengths from none to full, rows past a memory poisoned, and the refusals."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from synthetic import to_storage
from tests import operators_ref as ref
from tests.gpu_util import TOL_MAXABS, TOL_MAXABS_I8, TORCH_OUT, assert_close, assert_same_bytes, dev, host, make_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


def case(cache, qkv, B, Hq, Hkv, D, Lmax, lens, T=1, seed=41):
    w, inp = ref.step_case(cache, qkv, B, Hq, Hkv, D, Lmax, lens, T=T, seed=seed)
    rng = np.random.default_rng(seed + 1)
    inp["q_bias"] = to_storage(0.1 * rng.standard_normal(Hq * D).astype(np.float32), qkv)
    return w, inp


def run(w, inp, bias=True, out_dtype="f32", cuda_core=False, step=None):
    import torch
    own = step is None
    if own:
        step = make_step(w, force_cuda_core=cuda_core, out_dtype=out_dtype, q_len=w.q_len)
    q, kc, vc, sl = (dev(inp[x]) for x in ("q", "k_cache", "v_cache", "seq_lens"))
    sc = dev(inp["scales"]) if inp.get("scales") is not None else None
    out = torch.full((w.B, w.q_len, w.Hq, w.D), float("nan"), dtype=getattr(torch, TORCH_OUT[out_dtype]), device="cuda")
    before = ftd.ftd_kernel_launches()
    step.cross(q, sl, out, q_bias=dev(inp["q_bias"]) if bias else None, k_mem=kc, v_mem=vc, scales=sc)
    torch.cuda.synchronize()
    assert ftd.ftd_kernel_launches() == before + 1
    status = step.get_error()
    assert_same_bytes(host(kc, inp["k_cache"]), inp["k_cache"], "K memory")  # read only
    assert_same_bytes(host(vc, inp["v_cache"]), inp["v_cache"], "V memory")
    if own:
        step.close()
    return out.double().cpu().numpy(), status


def expect(w, inp, bias=True):
    q = inp["q"].reshape(w.B, w.q_len, w.Hq, w.D)
    return ref.cross(w, q, inp["q_bias"] if bias else None, inp["k_cache"], inp["v_cache"], inp.get("scales"),
                     inp["seq_lens"])


SHAPES = {
    "mha_bf16": ("bf16", "bf16", 8, 8, 128, False),
    "mha_f16_d64": ("f16", "f16", 4, 4, 64, False),
    "mha_f32": ("f32", "f32", 4, 4, 64, False),
    "mha_i8": ("i8", "f16", 8, 8, 128, False),
    "gqa_i8_d64": ("i8", "bf16", 8, 2, 64, False),
    "odd_group": ("bf16", "f32", 9, 3, 128, False),
    "gqa4_tc": ("bf16", "bf16", 16, 4, 128, False),
    "gqa8_tc": ("f16", "f16", 16, 2, 128, False),
    "gqa16_tc": ("bf16", "bf16", 32, 2, 128, False),
    "gqa8_tc_i8": ("i8", "f16", 16, 2, 128, False),
    "gqa8_cc": ("bf16", "bf16", 16, 2, 128, True),
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
LENS = [0, 1, 2, 31, 127, 128, 129, 500, -3, 640]


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("T", [1, 3, 4])
def test_shapes(shape, T):
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    if Hq * T > 200:
        T = 2 if T > 1 else 1
    w, inp = case(cache, qkv, len(LENS), Hq, Hkv, D, 640, LENS, T=T)
    got, status = run(w, inp, cuda_core=cc)
    assert status == ftd.FTD_OK
    want = expect(w, inp)
    assert_close(got, want, i8=cache == "i8", what=shape)
    for b, n in enumerate(LENS):
        if n <= 0:
            assert not got[b].any(), f"slot {b} without a memory"


@pytest.mark.parametrize("cache", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,T", [(64, 1, 1), (32, 1, 1), (64, 2, 1), (64, 1, 3), (16, 1, 2)])
def test_wide_and_narrow_blocks(cache, Hq, Hkv, T):
    """Multiples of 32 query rows: in 64- or 32-row blocks where the memories hold more tiles than SMs, else in
    16-row blocks."""
    for B, Lmax in ((3, 1024), (20, 1280), (40, 2048)):
        lens = np.random.default_rng(B).integers(0, Lmax + 1, B)
        if B == 40:
            lens = lens // 16
        w, inp = case(cache, cache, B, Hq, Hkv, 128, Lmax, lens, T=T)
        got, status = run(w, inp)
        assert status == ftd.FTD_OK
        assert_close(got, expect(w, inp), what=f"B {B}")


@pytest.mark.parametrize("out_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", ["mha_bf16", "gqa8_tc", "gqa8_tc_i8", "wide64"])
def test_half_output_without_bias(shape, out_dtype):
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = case(cache, qkv, 3, Hq, Hkv, D, 256, [200, 0, 77])
    got, _ = run(w, inp, bias=False, out_dtype=out_dtype, cuda_core=cc)
    want = expect(w, inp, bias=False)
    tol = (TOL_MAXABS_I8 if cache == "i8" else TOL_MAXABS) + np.abs(want) * ref.HALF_STEP[out_dtype]
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("shape", ["mha_bf16", "mha_f32", "gqa8_tc", "gqa8_tc_i8", "wide32", "gqa8_d64", "gqa8_i8_d64"])
def test_long_memory_split_over_blocks(shape):
    """One long memory and a short one: many pieces per segment, joined at the end."""
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = case(cache, qkv, 2, Hq, Hkv, D, 8192, [8191, 5], T=2)
    got, status = run(w, inp, cuda_core=cc)
    assert status == ftd.FTD_OK
    assert_close(got, expect(w, inp), i8=cache == "i8", what=shape)


@pytest.mark.parametrize("shape", ["mha_bf16", "gqa8_tc", "wide32", "gqa8_tc_i8"])
def test_too_long_memory_is_skipped_and_reported(shape):
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = case(cache, qkv, 3, Hq, Hkv, D, 256, [256, 256, 256], T=4)
    inp["seq_lens"][:] = [256, 257, 2 ** 31 - 1]
    got, status = run(w, inp, cuda_core=cc)
    assert status == ftd.FTD_ERR_SEQ_OVERFLOW
    assert not got[1:].any()
    assert_close(got[:1], expect(w, inp)[:1], i8=cache == "i8", what=shape)


@pytest.mark.parametrize("shape", ["wide32", "wide64", "two_wide"])
@pytest.mark.parametrize("T", [1, 2])
def test_wide_lengths(shape, T):
    """The edge lengths on the wide kernel (memories long enough for its blocks)."""
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    w, inp = case(cache, qkv, len(LENS), Hq, Hkv, D, 2560, LENS, T=T)
    got, status = run(w, inp)
    assert status == ftd.FTD_OK
    assert_close(got, expect(w, inp), what=shape)


@pytest.mark.parametrize("shape", ["gqa8_tc", "gqa16_tc", "mha_bf16", "wide32"])
def test_large_batches(shape):
    """Up to the largest batch: past 788 slots the 16-row blocks' split has no room for its weights."""
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    for B in (788, 789, 1024):
        lens = np.random.default_rng(B).integers(0, 33, B)
        lens[7], lens[B - 1] = 32, 0
        w, inp = case(cache, qkv, B, Hq // Hkv, 1, D, 32, lens)
        got, status = run(w, inp, cuda_core=cc)
        assert status == ftd.FTD_OK
        assert_close(got, expect(w, inp), what=f"{shape} B {B}")


def test_every_memory_empty():
    import torch
    w, inp = case("bf16", "bf16", 4, 8, 1, 128, 128, [0, 0, 0, 0])
    inp["seq_lens"][:] = [0, -1, 0, -2 ** 31]
    got, status = run(w, inp)
    assert status == ftd.FTD_OK and not got.any()


def test_pool_memory_graph_and_late_lengths():
    """The context's own pool as memory, a captured call replayed with other lengths, and lengths
    written by the kernel before the call."""
    import torch
    from tests.gpu_util import device_view
    w, inp = case("f16", "f16", 3, 16, 2, 128, 512, [512, 512, 512], T=2)
    step = make_step(w, q_len=2)
    kp, vp, _ = step.cache_ptrs()
    for ptr, name in ((kp, "k_cache"), (vp, "v_cache")):
        device_view(ptr, inp[name].shape, np.float16).copy_(dev(inp[name]))
    q, bias = dev(inp["q"]), dev(inp["q_bias"])
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.empty((3, 2, 16, 128), device="cuda")
    step.cross(q, lens, out, q_bias=bias)
    torch.cuda.synchronize()
    assert not out.any()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.cross(q, lens, out, q_bias=bias)
    for ls in ([512, 0, 33], [1, 400, 128]):
        lens.copy_(torch.tensor(ls, dtype=torch.int32))
        inp["seq_lens"][:] = ls
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert_close(out.double().cpu().numpy(), expect(w, inp), what=str(ls))
    src = torch.tensor([300, 511, 2], dtype=torch.int32, device="cuda")
    inp["seq_lens"][:] = [300, 511, 2]
    s = torch.cuda.current_stream().cuda_stream
    assert ftd.ftd_debug_late_lengths(src.data_ptr(), lens.data_ptr(), 3, 300, s) == ftd.FTD_OK
    step.cross(q, lens, out, q_bias=bias)
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    assert_close(out.double().cpu().numpy(), expect(w, inp), what="late lengths")
    step.close()


def test_step_and_cross_share_a_context():
    """A step after a cross call on the same context gives the step's bytes."""
    import torch
    w, inp = case("bf16", "bf16", 3, 16, 2, 128, 256, [200, 3, 17])
    step = make_step(w)
    q, kn, vn, b, sl = (dev(inp[x]) for x in ("q", "k_new", "v_new", "bias", "seq_lens"))
    outs = []
    for i in range(2):
        kc, vc = dev(inp["k_cache"]), dev(inp["v_cache"])
        out = torch.empty((3, 16, 128), device="cuda")
        if i:
            step.cross(q, sl, torch.empty_like(out), k_mem=dev(inp["k_cache"]), v_mem=dev(inp["v_cache"]))
        step(q, kn, vn, sl, out, bias=b, k_cache=kc, v_cache=vc)
        torch.cuda.synchronize()
        outs.append(out)
    assert step.get_error() == ftd.FTD_OK
    assert torch.equal(outs[0], outs[1])
    step.close()


@pytest.mark.parametrize("shape", ["mha_f16_d64", "mha_i8", "gqa8_tc", "gqa8_tc_i8", "gqa8_d64", "wide32", "wide64"])
def test_withheld_copy_times_out_and_the_next_call_is_right(shape):
    """Bounded waits: block 0's first copy is never issued, the call reports it, the next ones are whole."""
    import torch
    cache, qkv, Hq, Hkv, D, cc = SHAPES[shape]
    # (long memories, of which little is used, for the wide kernel's blocks)
    w, inp = case(cache, qkv, 2, Hq, Hkv, D, 12288 if shape.startswith("wide") else 512, [500, 130], T=2)
    step = make_step(w, q_len=2, wait_limit_us=2000)
    d = {x: dev(inp[x]) for x in ("q", "k_cache", "v_cache", "seq_lens", "q_bias")}
    sc = dev(inp["scales"]) if inp.get("scales") is not None else None
    out = torch.empty((2, 2, Hq, D), device="cuda")
    call = lambda: step.cross(d["q"], d["seq_lens"], out, q_bias=d["q_bias"], k_mem=d["k_cache"],  # noqa: E731
                              v_mem=d["v_cache"], scales=sc)
    assert ftd.ftd_debug_stall_next(step.ctx, 1) == ftd.FTD_OK
    call()
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_ERR_DEVICE_TIMEOUT
    for _ in range(2):
        call()
        torch.cuda.synchronize()
        assert step.get_error() == ftd.FTD_OK
        assert_close(out.double().cpu().numpy(), expect(w, inp), i8=cache == "i8", what=shape)
    step.close()


def test_refusals():
    w, _ = case("bf16", "bf16", 2, 8, 8, 128, 256, [1, 1])
    n = ftd.ftd_kernel_launches()
    for opts in (dict(window=64), dict(page_size=128, num_pages=4)):
        step = make_step(w, **opts)
        assert ftd.ftd_cross_mha(step.ctx, 256, 0, 0, 0, 256, 0, 256, 0) == ftd.FTD_ERR_INVALID_ARG
        step.close()
    step = make_step(w)
    ok = dict(q=256, bias=0, k=256, v=256, lens=256, scales=0, out=256)
    for bad in (dict(q=0), dict(lens=0), dict(out=0), dict(q=257), dict(bias=257), dict(k=264), dict(v=264),
                dict(out=264), dict(lens=258)):
        a = dict(ok, **bad)
        st = ftd.ftd_cross_mha(step.ctx, a["q"], a["bias"], a["k"], a["v"], a["lens"], a["scales"], a["out"], 0)
        assert st == ftd.FTD_ERR_INVALID_ARG and ftd.ftd_last_error(), bad
    step.close()
    assert ftd.ftd_kernel_launches() == n
