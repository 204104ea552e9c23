"""Which kernel the scored step and cross attention take, and the wide kernel's paths that only long
contexts or large batches reach: references that move all along a context, queries without a bias,
memories that are too long, half outputs."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from tests import operators_ref as ref
from tests import test_cross_gpu as cross
from tests import test_scored_gpu as scored
from tests.gpu_util import TOL_MAXABS, assert_close, make_step, rising_scores

pytestmark = pytest.mark.gpu
STEP, SCORED, CROSS = 0, 1, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


def choice(step, entry):
    st, rows, tc = ftd.ftd_debug_kernel(step.ctx, entry)
    assert st == ftd.FTD_OK
    return rows, tc


# cache, query heads, kv heads, head_dim, tokens, batch, max_len -> (rows, tensor cores) of the step and of the other two
CHOICES = [
    ("bf16", 8, 8, 128, 1, 10, 640, (1, False), (1, False)),
    ("bf16", 8, 8, 128, 3, 10, 640, (1, False), (3, True)),
    ("f16", 16, 8, 128, 1, 10, 640, (2, False), (2, False)),
    ("f32", 8, 1, 128, 1, 4, 640, (8, False), (8, False)),
    ("f16", 4, 4, 64, 4, 10, 640, (4, False), (4, True)),
    ("bf16", 16, 4, 128, 1, 10, 640, (4, True), (4, True)),
    ("bf16", 14, 2, 128, 1, 10, 640, (1, False), (7, True)),
    ("f16", 17, 1, 128, 1, 10, 640, (1, False), (1, False)),
    ("bf16", 32, 2, 128, 1, 10, 640, (16, True), (16, True)),
    ("i8", 8, 8, 128, 3, 10, 640, (1, False), (1, False)),
    ("i8", 8, 2, 128, 1, 10, 640, (4, False), (4, True)),
    ("i8", 8, 2, 64, 1, 10, 640, (4, False), (4, False)),
    ("i8", 16, 2, 64, 1, 10, 640, (8, False), (8, True)),
    ("i8", 16, 2, 128, 1, 10, 640, (8, True), (8, True)),
    # the wide kernel, unless a context's tiles of 128 positions are no more than the SMs
    ("f16", 32, 1, 128, 1, 10, 640, (32, True), (16, True)),
    ("f16", 64, 1, 128, 1, 10, 640, (64, True), (16, True)),
    ("f16", 64, 1, 128, 1, 10, 2048, (64, True), (64, True)),
    ("f16", 32, 1, 128, 1, 10, 2048, (32, True), (32, True)),
    ("bf16", 128, 1, 128, 1, 10, 1024, (64, True), (64, True)),
    ("bf16", 64, 2, 64, 1, 40, 2048, (8, False), (16, True)),
]


@pytest.mark.parametrize("case", CHOICES, ids=lambda c: "-".join(map(str, c[:7])))
def test_choices(case):
    cache, Hq, Hkv, D, T, B, Lmax, step_choice, other = case
    step = ftd.DecodeStep(B, Hq, Hkv, D, Lmax, "f16" if cache == "i8" else cache, cache, q_len=T)
    assert choice(step, STEP) == step_choice
    assert choice(step, SCORED) == choice(step, CROSS) == other
    step.close()
    step = ftd.DecodeStep(B, Hq, Hkv, D, Lmax, "f16" if cache == "i8" else cache, cache, q_len=T, kernel=ftd.FTD_KERNEL_CUDA_CORE)
    assert not any(choice(step, e)[1] for e in (STEP, SCORED, CROSS))
    step.close()


def test_refusals():
    step = ftd.DecodeStep(1, 2, 2, 64, 16, "f16", "f16")
    for e in (-1, 3):
        assert ftd.ftd_debug_kernel(step.ctx, e)[0] == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_debug_kernel(0, 0)[0] == ftd.FTD_ERR_INVALID_ARG
    step.close()


WIDE = {"wide32": ("bf16", 32, 1, 32), "wide64": ("f16", 64, 1, 64), "two_wide": ("bf16", 128, 1, 64)}


def wide_case(shape, lens, Lmax, T=1, entry=SCORED, **opts):
    """A case with more tiles than SMs, and its context, on the wide kernel's blocks."""
    cache, Hq, Hkv, rows = WIDE[shape]
    if entry == SCORED:
        w, inp = ref.step_case(cache, cache, len(lens), Hq, Hkv, 128, Lmax, lens, T=T)
    else:
        w, inp = cross.case(cache, cache, len(lens), Hq, Hkv, 128, Lmax, lens, T=T)
    step = make_step(w, q_len=T, scored=entry == SCORED, **opts)
    assert choice(step, entry) == (64 if Hq * T // Hkv % 64 == 0 else rows, True)
    return w, inp, step


@pytest.mark.parametrize("shape", list(WIDE))
@pytest.mark.parametrize("T", [1, 2])
def test_rising_scores(shape, T):
    """Every row's reference moves again and again inside a block's tiles: O is rescaled, the scores read once more."""
    w, inp, step = wide_case(shape, [8190, 4000, 700], 8192, T=T)
    scored.check(w, rising_scores(w, inp), step=step)
    step.close()


@pytest.mark.parametrize("shape", list(WIDE))
def test_weights_without_bias(shape):
    w, inp, step = wide_case(shape, [5000, 200, 7, 128], 6400)
    scored.run(w, inp, bias=False, step=step)
    step.close()


@pytest.mark.parametrize("shape", list(WIDE))
def test_slots_without_work(shape):
    """Inactive and overflowing slots among the others, one and several tokens."""
    for T in (1, 3):
        if WIDE[shape][1] * T > 200:
            continue
        w, inp, step = wide_case(shape, [-1, 6400, 100, 6400 - T, 6401], 6400, T=T)
        scored.check(w, inp, step=step)
        step.close()


@pytest.mark.parametrize("shape", list(WIDE))
@pytest.mark.parametrize("T", [1, 4])
def test_too_long_memory_is_skipped_and_reported(shape, T):
    T = 1 if WIDE[shape][1] * T > 256 else T
    w, inp, step = wide_case(shape, [6400, 6400, 6400, 90], 6400, T=T, entry=CROSS)
    inp["seq_lens"][:] = [6400, 6401, 2 ** 31 - 1, 90]
    got, status = cross.run(w, inp, step=step)
    assert status == ftd.FTD_ERR_SEQ_OVERFLOW
    assert not got[1:3].any()
    want = cross.expect(w, inp)
    assert_close(got[[0, 3]], want[[0, 3]], what=shape)
    step.close()


@pytest.mark.parametrize("out_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", list(WIDE))
def test_half_output_without_bias(shape, out_dtype):
    w, inp, step = wide_case(shape, [6000, 0, 77], 6656, entry=CROSS, out_dtype=out_dtype)
    got, _ = cross.run(w, inp, bias=False, out_dtype=out_dtype, step=step)
    want = cross.expect(w, inp, bias=False)
    assert np.all(np.abs(got - want) <= TOL_MAXABS + np.abs(want) * ref.HALF_STEP[out_dtype])
    step.close()
