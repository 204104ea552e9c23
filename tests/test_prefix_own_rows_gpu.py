"""The slots' own rows where the prefix's kernel takes them: references that move from tile to tile, and a copy that never
comes."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from synthetic import to_storage
from tests import operators_ref as ref
from tests.gpu_util import make_step
from tests.test_prefix_gpu import case, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


def lengths(B, lmax, T):
    return [0, lmax - T, 129, -1] + [int(x) for x in np.random.default_rng(B).integers(0, lmax - T + 1, B - 4)]


@pytest.mark.parametrize("cache,out,D", [("bf16", "bf16", 128), ("f16", "f16", 64), ("f16", "f32", 128), ("bf16", "f32", 64)])
@pytest.mark.parametrize("heavy", [4.0, 30.0, -30.0])
@pytest.mark.parametrize("B,T", [(40, 1), (5, 1)])
def test_rising_scores(cache, out, D, heavy, B, T):
    """Own keys that grow along a slot's rows (or shrink), in segments of one tile to eight, several of them a block's."""
    lmax, P = 1024, 300
    lens = lengths(B, lmax, T)
    w, inp = case(cache, cache, B, 48, 2, D, lmax, lens, P, [P - 7 * (b % 5) for b in range(B)], T=T)
    grow = 1.0 + heavy * (np.arange(lmax) if heavy > 0 else np.arange(lmax) - lmax) / lmax
    x = ref.widen(inp["k_cache"], cache)
    inp["k_cache"] = np.where(np.isnan(x), inp["k_cache"], to_storage((np.nan_to_num(x) * grow[:, None]).astype(np.float32), cache))
    run(w, inp, out_dtype=out, bias=out == "f32")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("B", [4, 64])
def test_waits_that_run_out(out, B):
    """Slots that see nothing of the prefix, so that the copy that is withheld, block 0's first, is of an own tile: the bounded waits give
    up, the error is reported, and the next call is right.  With one tile a block, and with several under way."""
    lmax = 1024
    w, inp = case("bf16", "bf16", B, 48, 2, 128, lmax, lengths(B, lmax, 1), 200, [0] * B, bias=None)
    step = make_step(w, out_dtype=out, wait_limit_us=2000)
    step.enable_prefix()
    run(w, inp, out_dtype=out, step=step)
    assert ftd.ftd_debug_stall_next(step.ctx, 1) == ftd.FTD_OK
    run(w, inp, out_dtype=out, step=step, status=ftd.FTD_ERR_DEVICE_TIMEOUT, values=False)
    run(w, inp, out_dtype=out, step=step)
    step.close()


@pytest.mark.parametrize("group,T", [(1, 1), (3, 1), (4, 1), (5, 1), (7, 1), (8, 1), (3, 3), (11, 1), (12, 1), (7, 2), (5, 3), (16, 1), (1, 13)])
@pytest.mark.parametrize("cache,qkv,D,page", [("bf16", "bf16", 128, 0), ("f16", "f16", 64, 128), ("bf16", "f32", 64, 0), ("f16", "f16", 128, 256)])
def test_by_the_steps_kernel(group, T, cache, qkv, D, page):
    """Few query rows a slot and enough own rows that the step's kernel takes them beside the prefix."""
    B, lmax = 40, 1024
    lens = lengths(B, lmax, T)
    w, inp = case(cache, qkv, B, 2 * group, 2, D, lmax, lens, 300, [300 - 7 * (b % 5) for b in range(B)], T=T)
    run(w, inp, page=page)
    run(w, inp, out_dtype="bf16" if qkv == "f32" else qkv, page=page, bias=False)
