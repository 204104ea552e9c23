"""Rows appended by the step behind a shared prefix are the step's own, bit for bit, INT8 ones the scored step's."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from tests import operators_ref as ref
from tests.gpu_util import assert_same_bytes, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


@pytest.mark.parametrize("cache,qkv", [("i8", "f16"), ("i8", "bf16"), ("i8", "f32"), ("bf16", "f32"), ("f16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("Hq,Hkv,D,T", [(4, 4, 128, 1), (16, 2, 128, 1), (8, 2, 64, 2), (8, 8, 64, 1)])
@pytest.mark.parametrize("bias", [None, 0.1])
def test_appended_rows(cache, qkv, Hq, Hkv, D, T, bias):
    import torch
    B, Lmax, P = 48, 160, 200
    w, inp = ref.step_case(cache, qkv, B, Hq, Hkv, D, Lmax, [(7 * b) % 150 for b in range(B)], T=T, bias=bias)
    args = [dev(inp[x]) for x in ("q", "k_new", "v_new", "seq_lens")]
    storage = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}[cache]
    pre = torch.zeros((Hkv, P, D), dtype=storage, device="cuda")
    psc = torch.ones((2, Hkv, P), device="cuda") if cache == "i8" else None
    after = []
    for shared in (False, True):
        step = ftd.DecodeStep(B, Hq, Hkv, D, Lmax, qkv, cache, q_len=T)
        kc, vc = dev(inp["k_cache"]), dev(inp["v_cache"])
        sc = dev(inp["scales"]) if cache == "i8" else None
        out = torch.empty((B, T, Hq, D), device="cuda")
        kw = dict(bias=dev(inp["bias"]) if bias else None, k_cache=kc, v_cache=vc, scales=sc)
        if shared:
            step.enable_prefix()
            step.prefix(*args, dev(np.full(B, P, np.int32)), out, k_prefix=pre, v_prefix=pre.clone(), prefix_scales=psc, **kw)
        else:
            step(*args, out, **kw)
        torch.cuda.synchronize()
        assert step.get_error() == ftd.FTD_OK
        after.append((host(kc, inp["k_cache"]), host(vc, inp["v_cache"]), None if sc is None else sc.cpu().numpy()))
        step.close()
    (k, v, scales), got = after
    if cache == "i8":
        for b, L in enumerate(inp["seq_lens"]):
            for i, (x, n) in enumerate(((k, "k"), (v, "v"))):
                x[b, :, L:L + T], scales[i, b, :, L:L + T] = ref.appended_i8(w, inp, b, n)
        assert_same_bytes(got[2], scales, "scales")
    assert_same_bytes(got[0], k, "K")
    assert_same_bytes(got[1], v, "V")
