"""A prefix that lies in what the same call writes is refused on the host, before any launch."""
import pytest

import decode_step_masked_gb300 as ftd
from tests.gpu_util import device_view

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "i8"])
@pytest.mark.parametrize("pool", [False, True])
def test_refused(cache, pool):
    import torch
    ftd.build_library()
    B, D, lmax, P = 3, 64, 64, 40
    step = ftd.DecodeStep(B, 2, 1, D, lmax, "bf16", cache)
    step.enable_prefix()
    dt, np_dt, i8 = (torch.int8, "int8", True) if cache == "i8" else (torch.bfloat16, "int16", False)
    if pool:
        k, v, s = step.cache_ptrs()
        kc, vc = (device_view(x, (B, 1, lmax, D), np_dt) for x in (k, v))
        sc = device_view(s, (2, B, 1, lmax), "float32") if i8 else None
    else:
        kc, vc = (torch.zeros((B, 1, lmax, D), dtype=dt, device="cuda") for _ in range(2))
        sc = torch.ones((2, B, 1, lmax), device="cuda") if i8 else None
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    apart = torch.zeros((1, P, D), dtype=kc.dtype, device="cuda")
    good_sc = torch.ones((2, 1, P), device="cuda") if i8 else None
    args = (z(B, 2, D), z(B, 1, D), z(B, 1, D), i(3, 0, -1), i(P, P, P), torch.zeros((B, 2, D), device="cuda"))
    kw = dict(k_prefix=apart, v_prefix=apart, prefix_scales=good_sc)
    if not pool:
        kw.update(k_cache=kc, v_cache=vc, scales=sc)
    ends = apart.new_zeros(kc.numel() + P * D)
    bad = [dict(k_prefix=kc[2, :, :P]), dict(v_prefix=kc[0, :, lmax - P:]), dict(k_prefix=vc[1, :, 8:8 + P]), dict(v_prefix=vc[2, :, :P])]
    few = args[5].view(kc.dtype).view(1, -1, D)  # out as rows of the cache type
    rows = few.shape[1]
    bad += [dict(k_prefix=few, v_prefix=apart[:, :rows], prefix_scales=good_sc[:, :, :rows].contiguous() if i8 else None)]
    if not pool:  # the prefix's last row, or the cache's
        bad += [dict(k_cache=ends[:kc.numel()].view_as(kc), k_prefix=ends[kc.numel() - D:kc.numel() - D + P * D].view(1, P, D))]
    if i8:
        bad += [dict(prefix_scales=sc.view(-1)[8:8 + 2 * P].view(2, 1, P))]
    n = ftd.ftd_kernel_launches()
    for b in bad:
        with pytest.raises(ftd.FtdError, match="overlaps"):
            step.prefix(*args, **dict(kw, **b))
    assert ftd.ftd_kernel_launches() == n
    good = [{}]
    if not pool:  # next to each other
        good += [dict(k_cache=ends[:kc.numel()].view_as(kc), k_prefix=ends[kc.numel():].view(1, P, D))]
    for g in good:
        step.prefix(*args, **dict(kw, **g))
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    step.close()
