"""ftd_rope_qkv refuses an output that overlaps the positions of any axis, the last one's among them."""
import pytest

import decode_step_masked_gb300 as ftd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_outputs_over_any_axis_are_refused(axes):
    import torch
    ftd.build_library()
    n, hq, hkv, d = 8, 4, 2, 64
    step = ftd.DecodeStep(1, hq, hkv, d, 16, "f16", "f16")
    step.set_rope(axes, [32 * (a + 1) // axes - 32 * a // axes for a in range(axes)])
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    src = torch.zeros(n * (hq + 2 * hkv) * d, dtype=torch.float16, device="cuda")
    q, k, v = (src.data_ptr() + 2 * n * d * h for h in (0, hq, hq + hkv))
    base = buf.data_ptr() + 4096  # (positions below it stay inside the buffer)
    qo, ko, vo = (base + 2 * n * d * h for h in (0, hq, hq + hkv))
    end = base + 2 * n * d * (hq + 2 * hkv)  # the outputs are [base, end)
    launches = ftd.ftd_kernel_launches()

    def call(positions):
        return ftd.ftd_rope_qkv(step.ctx, q, k, v, 0, 0, 0, positions, n, qo, ko, vo, 0)
    for a in range(axes):
        # axis a's last entry on the outputs' first bytes, and its first entry on their last ones
        for positions in (qo + 4 - 4 * n * (a + 1), end - 4 - 4 * n * a):
            assert call(positions) == ftd.FTD_ERR_INVALID_ARG and "positions" in ftd.ftd_last_error(), a
    assert ftd.ftd_kernel_launches() == launches
    assert call(base - 4 * n * axes) == ftd.FTD_OK and call(end) == ftd.FTD_OK  # just below and just behind them
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    step.close()
