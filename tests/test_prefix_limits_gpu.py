"""The longest prefix that the kernels' tile counts hold."""
import pytest

import decode_step_masked_gb300 as ftd

pytestmark = pytest.mark.gpu


# blocks of 64 query rows on CUDA cores, of 256 on the tensor cores, 128 with q as a pair
@pytest.mark.parametrize("qkv,cache,block", [("f32", "f32", 64), ("bf16", "bf16", 256), ("f32", "bf16", 128), ("f16", "i8", 256)])
def test_tiles_that_pass_31_bits_are_refused(qkv, cache, block):
    import torch
    ftd.build_library()
    B, Hq, D = 1024, 32, 64  # 32768 query rows of one kv head
    step = ftd.DecodeStep(B, Hq, 1, D, 128, qkv, cache, page_size=128, num_pages=4)
    step.enable_prefix()
    z = lambda *s: torch.zeros(s, dtype=torch.float32, device="cuda")  # noqa: E731
    q, kv, out = z(B, Hq, D), z(B, 1, D), z(B, Hq, D)
    lens = torch.full((B,), -1, dtype=torch.int32, device="cuda")  # no slot works, and none sees anything
    table, pre = torch.zeros((B, 1), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(rows):
        return ftd.ftd_decode_mha_prefix(step.ctx, q.data_ptr(), kv.data_ptr(), kv.data_ptr(), 0, 0, 0, table.data_ptr(), lens.data_ptr(), 0,
                                         0, 0, 0, pre.data_ptr(), rows, lens.data_ptr(), out.data_ptr(), 0)

    tiles = (1 << 31) // (B * Hq // block)
    n = ftd.ftd_kernel_launches()
    for rows in (64 * tiles, 64 * tiles - 63, (1 << 31) - 1):
        if rows < 1 << 31:
            assert call(rows) == ftd.FTD_ERR_INVALID_ARG
            assert "prefix_rows" in ftd.ftd_last_error()
    assert ftd.ftd_kernel_launches() == n
    assert call(64 * tiles - 64) == ftd.FTD_OK
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK and not out.any()
    step.close()
