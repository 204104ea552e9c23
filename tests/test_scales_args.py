"""INT8 scales that hold more than the context's two planes: the second plane has to begin where the kernels look for it.
Needs no GPU."""
import torch

from tests.test_prefix_args import step_args
from tests.test_serving_args import B, D, HKV, HQ, LMAX, T, check, f16, i32, make  # noqa: F401 (make is a fixture)

SCALES = lambda *s: torch.zeros(s)  # noqa: E731


def cases(planes):
    """Scales that begin with [2][planes][HKV][rows], and those whose second plane lies elsewhere."""
    n, rows = planes
    good = [SCALES(2, n, HKV, rows), SCALES(3, n, HKV, rows), SCALES(2 * n * HKV * rows), SCALES(3 * n * HKV * rows)]
    bad = [SCALES(2, n + 1, HKV, rows), SCALES(2, n, HKV, rows + 16), SCALES(2, n, HKV + 1, rows), SCALES(1, n, HKV, rows)]
    return [dict(scales=s) for s in good], [dict(scales=s) for s in bad]


def test_norm_rope(make):  # noqa: F811
    n = 5
    args = dict(q=f16(n, HQ, D), k=f16(n, HKV, D), v=f16(n, HKV, D), positions=i32(2, n), q_out=f16(n, HQ, D), slots=i32(n))
    check(make("i8").norm_rope, args, *cases((B, LMAX)))
    check(make("i8", max_len=256, page_size=128, num_pages=7).norm_rope, args, *cases((7, 128)))


def test_prefix(make):  # noqa: F811
    codes = torch.zeros((HKV, 70, D), dtype=torch.int8)
    check(make("i8").prefix, dict(step_args(), k_prefix=codes, v_prefix=codes, prefix_scales=SCALES(2, HKV, 70)), *cases((B, LMAX)))
    check(make("i8", max_len=256, page_size=128, num_pages=7).prefix,
          dict(step_args(), k_prefix=None, v_prefix=None, block_table=i32(B, 2), prefix_table=i32(3)), *cases((7, 128)))


def test_larger_rows_of_heads(make):  # noqa: F811
    """Buffers kept for larger batches, however their rows are cut."""
    check(make().prefix, step_args(), [dict(q=f16(B + 1, T * HQ * D)), dict(k_new=f16((B + 1) * T, HKV * D)), dict(out=torch.zeros(B + 2, T, HQ * D))], [])
