"""What DecodeStep.prefix refuses of the step's own tensors before the library is called.  Needs no GPU."""
import pytest
import torch

from tests.test_serving_args import B, D, HKV, HQ, LMAX, T, check, f16, i32, make  # noqa: F401 (make is a fixture)


def step_args(out=torch.float32, qkv=torch.float16):
    return dict(q=torch.zeros(B, T, HQ, D, dtype=qkv), k_new=torch.zeros(B, T, HKV, D, dtype=qkv), v_new=torch.zeros(B, T, HKV, D, dtype=qkv),
                seq_lens=i32(B), prefix_lens=i32(B), out=torch.zeros(B, T, HQ, D, dtype=out), k_prefix=f16(HKV, 70, D), v_prefix=f16(HKV, 70, D))


def test_types_and_sizes(make):  # noqa: F811
    cache = f16(B, HKV, LMAX, D)
    check(make().prefix, step_args(),
          [dict(q=f16(B * T, HQ * D)), dict(q=f16(B + 1, T, HQ, D)), dict(out=torch.zeros(B + 2, T, HQ, D)), dict(bias=f16((HQ + 2 * HKV) * D)),
           dict(k_cache=cache, v_cache=cache.clone()), dict(k_cache=f16(B + 1, HKV, LMAX, D)), dict(k_new=f16(B * T * HKV * D))],
          [dict(q=f16(B, 1, HQ, D)), dict(q=f16(B, T, HQ, D).float()), dict(q=f16(B, T, HQ, 2 * D)[..., :D]), dict(q=f16(B, HQ, T, D).transpose(1, 2)),
           dict(k_new=f16(B, T, HKV - 1, D)), dict(k_new=f16(B, T, HKV, D).float()), dict(v_new=f16(B - 1, T, HKV, D)),
           dict(v_new=f16(B, T, 2 * HKV, D)[:, :, ::2]), dict(out=f16(B, T, HQ, D)), dict(out=torch.zeros(B, T, HQ - 1, D)),
           dict(out=torch.zeros(B, T, HQ, D, dtype=torch.float64)), dict(out=torch.zeros(B, HQ, T, D).transpose(1, 2)),
           dict(bias=f16(HQ * D)), dict(bias=torch.zeros((HQ + 2 * HKV) * D)), dict(k_cache=cache[:2]), dict(v_cache=cache.float()),
           dict(k_cache=f16(B, LMAX, HKV, D).transpose(1, 2)), dict(v_cache=f16(B + 1, LMAX, HKV, D))])


@pytest.mark.parametrize("out,dtype", [("f16", torch.float16), ("bf16", torch.bfloat16)])
def test_16_bit_outputs(make, out, dtype):  # noqa: F811
    check(make(out_dtype=out).prefix, step_args(out=dtype), [], [dict(out=torch.zeros(B, T, HQ, D)), dict(out=torch.zeros(B, T, HQ, D // 2))])


def test_int8_and_pages(make):  # noqa: F811
    codes = torch.zeros((HKV, 70, D), dtype=torch.int8)
    cache, sc = torch.zeros((B, HKV, LMAX, D), dtype=torch.int8), torch.zeros(2, B, HKV, LMAX)
    check(make("i8").prefix, dict(step_args(), k_prefix=codes, v_prefix=codes, prefix_scales=torch.zeros(2, HKV, 70)),
          [dict(scales=sc), dict(k_cache=cache, v_cache=cache.clone(), scales=sc)],
          [dict(scales=sc[:1]), dict(scales=sc.half()), dict(scales=sc.double()), dict(k_cache=cache.half()), dict(v_cache=cache[1:])])
    paged = dict(step_args(), k_prefix=None, v_prefix=None, block_table=i32(B, 2), prefix_table=i32(3))
    pages = f16(7, HKV, 128, D)
    check(make(max_len=256, page_size=128, num_pages=7).prefix, paged, [dict(k_cache=pages, v_cache=pages.clone())],
          [dict(k_cache=pages[:6]), dict(v_cache=f16(7, 128, HKV, D).transpose(1, 2)), dict(out=f16(B, T, HQ, D))])
