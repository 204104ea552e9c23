"""Norms with rotary positions, block tables and the step behind a shared prefix on the host: refusals that need no
context, and what DecodeStep's methods refuse before the library is called.  Needs no GPU."""
import types

import pytest
import torch

import decode_step_masked_gb300 as ftd

B, HQ, HKV, D, LMAX, T = 3, 4, 2, 64, 32, 2


class Called(Exception):
    pass


@pytest.fixture
def make(monkeypatch):
    """DecodeSteps without a context, whose library calls raise Called."""
    def call(*_):
        raise Called
    names = ("ftd_norm_rope_qkv", "ftd_build_tables", "ftd_enable_prefix", "ftd_decode_mha_prefix")
    monkeypatch.setattr(ftd, "load_library", lambda: types.SimpleNamespace(**{n: call for n in names}))
    monkeypatch.setattr(ftd, "ftd_init", lambda cfg, stream=0: (ftd.FTD_OK, 0))
    monkeypatch.setattr(ftd, "ftd_set_rope", lambda ctx, cfg: ftd.FTD_OK)
    monkeypatch.setattr(ftd, "_current_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def make(cache="f16", **kw):
        s = ftd.DecodeStep(B, HQ, HKV, D, kw.pop("max_len", LMAX), "f16", cache, stream=0, q_len=T, **kw)
        s.set_rope(2, [16, 16])
        return s
    return make


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def check(fn, args, good, bad):
    for kw in [{}] + good:
        with pytest.raises(Called):
            fn(**dict(args, **kw))
    for kw in bad:
        with pytest.raises(ValueError):
            fn(**dict(args, **kw))


def test_null_context():
    ftd.build_library()
    n = ftd.ftd_kernel_launches()
    assert ftd.ftd_norm_rope_qkv(0, 16, 16, 16, 0, 0, 0, 0, 0, 1e-6, 0.0, 16, 1, 16, 16, 16, 0, 0, 0, 0, 0) == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_build_tables(0, *[16] * 10, 1, 0) == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_enable_prefix(0, 0) == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_decode_mha_prefix(0, *[16] * 13, 1, 16, 16, 0) == ftd.FTD_ERR_INVALID_ARG
    assert "ctx is NULL" in ftd.ftd_last_error()
    assert ftd.ftd_kernel_launches() == n


def test_norm_rope_arguments(make):
    n, w = 5, f16(D)
    dense = dict(q=f16(n, HQ, D), k=f16(n, HKV, D), v=f16(n, HKV, D), positions=i32(2, n), q_out=f16(n, HQ, D), k_out=f16(n, HKV, D),
                 v_out=f16(n, HKV, D), bias=f16((HQ + 2 * HKV) * D), q_weight=w, k_weight=w)
    fused = f16(n, (HQ + 2 * HKV) * D)
    check(make().norm_rope, dense,
          [dict(q_weight=None), dict(k_weight=None, bias=None), dict(v=None, v_out=None), dict(weight_offset=1.0),
           dict(q=fused[:, :HQ * D], k=fused[:, HQ * D:(HQ + HKV) * D], v=fused[:, (HQ + HKV) * D:])],
          [dict(q_weight=f16(D - 1)), dict(k_weight=w.float()), dict(q_weight=f16(2 * D)[::2]), dict(positions=i32(2, n).long()),
           dict(positions=i32(n)), dict(k=dense["k"][:4]), dict(q_out=fused[:, :HQ * D]), dict(bias=f16(HQ * D)),
           dict(k=fused[:, HQ * D:(HQ + HKV) * D])])
    fill = dict(dense, k_out=None, v_out=None, slots=i32(n))
    cache = f16(B, HKV, LMAX, D)
    check(make().norm_rope, fill, [dict(k_cache=cache, v_cache=cache.clone()), dict(k_cache=f16(B + 2, HKV, LMAX, D))],
          [dict(slots=i32(n).long()), dict(slots=i32(n - 1)), dict(slots=i32(2 * n)[::2]), dict(k_cache=cache.float()),
           dict(v_cache=cache[:2]), dict(k_cache=f16(B + 1, LMAX, HKV, D)), dict(k_cache=cache.transpose(1, 2))])
    sc = torch.zeros(2, B, HKV, LMAX)
    codes = torch.zeros((B, HKV, LMAX, D), dtype=torch.int8)
    check(make("i8").norm_rope, dict(fill, k_cache=codes, v_cache=codes.clone()), [dict(scales=sc)],
          [dict(scales=sc[:1]), dict(scales=sc.half()), dict(k_cache=cache)])


def test_tables_arguments(make):
    lens, table, pool = i32(B), i32(B, 2), i32(7)
    flat = dict(old_lens=lens, new_lens=lens.clone(), served=lens)
    check(make().tables, flat,
          [dict(slots=i32(40), positions=i32(40)), dict(offsets=i32(B + 1)), dict(slots=i32(0)), dict(old_lens=i32(B + 2))],
          [dict(old_lens=lens.long()), dict(new_lens=i32(B - 1)), dict(served=lens.float()), dict(offsets=i32(B)),
           dict(slots=i32(40), positions=i32(41)), dict(slots=i32(40).long()), dict(positions=i32(80)[::2])])
    paged = make(max_len=256, page_size=128, num_pages=7)
    check(paged.tables, dict(flat, block_table=table, free_pages=pool, n_free=i32(1)), [dict(n_free_out=i32(1))],
          [dict(block_table=table.long()), dict(block_table=i32(B, 3)), dict(free_pages=i32(6)), dict(free_pages=pool.float()),
           dict(n_free=i32(1).long()), dict(n_free_out=i32(0))])


def test_prefix_arguments(make):
    lens, k = i32(B), f16(HKV, 70, D)
    args = dict(q=f16(B, T, HQ, D), k_new=f16(B, T, HKV, D), v_new=f16(B, T, HKV, D), seq_lens=lens, prefix_lens=lens,
                out=torch.zeros(B, T, HQ, D))
    with pytest.raises(Called):
        make().enable_prefix()
    check(make().prefix, args, [dict(k_prefix=k, v_prefix=k), dict(k_prefix=f16(HKV, 0, D), v_prefix=f16(HKV, 0, D))],
          [dict(k_prefix=k), dict(v_prefix=k), dict(k_prefix=k, v_prefix=f16(HKV, 71, D)), dict(k_prefix=k.float(), v_prefix=k.float()),
           dict(k_prefix=f16(70, HKV, D), v_prefix=f16(70, HKV, D)), dict(k_prefix=k.transpose(0, 1), v_prefix=k.transpose(0, 1)),
           dict(prefix_lens=lens.long()), dict(prefix_lens=i32(B - 1)), dict(seq_lens=lens.float())])
    codes = torch.zeros((HKV, 70, D), dtype=torch.int8)
    sc = torch.zeros(2, HKV, 70)
    check(make("i8").prefix, dict(args, k_prefix=codes, v_prefix=codes), [dict(prefix_scales=sc)],
          [dict(prefix_scales=sc[:1]), dict(prefix_scales=sc.double()), dict(prefix_scales=torch.zeros(2, HKV, 71))])
    paged = make(max_len=256, page_size=128, num_pages=7)
    check(paged.prefix, dict(args, block_table=i32(B, 2), prefix_table=i32(3)), [dict(prefix_table=i32(0)), dict(prefix_table=None)],
          [dict(prefix_table=i32(3).long()), dict(prefix_table=i32(6)[::2]), dict(block_table=i32(B, 3))])
