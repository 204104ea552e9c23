"""What DecodeStep's methods for the operators around the step refuse before the library is called: types,
sizes and strides that its pointers cannot show.  Needs no GPU."""
import types

import pytest
import torch

import decode_step_masked_gb300 as ftd

B, HQ, HKV, D, LMAX, T = 3, 4, 2, 64, 32, 2


class Called(Exception):
    pass


@pytest.fixture
def step(monkeypatch):
    """A DecodeStep without a context, whose library calls raise Called."""
    def call(*_):
        raise Called
    names = ("ftd_rope_qkv", "ftd_decode_mha_scored", "ftd_cache_evict", "ftd_cross_mha")
    monkeypatch.setattr(ftd, "load_library", lambda: types.SimpleNamespace(**{n: call for n in names}))
    monkeypatch.setattr(ftd, "ftd_init", lambda cfg, stream=0: (ftd.FTD_OK, 0))
    monkeypatch.setattr(ftd, "ftd_set_rope", lambda ctx, cfg: ftd.FTD_OK)
    monkeypatch.setattr(ftd, "_current_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    s = ftd.DecodeStep(B, HQ, HKV, D, LMAX, "f16", "f16", stream=0, q_len=T)
    s.set_rope(2, [16, 16])
    return s


def rope_args(n=5):
    z = lambda h: torch.zeros((n, h, D), dtype=torch.float16)  # noqa: E731
    return dict(q=z(HQ), k=z(HKV), v=z(HKV), positions=torch.zeros((2, n), dtype=torch.int32), q_out=z(HQ), k_out=z(HKV),
                v_out=z(HKV), bias=torch.zeros((HQ + 2 * HKV) * D, dtype=torch.float16))


def test_rope_arguments(step):
    ok = rope_args()
    fused = torch.zeros((5, (HQ + 2 * HKV) * D), dtype=torch.float16)
    good = [{}, dict(v=None, v_out=None), dict(bias=None), dict(bias=torch.zeros((HQ + 2 * HKV, D), dtype=torch.float16)),
            dict(q=fused[:, :HQ * D], k=fused[:, HQ * D:(HQ + HKV) * D], v=fused[:, (HQ + HKV) * D:]),
            dict(q_out=ok["q_out"].view(5, HQ * D)), dict(q=ok["q"].view(torch.int16)),  # (bits of the same width)
            dict(positions=torch.zeros(10, dtype=torch.int32)),
            # buffers kept for larger calls, and what the library itself refuses
            dict(positions=torch.zeros(64, dtype=torch.int32)), dict(positions=torch.zeros((4, 5), dtype=torch.int32)),
            dict(k=torch.zeros((9, HKV, D), dtype=torch.float16)), dict(q_out=torch.zeros((9, HQ, D), dtype=torch.float16)),
            dict(k_out=torch.zeros((9, HKV * D), dtype=torch.float16)), dict(v_out=torch.zeros(9 * HKV * D, dtype=torch.float16)),
            dict(bias=torch.zeros((HQ + 2 * HKV) * D + 7, dtype=torch.float16)), dict(v=None), dict(v_out=None)]
    for kw in good:
        with pytest.raises(Called):
            step.rope(**dict(ok, **kw))
    with pytest.raises(Called):
        step.rope(**rope_args(0))
    p, z = ok["positions"], ok["q"]
    bad = [dict(positions=p.long()), dict(positions=p.float()), dict(positions=p[:1]), dict(positions=p[:, :4].contiguous()),
           dict(positions=torch.zeros((5, 2), dtype=torch.int32).t()), dict(k=ok["k"][:4]), dict(v=ok["v"][:4]),
           dict(q=torch.zeros((5, HQ * D + 1), dtype=torch.float16)), dict(q=z.float()), dict(k=ok["k"].float()),
           dict(v=ok["v"].float()), dict(q_out=z[:4]), dict(q_out=z.float()), dict(k_out=ok["k"][:4]), dict(v_out=ok["v"][:4]),
           dict(q_out=fused[:, :HQ * D]), dict(k_out=fused[:, :HKV * D]), dict(v_out=fused[:, :HKV * D]),
           dict(positions=torch.zeros((2, 8), dtype=torch.int32)), dict(q_out=torch.zeros((9, HQ, D + 8), dtype=torch.float16)),
           dict(k_out=torch.zeros((9, HKV * D + 64), dtype=torch.float16)), dict(bias=ok["bias"][:-1]), dict(bias=ok["bias"].float()),
           dict(bias=torch.zeros(2 * (HQ + 2 * HKV) * D, dtype=torch.float16)[::2])]
    for kw in bad:
        with pytest.raises(ValueError):
            step.rope(**dict(ok, **kw))


def test_scored_evict_and_cross_arguments(step):
    lens, plane = torch.zeros(B, dtype=torch.int32), torch.zeros((B, HKV, LMAX))
    pos = plane.int()
    q, kn, out = torch.zeros((B, T, HQ, D), dtype=torch.float16), torch.zeros((B, T, HKV, D), dtype=torch.float16), torch.zeros((B, T, HQ, D))
    calls = [(step.scored, dict(q=q, k_new=kn, v_new=kn, seq_lens=lens, next_pos=lens, acc=plane, positions=pos, out=out),
              [dict(acc_out=plane.clone()), dict(positions=None, next_pos=None)]),
             (step.evict, dict(acc=plane, positions=pos, seq_lens=lens, next_pos=lens, new_lens=lens, budget=8),
              [dict(acc_out=plane.clone(), positions_out=pos.clone())]),
             (step.cross, dict(q=q, mem_lens=lens, out=out), [])]
    ints = {"seq_lens": lens, "next_pos": lens, "new_lens": lens, "mem_lens": lens, "positions": pos, "positions_out": pos}
    floats = {"acc": plane, "acc_out": plane}
    for fn, args, more in calls:
        for kw in [{}] + more:
            with pytest.raises(Called):
                fn(**dict(args, **kw))
        names = [n for n in list(ints) + list(floats) if n in args or any(n in m for m in more)]
        for name in names:
            x = ints.get(name, floats.get(name))
            bad = [x.long() if name in ints else x.double(), x.float() if name in ints else x.half(), x[:-1],
                   torch.stack([x, x], -1)[..., 0]]
            if x.dim() == 3:
                bad += [torch.cat([x, x], 2), torch.cat([x, x], 1)]  # (another context's layout)
            # a buffer kept for more slots, and a flat one
            for y in (torch.cat([x, x]), torch.cat([x, x]).view(-1)):
                with pytest.raises(Called):
                    fn(**dict(args, **{name: y}))
            for y in bad:
                with pytest.raises(ValueError):
                    fn(**dict(args, **{name: y}))


def test_paged_planes(step, monkeypatch):
    """A paged context's planes are [num_pages][Hkv][page_size]."""
    s = ftd.DecodeStep(B, HQ, HKV, D, 256, "f16", "f16", stream=0, page_size=128, num_pages=7)
    lens, plane, table = torch.zeros(B, dtype=torch.int32), torch.zeros((7, HKV, 128)), torch.zeros((B, 2), dtype=torch.int32)
    args = dict(acc=plane, positions=plane.int(), seq_lens=lens, next_pos=lens, new_lens=lens, budget=8, block_table=table)
    for kw in ({}, dict(acc=torch.zeros((9, HKV, 128))), dict(block_table=torch.zeros((B + 2, 2), dtype=torch.int32))):
        with pytest.raises(Called):
            s.evict(**dict(args, **kw))
    for kw in (dict(acc=plane[:6]), dict(acc=torch.zeros((B, HKV, 256))), dict(block_table=table.long()), dict(block_table=table[:, :1]),
               dict(block_table=torch.zeros((B, 3), dtype=torch.int32)), dict(acc=torch.zeros((9, HKV, 256))),
               dict(block_table=table[:2])):
        with pytest.raises(ValueError):
            s.evict(**dict(args, **kw))
