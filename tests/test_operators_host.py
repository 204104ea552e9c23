"""The operators around the step on the host: refusals that need no context, the rotary
configuration's layout, row strides, and the plain eviction that the GPU tests compare with."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import decode_step_masked_gb300 as ftd
from tests import operators_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    ftd.build_library()
    return ftd.load_library()


def test_null_context(lib):
    n = ftd.ftd_kernel_launches()
    assert ftd.ftd_set_rope(0, ftd.FtdRopeConfig()) == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_rope_qkv(0, 16, 16, 0, 0, 0, 0, 16, 1, 16, 16, 0, 0) == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_enable_scores(0, 0) == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_decode_mha_scored(0, *[16] * 14, 0) == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_cache_evict(0, *[16] * 11, 1, 0, 0, 0) == ftd.FTD_ERR_INVALID_ARG
    assert ftd.ftd_cross_mha(0, 16, 0, 16, 16, 16, 0, 16, 0) == ftd.FTD_ERR_INVALID_ARG
    assert "ctx is NULL" in ftd.ftd_last_error()
    assert ftd.ftd_kernel_launches() == n


def test_rope_config_matches_header():
    with open(os.path.join(ROOT, "include", "ftd.h")) as f:
        text = f.read()
    body = re.search(r"typedef struct \{([^}]*)\} ftd_rope_config;", text).group(1)
    names = re.findall(r"\b([a-z_]+)(?:\[4\])?\s*;", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
    assert names == [f for f, _ in ftd.FtdRopeConfig._fields_]
    assert ctypes.sizeof(ftd.FtdRopeConfig) == 48  # 8 ints, a double, a pointer


def test_row_strides():
    x = torch.zeros(4, 6, 40)
    rs = ftd._row_stride
    assert rs(x, 40, 8) == 0 and rs(x.view(24, 40), 40, 8) == 0 and rs(x.view(24, 5, 8), 40, 8) == 0
    assert rs(x[..., 8:24], 16, 8) == 40 and rs(x.view(4, 6, 5, 8)[..., 1:3, :], 16, 8) == 40
    assert rs(x[:, :1, :16], 16, 8) == 240 and rs(x[:1, :, :16], 16, 8) == 40
    assert rs(x[:1, :1, :16], 16, 8) == 0
    for bad in (x[:, :3, :16], x[..., ::2], x.transpose(0, 1)[..., :16], x.view(4, 6, 5, 8)[..., ::2, :]):
        with pytest.raises(ValueError):
            rs(bad, bad.shape[-1] if bad.dim() == 3 else 24, 8)


def test_plain_eviction():
    """The restatement itself, on cases worked by hand."""
    acc = np.array([5.0, 1.0, 4.0, 2.0, 3.0, 0.5], np.float32)
    pos = np.arange(6)
    assert ref.evict_moves(acc, pos, 6, 6, 3, 0, 0) == [(4, 1)]            # keeps 0, 2, 4
    assert ref.evict_moves(acc, pos, 6, 6, 3, 2, 0) == [(4, 1), (5, 2)]    # keeps 0 and the newest two
    assert ref.evict_moves(acc, pos, 6, 6, 3, 1, 2) == [(5, 2)]            # keeps 0, 1 and the newest
    assert ref.evict_moves(np.ones(6, np.float32), pos, 6, 6, 3, 0, 0) == []  # ties: the lower rows
    assert ref.evict_moves(np.array([np.nan, -np.inf, 1.0], np.float32), np.arange(3), 3, 3, 2, 0, 0) == [(2, 0)]
    assert ref.evict_moves(acc, pos, 3, 6, 3, 0, 0) == []
