"""The order in which ftd_cache_evict keeps rows, on the inputs where it can go wrong: zeros of both
signs, positions before 0 and from next_pos on, and planes that may not overlap."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from synthetic import Workload
from tests.gpu_util import dev, make_step
from tests.test_evict_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


def moves(acc, pos, L, next_pos, budget, recent, sinks):
    """(source, destination) rows of one kv head: rows at a position below sinks or at least
    next_pos - recent come first, then the larger weight (NaN below all), then the lower row."""
    if L <= budget:
        return []
    first = [int(pos[t]) < sinks or int(pos[t]) >= int(next_pos) - recent for t in range(L)]

    def key(t):
        if first[t]:
            return (0, 0, 0.0, t)
        a = float(acc[t])
        return (1, 1, 0.0, t) if a != a else (1, 0, -a, t)  # (-0.0 == 0.0)
    kept = set(sorted(range(L), key=key)[:budget])
    return list(zip((t for t in range(budget, L) if t in kept), (t for t in range(budget) if t not in kept)))


@pytest.mark.parametrize("L,budget", [(640, 400), (640, 1), (500, 499), (9000, 4000)])
@pytest.mark.parametrize("values", [(0.0, -0.0), (0.0, -0.0, 1.0, -1.0), (0.0, -0.0, 1e-45, -1e-45, np.nan, -np.inf)])
def test_zeros_of_both_signs_are_equal(L, budget, values):
    """Equal weights stay by the lower row, and 0.0 == -0.0."""
    rng = np.random.default_rng(L + budget)
    acc = rng.choice(np.array(values, np.float32), (2, 2, 16 * (-(-L // 16))))
    check("f16", 2, 2, 64, acc.shape[2], [L, L], budget, acc=acc)


def run_positions(acc, pos, lens, next_pos, budget, recent, sinks):
    """One eviction in place; K rows carry their row index.  Returns the rows each head holds afterwards."""
    import torch
    B, H, Lmax = acc.shape
    step = make_step(Workload("evict", B=B, Hq=H, Hkv=H, D=64, Lmax=Lmax, qkv_dtype="f32", cache_dtype="f32"), scored=True)
    k = torch.arange(Lmax, device="cuda", dtype=torch.float32).view(1, 1, Lmax, 1).expand(B, H, Lmax, 64).contiguous()
    v = -k
    a, p, sl, new = dev(acc), dev(pos), dev(np.asarray(lens, np.int32)), dev(np.zeros(B, np.int32))
    step.evict(a, p, sl, dev(np.asarray(next_pos, np.int32)), new, budget, recent=recent, sinks=sinks, k_cache=k, v_cache=v)
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    step.close()
    assert torch.equal(k, -v) and torch.equal(k, k[..., :1].expand_as(k))
    return k[..., 0].cpu().numpy().astype(np.int64), a.cpu().numpy(), p.cpu().numpy()


@pytest.mark.parametrize("recent,sinks", [(0, 0), (0, 5), (7, 0), (40, 5)])
@pytest.mark.parametrize("lo,hi", [(-60, 0), (0, 40), (-60, 40), (-2 ** 31, 2 ** 31 - 1)])
def test_positions_before_zero_and_from_next_pos_on(recent, sinks, lo, hi):
    """Protected are the positions below sinks, negative ones too, and those from next_pos - recent on,
    next_pos and later ones too (recent 0 among them)."""
    rng = np.random.default_rng(100 + recent + sinks)
    B, H, Lmax, budget = 3, 2, 320, 150
    lens, next_pos = [320, 151, 290], [320, 200, -3]
    acc = rng.random((B, H, Lmax)).astype(np.float32)
    pos = np.empty((B, H, Lmax), np.int32)
    for b in range(B):
        a, c = (lo, hi) if hi - lo > 1000 else (lo, next_pos[b] + hi) if next_pos[b] > 0 else (lo - 10, hi + 10)
        pos[b] = rng.integers(a, c, (H, Lmax))
        pos[b, :, 3] = rng.integers(0, 50)  # (at least one ordinary position)
    rows, a1, p1 = run_positions(acc, pos, lens, next_pos, budget, recent, sinks)
    for b in range(B):
        for h in range(H):
            want = np.arange(Lmax)
            for s, d in moves(acc[b, h], pos[b, h], lens[b], next_pos[b], budget, recent, sinks):
                want[d] = s
            assert np.array_equal(rows[b, h], want), (b, h)
            assert np.array_equal(a1[b, h], acc[b, h][want]) and np.array_equal(p1[b, h], pos[b, h][want])


def test_planes_of_different_kinds_are_apart():
    """An output plane may be its own input and nothing else's."""
    import torch
    w = Workload("evict", B=2, Hq=2, Hkv=2, D=64, Lmax=256, qkv_dtype="f16", cache_dtype="f16")
    step = make_step(w, scored=True)
    n = 2 * 2 * 256 * 4
    buf = torch.zeros(8 * n, dtype=torch.uint8, device="cuda")
    p = [buf.data_ptr() + i * n for i in range(8)]
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")  # (no slot has work: a call that is not refused moves nothing)
    q = torch.zeros(4096, dtype=torch.float16, device="cuda")
    before = ftd.ftd_kernel_launches()

    def evict(acc, acc_out, pos, pos_out):
        return ftd.ftd_cache_evict(step.ctx, 0, 0, 0, 0, lens.data_ptr(), lens.data_ptr(), acc, acc_out, pos, pos_out,
                                   lens.data_ptr(), 100, 0, 0, 0)
    for a, ao, s, so in ((p[0], 0, p[0], 0), (p[0], p[2], p[2], p[3]), (p[0], p[2], p[1], p[0]), (p[0], p[2], p[1], p[2]),
                         (p[0], 0, p[0] + n - 4, 0), (p[0], p[2], p[1], p[2] + 4), (p[1], p[2], p[0] + 4, 0)):
        assert evict(a, ao, s, so) == ftd.FTD_ERR_INVALID_ARG and ftd.ftd_last_error()
    # the scored step writes acc_out and positions
    skip = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    out = torch.zeros((2, 2, 64), device="cuda")

    def scored(acc, acc_out, pos):
        return ftd.ftd_decode_mha_scored(step.ctx, q.data_ptr(), q.data_ptr(), q.data_ptr(), 0, 0, 0, 0, skip.data_ptr(), 0,
                                         lens.data_ptr(), acc, acc_out, pos, out.data_ptr(), 0)
    for a, ao, s in ((p[0], 0, p[0]), (p[0], p[2], p[2]), (p[0], p[2], p[0]), (p[1], p[2], p[0] + 4), (p[0], p[2], p[2] + n - 4)):
        assert scored(a, ao, s) == ftd.FTD_ERR_INVALID_ARG and ftd.ftd_last_error()
    assert ftd.ftd_kernel_launches() == before
    assert evict(p[0], p[1], p[2], p[3]) == ftd.FTD_OK and evict(p[0], 0, p[1], 0) == ftd.FTD_OK
    assert scored(p[0], p[1], p[2]) == ftd.FTD_OK and scored(p[0], 0, p[1]) == ftd.FTD_OK and scored(p[0], p[0], 0) == ftd.FTD_OK
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    step.close()
