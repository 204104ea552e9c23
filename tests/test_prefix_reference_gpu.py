"""The running reference of an INT8 prefix's softmax, which moves in the middle of a tile: what such a move does to the
weights that the tile holds already, for the row that moves and for the other rows of its warp."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from synthetic import to_storage
from tests import operators_ref as ref
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

TILE, TILES, DIM = 128, 100, 128
EARLY = 64   # rows of a tile ahead of the one where a reference moves
AT = 70      # that row
LEAD = 8.0   # first element of a query that sees the steep keys
# a piece of the prefix that one block takes is at most 8 tiles (800 tiles and more than 100 blocks)
SUMS = (8 * TILE + 200) * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


def bf16(x):
    return ref.widen(to_storage(np.asarray(x, np.float32), "bf16"), "bf16")


def moved_twice(s, step):
    """What rounding a tile's early weights a second time, as pairs of bf16 numbers times the ratio of two references, would
    change each by (in units of the new reference).  s [TILES][TILE] scores in the log2 domain; a stream takes every
    step-th tile, and its reference is the largest score from row AT on of its tile before."""
    off = np.zeros_like(s)
    top = s[:, EARLY:].max(1)
    for i in range(step, TILES):
        w, a = np.exp2(s[i, :EARLY] - top[i - step]), np.exp2(top[i - step] - top[i])
        hi = bf16(w)
        lo = bf16(w - hi)
        off[i, :EARLY] = bf16(hi * a) + bf16(lo * a) - (hi + lo) * a
    return off


def run(s, steep, v, B, Hkv, qkv, leads):
    """Outputs [B][Hkv * 8][DIM] of slots that see a prefix of keys (steep, s) / q and values v [rows], alone.  A key has one element:
    the second, for a score of s in every query, or in rows where steep is not 0 the first, for a score of steep in the
    queries of `leads` (rows of a kv head), which are LEAD there, and of 0 in the others."""
    import torch
    scale = np.log2(np.e) / np.sqrt(DIM)
    P, Hq = s.size, 8 * Hkv
    codes = np.zeros((Hkv, P, DIM), np.int8)
    codes[:, :, 1] = np.where(steep == 0, 127, 0)
    codes[:, :, 0] = np.where(steep == 0, 0, 127)
    values = np.zeros((Hkv, P, DIM), np.int8)
    values[:] = np.where(np.arange(DIM) % 2, -v[:, None], v[:, None])
    ks = np.where(steep == 0, s / (127 * scale), steep / (127 * LEAD * scale)).astype(np.float32)
    psc = np.stack([np.broadcast_to(ks, (Hkv, P)), np.ones((Hkv, P), np.float32)]).astype(np.float32)
    q = np.zeros((B, Hkv, 8, DIM), np.float32)
    q[..., 1] = 1.0
    for r in leads:
        q[r // 8, :, r % 8, 0] = LEAD
    step = ftd.DecodeStep(B, Hq, Hkv, DIM, 32, qkv, "i8")
    step.enable_prefix()
    new = dev(to_storage(np.zeros((B, Hkv, DIM), np.float32), qkv))
    out = torch.full((B, Hkv, 8, DIM), float("nan"), device="cuda")
    step.prefix(dev(to_storage(q.reshape(B, Hq, DIM), qkv)), new, new, dev(np.zeros(B, np.int32)), dev(np.full(B, P, np.int32)), out,
                k_prefix=dev(codes), v_prefix=dev(values), prefix_scales=dev(psc))
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    step.close()
    return out.double().cpu().numpy().transpose(0, 2, 1, 3).reshape(8 * B, Hkv, DIM), ks.astype(np.float64) * 127 * scale


def bound(s, v, extra=0.0):
    """The outputs' one value, of alternating sign, and its bound.  A score is one product, scaled twice and compared with the reference: four
    half steps, twice with the sum; a weight's pair is off by 2^-16; sums as above.  (The new row, of score 0, counts.)"""
    x = np.append(s, 0.0)
    w = np.exp2(x - x.max())
    p = w / w.sum()
    p = p[:-1]
    return (p * v).sum(), (p * np.abs(v)).sum() * (2 * 4 * 2.0 ** -24 * np.abs(s).max() * np.log(2.0) + 2.0 ** -16 + SUMS + extra)


def ramp(step):
    """Scores that rise a little along every tile, with a key in each tile, behind its first 32 rows, that one query alone sees: it
    moves that query's reference by 60 and more."""
    t = np.arange(TILES * TILE).reshape(TILES, TILE)
    s = 0.37 * (t + 1) / TILE
    steep = np.zeros(s.shape)
    steep[:, AT] = 60.0 * (1 + np.arange(TILES))
    v = np.sign(moved_twice(s, step)).astype(np.int8)
    v[:, AT] = 1
    return s.reshape(-1), steep.reshape(-1), v.reshape(-1)


SHAPES = {"one_block": (5, 8, 2), "two_blocks": (40, 4, 1)}  # slots, kv heads, and every which tile is a stream's


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("qkv", ["f16", "bf16", "f32"])
def test_a_row_that_leaps(shape, qkv):
    """One row of a warp leaps in every tile, the others rise a little: the weights that the tile holds already stay those of the
    scores.  (Twice rounded they would be off by 2^-8.)"""
    B, hkv, every = SHAPES[shape]
    s, steep, v = ramp(every)
    leads = [3, 35]
    got, eff = run(s, steep, v, B, hkv, qkv, leads)
    assert np.all(np.isfinite(got))
    sign = np.where(np.arange(DIM) % 2, -1.0, 1.0)
    want, tol = bound(np.where(steep == 0, eff, 0.0), v, extra=2.0 ** -8)
    rest = np.setdiff1d(np.arange(8 * B), leads)
    assert np.all(np.abs(got[rest] - want * sign) <= tol), float(np.abs(got[rest] - want * sign).max() / tol)
    # the row that leaps sees nothing but the last steep key
    assert np.all(np.abs(got[leads] - sign) <= 2.0 ** -16 + SUMS)


def second_roundings(off, s, v):
    """What the weights' second roundings (in units of each tile's reference) would change the outputs by."""
    x = np.append(s, 0.0)
    top = s.reshape(TILES, TILE)[:, EARLY:].max(1)
    return abs((off * np.exp2(top - x.max())[:, None] * v.reshape(TILES, TILE)).sum() / np.exp2(x - x.max()).sum())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("qkv", ["f16", "bf16", "f32"])
def test_neighbours_of_a_row_that_leaps(shape, qkv):
    """The others' weights stay pairs, whose roundings are far below those of a second one, which would add up here."""
    B, hkv, every = SHAPES[shape]
    s, steep, v = ramp(every)
    leads = [3, 35]
    got, eff = run(s, steep, v, B, hkv, qkv, leads)
    want, tol = bound(np.where(steep == 0, eff, 0.0), v)
    assert second_roundings(moved_twice(s.reshape(TILES, TILE), every), s, v) > 4 * tol
    sign = np.where(np.arange(DIM) % 2, -1.0, 1.0)
    rest = np.setdiff1d(np.arange(8 * B), leads)
    err = np.abs(got[rest] - want * sign)
    assert np.all(np.isfinite(err)) and np.all(err <= tol), float(err.max() / tol)


def cliffs(step):
    """The prefix's last tiles: scores that come as near to the reach of the running reference as they may, then one that passes it,
    so that the weights behind the move weigh no more than those ahead of it."""
    s, h = np.zeros((TILES, TILE)), np.zeros(TILES)
    rng = np.random.default_rng(4)
    for i in range(TILES - 6, TILES):
        if i - step < TILES - 6:
            continue
        low = h[i - step]
        s[i] = low + 39.0 + 0.9 * rng.random(TILE)
        s[i, AT] = h[i] = low + 40.6
    # (the pattern's own moved_twice: the reference of a stream's tile before is that tile's cliff)
    off = moved_twice(s, step)
    off[:TILES - 6 + step] = 0.0
    v = np.sign(off).astype(np.int8)
    return s.reshape(-1), off, v.reshape(-1)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("qkv", ["f16", "f32"])
def test_weights_ahead_of_a_move_that_count(shape, qkv):
    """Every row moves in the middle of a tile, by little more than the weights before it are above the old reference."""
    B, hkv, every = SHAPES[shape]
    s, off, v = cliffs(every)
    got, eff = run(s, np.zeros(s.shape), v, B, hkv, qkv, [])
    want, tol = bound(eff, v)
    assert second_roundings(off, s, v) > 4 * tol
    err = np.abs(got - want * np.where(np.arange(DIM) % 2, -1.0, 1.0))
    assert np.all(np.isfinite(err)) and np.all(err <= tol), float(err.max() / tol)
