"""The step behind a shared prefix on weights whose roundings to one 16-bit number all pull the same way: a row's
weights are held as pairs of numbers, as the step holds them, whatever the type of its output."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from synthetic import to_storage
from tests import operators_ref as ref
from tests.gpu_util import TORCH_OUT, dev

pytestmark = pytest.mark.gpu

ROWS = 200


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


def single(x, dt):
    """x rounded to one number of the type that weights are made of (INT8 caches: bf16)."""
    dt = "bf16" if dt == "i8" else dt
    return ref.widen(to_storage(np.asarray(x, np.float32), dt), dt)


def rows_of(cache, D, q0):
    """First elements k of ROWS keys (the others are 0) and the signs of their values: row 0 has the largest score, 0, and the
    value 0; a later one's weight is in [1/2, 1), at least a quarter of a half step off when rounded to one number, and its value's
    sign is that rounding's, so that the roundings add up while the weights themselves nearly cancel."""
    rng = np.random.default_rng(8)
    k = -rng.uniform(0.05, 0.98, 40 * ROWS) * np.sqrt(D) * np.log(2.0) / q0
    if cache != "i8":
        k = ref.widen(to_storage(k.astype(np.float32), cache), cache)
    else:
        k = (k / 127).astype(np.float32).astype(np.float64) * 127  # (code 127 times a scale)
    w = np.exp(k * q0 / np.sqrt(D))
    off = single(w, cache) - w
    half = ref.HALF_STEP["bf16" if cache == "i8" else cache] / 2  # of numbers in [1/2, 1)
    keep = np.flatnonzero((np.abs(off) >= half / 4) & (w > 0.5) & (w < 1.0))
    up, down = ([i for i in keep if (off[i] > 0) == s] for s in (True, False))
    at, total = [], 0.0
    while len(at) < ROWS - 1:
        side = down if total > 0 else up
        i = side.pop()
        at.append(i)
        total += w[i] * (1 if side is up else -1)
    return np.concatenate([[0.0], k[at]]), np.concatenate([[0.0], np.sign(off[at])])


@pytest.mark.parametrize("cache,qkv,out,bias", [("bf16", "bf16", "bf16", False), ("bf16", "bf16", "bf16", True), ("bf16", "f32", "bf16", False),
                                                ("f16", "f16", "f16", False), ("f16", "f16", "f16", True), ("f16", "f16", "f32", False),
                                                ("bf16", "bf16", "f32", False), ("i8", "bf16", "bf16", False), ("i8", "f16", "f16", True)])
@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("B,Hq,Hkv,D", [(3, 4, 2, 128), (40, 8, 1, 64)])
def test_roundings_that_add_up(cache, qkv, out, bias, where, B, Hq, Hkv, D):
    """A weight as a pair is off by 2^-16 of it (bf16; fp16 2^-21, and 2^-25 of the largest where it is below the type's normal
    range), its score by D + 8 half steps of the one product in it, twice with the sum it is divided by, and the sums
    over the rows add a half step each; out is rounded once.  One number a weight would be off by many times that."""
    import torch
    q0 = 1.0 + (ref.HALF_STEP[qkv] if bias else 0.0)  # with its bias no number of the type
    k, sign = rows_of(cache, D, q0)
    storage = {"f32": np.float32, "f16": np.float16, "bf16": np.uint16, "i8": np.int8}[cache]
    values = sign[:, None] * np.where(np.arange(D) % 2, -1.0, 1.0)
    far = -4096.0  # a key that has no weight

    def put(first, vals, n):
        """Keys and values [n][D] in the cache's storage, and the scales [2][n] (INT8)."""
        if cache == "i8":
            kk, vv = np.zeros((n, D), np.int8), vals.astype(np.int8)
            kk[:, 0] = np.where(first == 0, 0, -127)
            return kk, vv, np.stack([np.where(first == 0, 1.0, -first / 127), np.ones(n)]).astype(np.float32)
        kk = np.zeros((n, D), np.float32)
        kk[:, 0] = first
        return to_storage(kk, cache), to_storage(vals.astype(np.float32), cache), None

    real = put(k, values, ROWS)
    none = put(np.array([far]), np.ones((1, D)), 1)
    pre, own = (real, none) if where == "prefix" else (none, real)
    P, lens = (ROWS, 0) if where == "prefix" else (1, ROWS)
    Lmax = 256
    step = ftd.DecodeStep(B, Hq, Hkv, D, Lmax, qkv, cache, out_dtype=out)
    step.enable_prefix()
    heads = lambda a: np.ascontiguousarray(np.broadcast_to(a, (Hkv,) + a.shape))  # noqa: E731
    kc, vc = (np.zeros((B, Hkv, Lmax, D), storage) for _ in range(2))
    sc = np.ones((2, B, Hkv, Lmax), np.float32) if cache == "i8" else None
    kw = {}
    if where == "own":
        kc[:, :, :ROWS], vc[:, :, :ROWS] = own[0], own[1]
        if cache == "i8":
            sc[:, :, :, :ROWS] = own[2][:, None, None]
    if cache == "i8":
        kw = dict(scales=dev(sc), prefix_scales=dev(np.ascontiguousarray(np.broadcast_to(pre[2][:, None], (2, Hkv, P)))))
    q, kn, vn = (np.zeros((B, h, D), np.float32) for h in (Hq, Hkv, Hkv))
    q[..., 0], kn[..., 0] = 1.0, far
    b = np.zeros(((Hq + 2 * Hkv) * D,), np.float32)
    b[0:Hq * D:D] = q0 - 1.0
    q, kn, vn, b = (dev(to_storage(x, qkv)) for x in (q, kn, vn, b))
    got = torch.full((B, Hq, D), float("nan"), dtype=getattr(torch, TORCH_OUT[out]), device="cuda")
    step.prefix(q, kn, vn, dev(np.full(B, lens, np.int32)), dev(np.full(B, P, np.int32)), got, k_prefix=dev(heads(pre[0])),
                v_prefix=dev(heads(pre[1])), k_cache=dev(kc), v_cache=dev(vc), bias=b if bias else None, **kw)
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    step.close()
    w = np.exp(k * q0 / np.sqrt(D))
    want, av = (w[:, None] * values).sum(0) / w.sum(), (w[:, None] * np.abs(values)).sum(0) / w.sum()
    e = np.abs(k).max() * q0 / np.sqrt(D) * (D + 8) * 2.0 ** -24
    pair = 2.0 ** -21 if cache == "f16" else 2.0 ** -16
    tol = av * (2 * e + pair + (ROWS + 32) * 2.0 ** -24) + (ROWS * 2.0 ** -25 if cache == "f16" else 0.0)
    if out != "f32":
        tol = tol + np.abs(want) * ref.HALF_STEP[out] * (1 + 2.0 ** -7) + (2.0 ** -25 if out == "f16" else 0.0)
    coarse = np.abs(((single(w, cache) - w)[:, None] * values).sum(0)) / w.sum()
    assert np.all(coarse > 2 * tol)  # (what single numbers would be off by)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(np.isfinite(err)) and np.all(err <= tol), float((err / tol).max())
