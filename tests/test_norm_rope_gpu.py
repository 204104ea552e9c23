"""ftd_norm_rope_qkv against the formula in 64 bits: types, head dimensions, rotary dimensions and axes, one token to
thousands, fused and dense sources, unaligned rows, weights with an offset or of one kind of head only, dense outputs and
fills of contiguous and paged caches of every type, padded tokens, and the refusals."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from tests import operators_ref as ref
from tests.gpu_util import dev
from tests.test_rope_gpu import TORCH, sections_of, typed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


U = 2.0 ** -24  # half a step of binary32


def normed(z, w, eps, offset):
    """Heads z [n][H][D] and the bound of the kernel's error of each element.  Per element, in half steps U of its
    value: the bias add 1; the sum of squares 2 (of the add) + 16 (its chain, then three exchanges: 19), halved by the root
    with the mean's product and eps: (2 + 19 + 2) / 2 < 12; rsqrtf at most 2 ulp: 4; the weight's add and the two
    products: 3.  20 in all."""
    if w is None:
        return z, U * np.abs(z)
    y = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * (w + offset)
    return y, 20 * U * np.abs(y)


def turned(y, e, pos, inv, axis, pairing, far):
    """y turned, and the bound: the incoming errors of a pair's two members, and ftd_rope_qkv's own (test_rope_gpu.tolerance)
    without its bias add."""
    t = ref.rope(y, pos, inv, axis, pairing)
    big = 2.0 * np.abs(y).max(-1, keepdims=True)
    return t, 2.0 * e.max(-1, keepdims=True) + big * (6 * U + 3 * 2.0 ** -53 * far)


def stored(y, dt):
    """Half a step of a stored value y."""
    if dt == "f32":
        return U * np.abs(y)
    return np.abs(y) * ref.HALF_STEP[dt] * (1 + 2.0 ** -10) + (2.0 ** -25 if dt == "f16" else 0.0)


def near(got, want, tol, what):
    assert np.all(np.isfinite(got)), what
    err = np.abs(got - want)
    assert np.all(err <= tol), (what, float((err / np.maximum(tol, 1e-300)).max()))


def run(Hq, Hkv, D, dt, n, cache="", page=0, axes=1, R=0, pairing="halves", order="sections", fused=True, bias=True, qw=True,
        kw=True, eps=1e-6, offset=0.0, far=5000, seed=1, shift=0, scale=1.0, pad=0):
    """One call; cache: the type of the cache that takes keys and values ("": dense outputs); pad: tokens without a slot."""
    import torch
    rng = np.random.default_rng(seed)
    R = R or D
    W = (Hq + 2 * Hkv) * D
    secs = sections_of(R // 2, axes)
    inv = 10000.0 ** (-np.arange(0, R, 2) / R)
    pos = rng.integers(-far, far, size=(axes, n)).astype(np.int32)
    b_t, b = typed(0.2 * rng.standard_normal(W), dt) if bias else (None, np.zeros(W))
    x_t, x = typed(scale * rng.standard_normal((n, W)), dt)
    q_t, qv = typed(1 + 0.3 * rng.standard_normal(D) - offset, dt) if qw else (None, None)
    k_t, kv = typed(1 + 0.3 * rng.standard_normal(D) - offset, dt) if kw else (None, None)
    if fused:
        buf = torch.zeros(n * W + 64, dtype=x_t.dtype, device="cuda")
        f = buf[shift:shift + n * W].view(n, W)
        f.copy_(x_t)
        q, k, v = f[:, :Hq * D], f[:, Hq * D:(Hq + Hkv) * D], f[:, (Hq + Hkv) * D:]
    else:
        q, k, v = (x_t[:, a:c].contiguous() for a, c in ((0, Hq * D), (Hq * D, (Hq + Hkv) * D), ((Hq + Hkv) * D, W)))
    outs = [torch.full((n, h, D), float("nan"), dtype=x_t.dtype, device="cuda") for h in (Hq, Hkv, Hkv)]
    z = (x + b).reshape(n, Hq + 2 * Hkv, D)
    ax = ref.pair_axes(axes, secs, order)
    yq, eq = turned(*normed(z[:, :Hq], qv, eps, offset), pos, inv, ax, pairing, far)
    yk, ek = turned(*normed(z[:, Hq:Hq + Hkv], kv, eps, offset), pos, inv, ax, pairing, far)
    yv, ev = z[:, Hq + Hkv:], U * np.abs(z[:, Hq + Hkv:])
    opts = dict(bias=b_t, q_weight=q_t, k_weight=k_t, eps=eps, weight_offset=offset)
    before = ftd.ftd_kernel_launches()
    if not cache:
        step = ftd.DecodeStep(1, Hq, Hkv, D, 16, dt, dt)
        step.set_rope(axes, secs, rotary_dim=R, pairing=pairing, order=order, inv_freq=inv)
        step.norm_rope(q, k, v, dev(pos), *outs, **opts)
        torch.cuda.synchronize()
        for name, o, y, e in zip("qkv", outs, (yq, yk, yv), (eq, ek, ev)):
            near(o.double().cpu().numpy(), y, e + stored(y, dt), name)
    else:
        B, unit = (1, page) if page else (3, -(-n // 3 // 16) * 16 + 32)
        units = -(-n // page) + 1 if page else B
        lmax = units * page if page else unit
        step = ftd.DecodeStep(B, Hq, Hkv, D, lmax, dt, cache, page_size=page, num_pages=units if page else 0)
        step.set_rope(axes, secs, rotary_dim=R, pairing=pairing, order=order, inv_freq=inv)
        slots = rng.permutation(units * unit)[:n].astype(np.int32)
        slots[n - pad:] = -1 - np.arange(pad)
        ct = torch.int8 if cache == "i8" else getattr(torch, TORCH[cache])
        fill = 77 if cache == "i8" else float("nan")
        kc, vc = (torch.full((units, Hkv, unit, D), fill, dtype=ct, device="cuda") for _ in range(2))
        sc = torch.full((2, units, Hkv, unit), float("nan"), device="cuda") if cache == "i8" else None
        step.norm_rope(q, k, v, dev(pos), outs[0], slots=dev(slots), k_cache=kc, v_cache=vc, scales=sc, **opts)
        torch.cuda.synchronize()
        near(outs[0].double().cpu().numpy(), yq, eq + stored(yq, dt), "q")
        live = slots >= 0
        u, r = slots[live] // unit, slots[live] % unit
        named = np.zeros((units, unit), bool)
        named[u, r] = True
        for name, c, y, e, plane in (("k", kc, yk, ek, 0), ("v", vc, yv, ev, 1)):
            c = c.double().cpu().numpy()
            rest = c.transpose(0, 2, 1, 3)[~named]
            assert np.all(rest == 77) if cache == "i8" else np.all(np.isnan(rest)), name + ": rows of no token"
            got, y, e = c[u, :, r], y[live], e[live]
            if cache != "i8":
                near(got, y, e + stored(y, cache), name)
                continue
            s = sc[plane].double().cpu().numpy()
            assert np.all(np.isnan(s.transpose(0, 2, 1)[~named]))
            s = s[u, :, r]
            top = np.abs(y).max(-1)
            # the largest magnitude's error, and the quotient's rounding
            near(s, top / 127, e.max(-1) / 127 + U * top / 127, name + " scales")
            assert np.all(np.abs(got) <= 127)
            # a code's half step (the quotient rounded: 127 U more) of the scale that was stored, and the value's error
            near(got * s[..., None], y, s[..., None] * (0.5 + 256 * U) + e, name)
    assert ftd.ftd_kernel_launches() == before + 1
    assert step.get_error() == ftd.FTD_OK
    step.close()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 64), (128, 64), (64, 8), (128, 22), (64, 2), (128, 120), (64, 52)])
@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
def test_types_and_rotary_dims(dt, D, R, pairing):
    """(8, 120 and 52 leave runs of 4, 4 and 2 pairs, 22 and 2 single ones: narrower accesses.)"""
    run(6, 2, D, dt, 5, R=R, pairing=pairing)


@pytest.mark.parametrize("cache", ["f32", "f16", "bf16", "i8"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,R,page", [(128, 128, 0), (64, 64, 128), (128, 24, 128), (64, 22, 0), (128, 6, 0)])
def test_fill_types(dt, cache, D, R, page):
    run(6, 3, D, dt, 41, cache=cache, page=page, R=R, pad=4)
    run(3, 1, D, dt, 7, cache=cache, page=page, R=R, pairing="adjacent", bias=False)


@pytest.mark.parametrize("n", [1, 2, 151, 608, 609, 4999])
@pytest.mark.parametrize("heads", [(1, 1), (7, 1), (32, 32), (64, 8)])
def test_lengths(n, heads):
    if n == 4999 and heads == (32, 32):
        n = 2501
    run(*heads, 128, "bf16", n, axes=3)
    run(*heads, 128, "bf16", n, axes=1, cache="bf16", page=256, pad=n // 10)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("order", ["sections", "interleaved"])
def test_axes(axes, order):
    run(4, 4, 128, "bf16", 37, axes=axes, order=order)
    run(4, 1, 64, "f32", 7, axes=axes, order=order, R=40, pairing="adjacent", cache="i8")


@pytest.mark.parametrize("qw,kw,offset", [(True, False, 0.0), (False, True, 1.0), (False, False, 0.0), (True, True, 1.0)])
def test_weights(qw, kw, offset):
    run(8, 2, 128, "f16", 33, qw=qw, kw=kw, offset=offset)
    run(8, 2, 64, "bf16", 33, qw=qw, kw=kw, offset=offset, cache="f16")


@pytest.mark.parametrize("shift", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_alignment(dt, shift):
    run(5, 1, 64, dt, 9, shift=shift)
    run(5, 1, 64, dt, 9, shift=shift, cache="i8")


@pytest.mark.parametrize("scale,eps", [(1e-3, 1e-6), (1e-3, 0.0), (200.0, 1e-6), (1e4, 1e-5)])
def test_magnitudes(scale, eps):
    run(4, 4, 128, "bf16", 9, scale=scale, eps=eps, bias=False)
    run(4, 4, 64, "f32", 9, scale=scale, eps=eps, bias=False, cache="i8")


def test_far_positions():
    run(2, 2, 128, "f32", 64, far=(1 << 31) - 1)


def test_zero_heads_and_in_place():
    """Heads of zeros stay zeros (INT8: codes 0, scale 1); outputs may be their own dense inputs."""
    import torch
    step = ftd.DecodeStep(2, 4, 2, 64, 32, "f16", "i8")
    step.set_rope()
    z = lambda h: torch.zeros((5, h, 64), dtype=torch.float16, device="cuda")  # noqa: E731
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    pos, slots = dev(np.arange(5, dtype=np.int32)[None]), dev(np.array([0, 1, 33, 63, -1], np.int32))
    kc, vc = (torch.full((2, 2, 32, 64), 5, dtype=torch.int8, device="cuda") for _ in range(2))
    sc = torch.zeros((2, 2, 2, 32), device="cuda")
    out = torch.full((5, 4, 64), float("nan"), dtype=torch.float16, device="cuda")
    step.norm_rope(z(4), z(2), z(2), pos, out, q_weight=w, k_weight=w, slots=slots, k_cache=kc, v_cache=vc, scales=sc)
    torch.cuda.synchronize()
    assert not out.any()
    for c, p in ((kc, sc[0]), (vc, sc[1])):
        at = ((0, 0), (0, 1), (1, 1), (1, 31))
        assert all(not c[b, :, r].any() and torch.all(p[b, :, r] == 1) for b, r in at)
        assert int((c != 5).any(-1).sum()) == 8 and int((p != 0).sum()) == 8
    x = torch.randn((5, 4, 64), device="cuda").half()
    k, v = torch.randn((5, 2, 64), device="cuda").half(), torch.randn((5, 2, 64), device="cuda").half()
    want = [torch.empty_like(t) for t in (x, k, v)]
    dense = ftd.DecodeStep(1, 4, 2, 64, 16, "f16", "f16")
    dense.set_rope()
    dense.norm_rope(x, k, v, pos, *want, q_weight=w, k_weight=w)
    dense.norm_rope(x, k, v, pos, x, k, v, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (x, k, v)))
    step.close(), dense.close()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_fill_is_the_dense_rows(dt):
    """Where qkv and cache type are one, the cache holds the dense outputs' bits; without weights, ftd_rope_qkv's values."""
    import torch
    n, Hq, Hkv, D = 19, 4, 2, 128
    t = getattr(torch, TORCH[dt])
    x = torch.randn((n, (Hq + 2 * Hkv) * D), device="cuda").to(t)
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:]
    w = torch.randn(D, device="cuda").to(t)
    step = ftd.DecodeStep(2, Hq, Hkv, D, 32, dt, dt)
    step.set_rope()
    pos = dev(np.arange(n, dtype=np.int32)[None] * 7)
    qo, ko, vo = (torch.empty((n, h, D), dtype=t, device="cuda") for h in (Hq, Hkv, Hkv))
    qo2 = torch.empty_like(qo)
    slots = dev(np.random.default_rng(2).permutation(64)[:n].astype(np.int32))
    kc, vc = (torch.zeros((2, Hkv, 32, D), dtype=t, device="cuda") for _ in range(2))
    step.norm_rope(q, k, v, pos, qo, ko, vo, q_weight=w, k_weight=w)
    step.norm_rope(q, k, v, pos, qo2, q_weight=w, k_weight=w, slots=slots, k_cache=kc, v_cache=vc)
    s = slots.long()
    assert torch.equal(qo, qo2)
    assert torch.equal(kc[s // 32, :, s % 32], ko) and torch.equal(vc[s // 32, :, s % 32], vo)
    step.norm_rope(q, k, v, pos, qo, ko, vo)
    q3, k3, v3 = (torch.empty_like(o) for o in (qo, ko, vo))
    step.rope(q, k, v, pos, q3, k3, v3)
    torch.cuda.synchronize()
    assert torch.equal(qo, q3) and torch.equal(ko, k3) and torch.equal(vo, v3)
    step.close()


@pytest.mark.parametrize("dt,shift", [("f16", 0), ("f16", 4), ("f32", 0), ("f32", 1), ("f32", 2)])
def test_codes_are_rounded_quotients(dt, shift):
    """INT8 codes are rint(x / absmax * 127) as IEEE divisions give it, exactly: halves and their neighbours (scales of
    a power of two make x / scale a half), rows of any magnitude, zeros, infinities and NaN."""
    import torch
    n, D = 1500, 128
    rng = np.random.default_rng(5)
    x = rng.standard_normal((n, D)).astype(np.float32)
    x[:700] *= np.exp2(rng.integers(-9, 9, (700, 1))).astype(np.float32)
    half = rng.integers(-127, 127, (400, D)) + 0.5
    half[:, 0] = 127.0  # the scale is 1, 2 or 1/4
    half *= np.exp2(rng.integers(-2, 2, (400, 1)))
    x[700:1100] = half
    if dt == "f32":  # and one step on either side of a half
        x[900:1100, 1:] = np.nextafter(x[900:1100, 1:], rng.choice([-1e9, 1e9], (200, D - 1)).astype(np.float32))
    x[1100:1110] = 0.0
    x[1110, 5] = np.inf
    x[1111, 7] = np.nan
    x[1112:1120] *= 1e-6
    x = x.astype(np.float16).astype(np.float32) if dt == "f16" else x
    step = ftd.DecodeStep(1, 1, 1, D, 1504, dt, "i8")
    step.set_rope()
    t = getattr(torch, TORCH[dt])
    v = torch.zeros(n * D + shift, dtype=t, device="cuda")[shift:].view(n, D)
    v.copy_(dev(x))
    zero, out = torch.zeros((n, D), dtype=t, device="cuda"), torch.empty((n, D), dtype=t, device="cuda")
    kc, vc = (torch.zeros((1, 1, 1504, D), dtype=torch.int8, device="cuda") for _ in range(2))
    sc = torch.zeros((2, 1, 1, 1504), device="cuda")
    step.norm_rope(zero, zero, v, dev(np.zeros((1, n), np.int32)), out, slots=dev(np.arange(n, dtype=np.int32)), k_cache=kc,
                   v_cache=vc, scales=sc)
    torch.cuda.synchronize()
    assert step.get_error() == ftd.FTD_OK
    ok = np.ones(n, bool)
    ok[1110:1112] = False
    amax = np.abs(x[ok]).max(1)
    scale = np.where(amax == 0, np.float32(1), amax / np.float32(127)).astype(np.float32)
    codes = np.rint(x[ok] / scale[:, None])
    assert np.abs(codes).max() <= 127
    assert np.array_equal(sc[1, 0, 0, :n].cpu().numpy()[ok], scale)
    assert np.array_equal(vc[0, 0, :n].cpu().numpy()[ok], codes.astype(np.int8))
    # beside an infinity the scale is infinite and every finite code is 0; beside a NaN the others are as without it
    others = np.arange(D) != 5
    assert np.isinf(float(sc[1, 0, 0, 1110])) and not vc[0, 0, 1110].cpu().numpy()[others].any()
    others = np.arange(D) != 7
    s = np.abs(x[1111, others]).max() / np.float32(127)
    assert np.array_equal(vc[0, 0, 1111].cpu().numpy()[others], np.rint(x[1111, others] / s).astype(np.int8))
    assert not kc.any() and bool((sc[0, 0, 0, :n] == 1).all())
    step.close()


def test_slots_past_the_end():
    """Slots past the cache write nothing and raise the error; the pool serves where no caches are given."""
    import torch
    from tests.gpu_util import device_view
    for opts, end in ((dict(), 64), (dict(page_size=128, num_pages=2), 256)):
        step = ftd.DecodeStep(2, 2, 1, 64, 32 if not opts else 256, "f32", "f32", **opts)
        step.set_rope()
        x = torch.ones((3, 2, 64), device="cuda")
        k = torch.ones((3, 1, 64), device="cuda")
        out = torch.empty_like(x)
        pos = dev(np.zeros((1, 3), np.int32))
        step.norm_rope(x, k, k.clone(), pos, out, slots=dev(np.array([end - 1, end, (1 << 31) - 1], np.int32)))
        torch.cuda.synchronize()
        assert step.get_error() == ftd.FTD_ERR_BAD_PAGE
        kp, vp, _ = step.cache_ptrs()
        for p in (kp, vp):
            rows = device_view(p, (end, 64), np.float32)
            assert bool((rows[end - 1] == 1).all()) and not rows[:end - 1].any()
        step.close()


def test_refusals():
    import torch
    step = ftd.DecodeStep(2, 4, 2, 64, 32, "f16", "f16")
    h = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    pos = torch.zeros((1, 5), dtype=torch.int32, device="cuda")
    ok = dict(q=h(5, 4, 64), k=h(5, 2, 64), v=h(5, 2, 64), positions=pos, q_out=h(5, 4, 64))
    kc, vc, slots = h(2, 2, 32, 64), h(2, 2, 32, 64), torch.zeros(5, dtype=torch.int32, device="cuda")
    with pytest.raises(ftd.FtdError, match="set_rope"):
        ftd.check(ftd.ftd_norm_rope_qkv(step.ctx, 16, 16, 16, 0, 0, 0, 0, 0, 1e-6, 0.0, 16, 1, 16, 16, 16, 0, 0, 0, 0, 0))
    step.set_rope()
    n = ftd.ftd_kernel_launches()
    fill = dict(slots=slots, k_cache=kc, v_cache=vc)
    dense = dict(k_out=h(5, 2, 64), v_out=h(5, 2, 64))
    for kw in (dict(), dict(k_out=dense["k_out"]), dict(dense, k_cache=kc), dict(fill, **dense), dict(fill, v=None),
               dict(fill, k_cache=ok["k"].new_zeros(2, 2, 32, 65)), dict(fill, v_cache=kc), dict(fill, slots=slots.long()),
               dict(fill, slots=slots[:4]), dict(fill, q_out=kc.view(-1)[:1280].view(5, 4, 64)), dict(dense, eps=-1.0),
               dict(dense, eps=float("nan")), dict(dense, weight_offset=float("inf")), dict(dense, q_weight=h(63)),
               dict(dense, k_weight=torch.zeros(64, device="cuda")), dict(dense, q_weight=ok["q_out"].view(-1)[:64]),
               dict(dense, q_out=ok["q"][:, :3]), dict(dense, v_out=dense["k_out"]), dict(fill, k_cache=kc.float())):
        with pytest.raises((ftd.FtdError, ValueError)):
            step.norm_rope(**dict(ok, **kw))
    assert ftd.ftd_kernel_launches() == n
    step.norm_rope(**dict(ok, **fill))
    step.norm_rope(**dict(ok, **dense))
    torch.cuda.synchronize()
    assert ftd.ftd_kernel_launches() == n + 2 and step.get_error() == ftd.FTD_OK
    step.close()
