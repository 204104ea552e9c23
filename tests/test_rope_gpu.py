"""ftd_rope_qkv against the formula in 64 bits (angles in extended precision): axes and
their orders, both pairings, partial rotation, one token to thousands, far and negative
positions, fused projections, unaligned rows, in place, and the refusals."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from tests import operators_ref as ref
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


TORCH = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def sections_of(pairs, axes):
    return [pairs * (a + 1) // axes - pairs * a // axes for a in range(axes)]


def make(Hq, Hkv, D, dt):
    return ftd.DecodeStep(1, Hq, Hkv, D, 16, dt, dt)


def typed(x, dt):
    """float array as a torch CUDA tensor of type dt, and its values as float64."""
    import torch
    t = torch.from_numpy(np.asarray(x, np.float32)).to(getattr(torch, TORCH[dt])).cuda()
    return t, t.double().cpu().numpy()


def tolerance(x, y, dt, pos_max):
    """x [n][H][D] turned into y.  cos and sin are off by the rounding of the wrapped angle (pi 2^-25),
    sincospi's ulp (2^-24) and what a 53-bit step leaves of the angle (3 2^-53 pos radians at most);
    then two products and a sum, and the bias add: seven half steps of |a| + |b| in all, |a| + |b| at
    most sqrt(2) times the pair's norm, bounded here by 2 max |x| of the head; then the store."""
    big = 2.0 * np.abs(x).max(axis=-1, keepdims=True)
    t = big * (7 * 2.0 ** -24 + 3 * 2.0 ** -53 * pos_max)
    if dt != "f32":
        t = t + np.abs(y) * ref.HALF_STEP[dt] * (1 + 2.0 ** -10) + (2.0 ** -25 if dt == "f16" else 0.0)
    return t


def check(Hq, Hkv, D, dt, n, axes=1, R=0, pairing="halves", order="sections", fused=True, bias=True, far=5000, seed=1,
          shift=0, theta=10000.0):
    """shift: elements by which the fused buffer starts past a 16-byte boundary."""
    import torch
    rng = np.random.default_rng(seed)
    R = R or D
    W = (Hq + 2 * Hkv) * D
    secs = sections_of(R // 2, axes)
    inv = theta ** (-np.arange(0, R, 2) / R)
    step = make(Hq, Hkv, D, dt)
    step.set_rope(axes, secs, rotary_dim=R, pairing=pairing, order=order, inv_freq=inv)
    pos = rng.integers(-far, far, size=(axes, n)).astype(np.int32)
    b_t, b = typed(0.2 * rng.standard_normal(W), dt) if bias else (None, np.zeros(W))
    x_t, x = typed(rng.standard_normal((n, W)), dt)
    if fused:
        buf = torch.zeros(n * W + 64, dtype=x_t.dtype, device="cuda")
        f = buf[shift:shift + n * W].view(n, W)
        f.copy_(x_t)
        q, k, v = f[:, :Hq * D], f[:, Hq * D:(Hq + Hkv) * D], f[:, (Hq + Hkv) * D:]
    else:
        q, k, v = (x_t[:, a:c].contiguous() for a, c in ((0, Hq * D), (Hq * D, (Hq + Hkv) * D), ((Hq + Hkv) * D, W)))
    outs = [torch.full((n, h, D), float("nan"), dtype=x_t.dtype, device="cuda") for h in (Hq, Hkv, Hkv)]
    before = ftd.ftd_kernel_launches()
    step.rope(q, k, v, dev(pos), *outs, bias=b_t)
    assert ftd.ftd_kernel_launches() == before + 1
    torch.cuda.synchronize()
    ax = ref.pair_axes(axes, secs, order)
    z = (x + b).reshape(n, Hq + 2 * Hkv, D)
    turned = ref.rope(z[:, :Hq + Hkv], pos, inv, ax, pairing)
    want = [turned[:, :Hq], turned[:, Hq:], z[:, Hq + Hkv:]]
    src = [z[:, :Hq], z[:, Hq:Hq + Hkv], z[:, Hq + Hkv:]]
    for name, o, y, s in zip("qkv", outs, want, src):
        got = o.double().cpu().numpy()
        err = np.abs(got - y)
        tol = tolerance(s, y, dt, far)
        assert np.all(np.isfinite(got)), name
        assert np.all(err <= tol), (name, float((err / tol).max()))
    step.close()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 64), (128, 64), (128, 32), (64, 8), (128, 22), (64, 2), (128, 120), (64, 52)])
@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
def test_types_and_rotary_dims(dt, D, R, pairing):
    """(8, 120 and 52 leave runs of 4, 4 and 2 pairs, 22 and 2 single ones: narrower accesses.)"""
    check(6, 2, D, dt, 5, axes=1, R=R, pairing=pairing)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("order", ["sections", "interleaved"])
def test_axes(axes, order):
    check(4, 4, 128, "bf16", 37, axes=axes, order=order)
    check(4, 1, 64, "f32", 7, axes=axes, order=order, R=40, pairing="adjacent")


@pytest.mark.parametrize("n", [1, 2, 3, 151, 152, 607, 608, 609, 4999])
@pytest.mark.parametrize("heads", [(1, 1), (7, 1), (32, 32), (64, 8)])
def test_lengths(n, heads):
    if n == 4999 and heads == (32, 32):
        n = 2501
    check(*heads, 128, "bf16", n, axes=3)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_far_positions(far):
    check(2, 2, 128, "f32", 64, far=far)
    check(2, 2, 64, "f32", 64, far=far, theta=1e6, pairing="adjacent")


@pytest.mark.parametrize("shift", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_alignment(dt, shift):
    check(5, 1, 64, dt, 9, shift=shift)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("fused", [False, True])
def test_sources(fused, bias):
    check(8, 2, 128, "f16", 33, fused=fused, bias=bias)


def test_default_theta_and_sections():
    import torch
    step = make(2, 2, 128, "f32")
    step.set_rope()
    x, xd = typed(np.random.default_rng(3).standard_normal((4, 2, 128)), "f32")
    pos = np.array([[0, 1, 77, 4096]], np.int32)
    q, k = x.clone(), x.clone()
    step.rope(q, k, None, dev(pos), q, k)
    torch.cuda.synchronize()
    inv = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    y = ref.rope(xd, pos, inv, [0] * 64, "halves")
    assert np.all(np.abs(q.double().cpu().numpy() - y) <= tolerance(xd, y, "f32", 4096))
    assert torch.equal(q, k)
    assert torch.equal(q[0], x[0])  # position 0 turns nothing
    step.close()


def test_in_place_and_without_values():
    """In place equals out of place, bit for bit; without a bias a value in place is left alone."""
    import torch
    rng = np.random.default_rng(4)
    Hq, Hkv, D, n = 6, 3, 128, 50
    step = make(Hq, Hkv, D, "bf16")
    step.set_rope(3, [16, 24, 24])
    q, _ = typed(rng.standard_normal((n, Hq, D)), "bf16")
    k, _ = typed(rng.standard_normal((n, Hkv, D)), "bf16")
    v, _ = typed(rng.standard_normal((n, Hkv, D)), "bf16")
    pos = dev(rng.integers(0, 500, size=(3, n)).astype(np.int32))
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    step.rope(q, k, v, pos, qo, ko, vo)
    v0 = v.clone()
    step.rope(q, k, v, pos, q, k, v)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(vo, v0) and torch.equal(v, v0)
    step.close()


def test_one_token_in_place_in_a_fused_row():
    import torch
    rng = np.random.default_rng(8)
    step = make(4, 2, 64, "f32")
    step.set_rope()
    row, x = typed(rng.standard_normal((1, 8 * 64)), "f32")
    q, k = row[:, :256], row[:, 256:384]
    pos = dev(np.array([[77]], np.int32))
    want = [torch.empty_like(q), torch.empty_like(k)]
    step.rope(q, k, None, pos, *want)
    step.rope(q, k, None, pos, q, k)
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert np.array_equal(row[:, 384:].double().cpu().numpy(), x[:, 384:])
    step.close()


def test_batched_token_axes():
    """[B, T, heads, D] and slices of a fused [B, T, W] projection."""
    import torch
    rng = np.random.default_rng(5)
    B, T, Hq, Hkv, D = 3, 4, 4, 2, 64
    step = make(Hq, Hkv, D, "f16")
    step.set_rope()
    W = (Hq + 2 * Hkv) * D
    x, _ = typed(rng.standard_normal((B, T, W)), "f16")
    pos = dev(rng.integers(0, 99, size=(1, B * T)).astype(np.int32))
    outs = [[torch.zeros((B, T, h, D), dtype=torch.float16, device="cuda") for h in (Hq, Hkv, Hkv)] for _ in range(2)]
    q, k, v = x[..., :Hq * D], x[..., Hq * D:(Hq + Hkv) * D], x[..., (Hq + Hkv) * D:]
    step.rope(q, k, v, pos, *outs[0])
    step.rope(q.contiguous(), k.contiguous(), v.contiguous(), pos, *outs[1])
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):  # rows of a transposed tensor are no fixed stride apart
        step.rope(q.transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), pos, *outs[0])
    step.close()


def test_graph_and_streams():
    import torch
    rng = np.random.default_rng(6)
    step = make(4, 4, 128, "bf16")
    step.set_rope()
    q, _ = typed(rng.standard_normal((9, 4, 128)), "bf16")
    k, _ = typed(rng.standard_normal((9, 4, 128)), "bf16")
    pos = dev(np.arange(9, dtype=np.int32)[None])
    want = [torch.empty_like(q), torch.empty_like(k)]
    step.rope(q, k, None, pos, *want)
    torch.cuda.synchronize()
    got = [torch.empty_like(q), torch.empty_like(k)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.rope(q, k, None, pos, *got)
    step.set_rope(theta=5.0)  # a captured call keeps the setting it was captured with
    for _ in range(2):
        got[0].zero_(), got[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    step.close()


def test_refusals():
    import torch
    step = make(4, 2, 64, "f16")
    z = torch.zeros(4096, dtype=torch.float16, device="cuda")
    pos = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    p, o = z.data_ptr(), torch.zeros(4096, dtype=torch.float16, device="cuda")
    op = o.data_ptr()

    def call(q=p, k=p + 1024, v=0, qs=0, ks=0, bias=0, positions=pos.data_ptr(), n=2, qo=op, ko=op + 2048, vo=0):
        return ftd.ftd_rope_qkv(step.ctx, q, k, v, qs, ks, bias, positions, n, qo, ko, vo, 0)
    assert call() == ftd.FTD_ERR_INVALID_ARG and "ftd_set_rope" in ftd.ftd_last_error()
    for kw in (dict(n_axes=0), dict(n_axes=5), dict(rotary_dim=63), dict(rotary_dim=66), dict(rotary_dim=-2),
               dict(n_axes=2, sections=[8, 8]), dict(n_axes=2, sections=[40, -8]), dict(theta=-1.0),
               dict(theta=float("nan")), dict(inv_freq=[float("inf")] * 32)):
        with pytest.raises(ftd.FtdError) as e:
            step.set_rope(**kw)
        assert e.value.status == ftd.FTD_ERR_INVALID_ARG, kw
    with pytest.raises(ValueError):
        step.set_rope(inv_freq=[1.0] * 31)
    assert ftd.ftd_set_rope(step.ctx, None) == ftd.FTD_ERR_INVALID_ARG
    step.set_rope()
    n0 = ftd.ftd_kernel_launches()
    for kw in (dict(q=0), dict(k=0), dict(positions=0), dict(qo=0), dict(ko=0), dict(v=p), dict(vo=op), dict(n=-1),
               dict(n=1 << 31), dict(qs=255), dict(ks=127), dict(q=p + 1), dict(qo=op + 1), dict(bias=p + 1),
               dict(positions=pos.data_ptr() + 2),
               dict(qo=p + 16), dict(qo=p, qs=512), dict(ko=op + 16), dict(qo=p + 1024), dict(bias=op)):
        assert call(**kw) == ftd.FTD_ERR_INVALID_ARG, kw
        assert ftd.ftd_last_error() != ""
    assert call(n=0) == ftd.FTD_OK
    assert ftd.ftd_kernel_launches() == n0
    assert call() == ftd.FTD_OK
    torch.cuda.synchronize()
    step.close()
