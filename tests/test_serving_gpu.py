"""The operators of a batch in pages run together, as a serving loop runs them: block tables and slot maps from the
lengths, a shared prompt and the slots' own prompts normed, turned and written by the slot map, then steps behind the prompt,
against one attention in 64 bits over everything that each slot has seen."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from tests import operators_ref as ref
from tests.gpu_util import dev, device_view

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


@pytest.mark.parametrize("cache,D,Hq,Hkv", [("bf16", 128, 16, 2), ("f16", 64, 4, 4), ("i8", 128, 16, 2), ("f32", 64, 6, 2)])
@pytest.mark.parametrize("graphed", [False, True])
def test_serving_loop(cache, D, Hq, Hkv, graphed):
    import torch
    qkv = "f16" if cache == "i8" else cache
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[qkv]
    B, page, lmax, num_pages, P, steps = 5, 128, 512, 24, 333, 6
    rng = np.random.default_rng(11)
    gen = torch.Generator(device="cuda").manual_seed(5)
    step = ftd.DecodeStep(B + 1, Hq, Hkv, D, lmax, qkv, cache, page_size=page, num_pages=num_pages)  # the last slot holds the prompt
    step.enable_prefix()
    step.set_rope()
    W = (Hq + 2 * Hkv) * D
    bias = (0.1 * torch.randn(W, generator=gen, device="cuda")).to(dt)
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt) for _ in range(2))
    inv = 10000.0 ** (-np.arange(0, D, 2) / D)
    axes = [0] * (D // 2)

    def heads(x, pos):
        """Query, key and value heads of projection rows x, in 64 bits."""
        z = (x.double().cpu().numpy() + bias.double().cpu().numpy()).reshape(len(pos), Hq + 2 * Hkv, D)
        out = []
        for a, b, w in ((0, Hq, qw), (Hq, Hq + Hkv, kw)):
            y = z[:, a:b]
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + EPS) * w.double().cpu().numpy()
            out.append(ref.rope(y, np.asarray(pos)[None], inv, axes, "halves"))
        return out + [z[:, Hq + Hkv:]]

    def split(x):
        return x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:]

    # ---- pages and rows of the prompt (slot B) and of the slots' own first tokens ----
    lens = torch.full((B + 1,), -1, dtype=torch.int32, device="cuda")
    own = [0, 1, 127, 128, 140]
    new = dev(np.array(own + [P], np.int32))
    table = torch.full((B + 1, lmax // page), -1, dtype=torch.int32, device="cuda")
    free, n_free = dev(rng.permutation(num_pages).astype(np.int32)), dev(np.array([num_pages], np.int32))
    cap = sum(own) + P + 9  # a padded batch
    slots, at = (torch.zeros(cap, dtype=torch.int32, device="cuda") for _ in range(2))
    offsets = torch.zeros(B + 2, dtype=torch.int32, device="cuda")
    step.tables(lens, new, lens, block_table=table, free_pages=free, n_free=n_free, offsets=offsets, slots=slots, positions=at)
    # own tokens come behind the prompt: their angles are those of position P + j
    owner = torch.searchsorted(offsets, torch.arange(cap, dtype=torch.int32, device="cuda"), right=True) - 1
    pos = torch.where(owner < B, at + P, at).to(torch.int32)
    x = torch.randn((cap, W), generator=gen, device="cuda").to(dt)
    q_out = torch.empty((cap, Hq, D), dtype=dt, device="cuda")
    step.norm_rope(*split(x), pos[None], q_out, bias=bias, q_weight=qw, k_weight=kw, eps=EPS, slots=slots)
    o = offsets.tolist()
    assert o[1:] == np.cumsum(own + [P]).tolist() and lens.tolist() == own + [P]
    _, k64, v64 = heads(x, pos.tolist())
    keys, values = ([a[o[b]:o[b + 1]] for b in range(B + 1)] for a in (k64, v64))
    prefix_table = table[B, :-(-P // page)].clone()
    seen = dev(np.array([P, P, 200, 0, P, 0], np.int32))
    # ---- steps: a page more where a slot needs one, norms and angles of the new tokens, attention ----
    grown, q1, k1, v1 = torch.empty_like(lens), *(torch.empty((B + 1, h, D), dtype=dt, device="cuda") for h in (Hq, Hkv, Hkv))
    out = torch.empty((B + 1, Hq, D), device="cuda")
    xs = torch.empty((B + 1, W), dtype=dt, device="cuda")
    active = lens.clone()
    active[B] = -1  # the prompt's slot takes no step

    def one_step():
        torch.add(active, 1, out=grown)
        grown[B:].fill_(-1)
        step.tables(active, grown, grown, block_table=table, free_pages=free, n_free=n_free)
        step.norm_rope(*split(xs), (active + P)[None], q1, k1, v1, bias=bias, q_weight=qw, k_weight=kw, eps=EPS)
        step.prefix(q1, k1, v1, active, seen, out, block_table=table, prefix_table=prefix_table)
        active.copy_(grown)

    graph = None
    if graphed:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            one_step()
    for i in range(steps):
        xs.copy_(torch.randn((B + 1, W), generator=gen, device="cuda"))
        before = active.tolist()
        graph.replay() if graphed else one_step()
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        assert not got[B].any()
        qn, kn, vn = heads(xs, [max(n, 0) + P if n >= 0 else 0 for n in before])
        for b in range(B):
            keys[b], values[b] = np.concatenate([keys[b], kn[b:b + 1]]), np.concatenate([values[b], vn[b:b + 1]])
            n = int(seen[b])
            k, v = (np.concatenate([a[B][:n], a[b]]).transpose(1, 0, 2).repeat(Hq // Hkv, 0) for a in (keys, values))
            s = np.einsum("hd,hnd->hn", qn[b], k) / np.sqrt(D)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            want = np.einsum("hn,hnd->hd", p, v)
            # q, k and v are rounded to the qkv type (a half step each) and, INT8, to codes (half a step of absmax / 127):
            # a score moves by the sum of |q_d k_d| times twice that, a weight by e twice over, the output by the values' own
            half = ref.HALF_STEP[qkv]
            code = 0.5 / 127 if cache == "i8" else 0.0
            mass = np.einsum("hd,hnd->hn", np.abs(qn[b]), np.abs(k)).max(1) / np.sqrt(D)
            top = np.abs(k).max(2, keepdims=True) * code
            e = mass * (2 * half + 2.0 ** -14) + (np.abs(qn[b])[:, None, :] * top).sum(2).max(1) / np.sqrt(D)
            av = np.einsum("hn,hnd->hd", p, np.abs(v) + np.abs(v).max(2, keepdims=True) * code)
            tol = av * (2 * np.expm1(e)[:, None] + half + 2.0 ** -14) + np.einsum("hn,hnd->hd", p, np.abs(v).max(2, keepdims=True) * code + 0 * v)
            err = np.abs(got[b] - want)
            assert np.all(err <= tol), (b, float((err / tol).max()))
    assert step.get_error() == ftd.FTD_OK
    assert active.tolist() == [n + steps for n in own] + [-1]
    # ---- everything ends: every page comes back ----
    last = active.clone()
    last[B] = P
    step.tables(last, torch.zeros_like(last), last, block_table=table, free_pages=free, n_free=n_free)
    torch.cuda.synchronize()
    assert int(n_free) == num_pages and sorted(free.tolist()) == list(range(num_pages))
    assert not last.any() and step.get_error() == ftd.FTD_OK
    step.close()
