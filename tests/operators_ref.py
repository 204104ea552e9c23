"""Plain 64-bit forms of the operators around the decode step, for the tests, in numpy and
apart from the library's code and from the C oracle."""
from __future__ import annotations

import numpy as np

from synthetic import Workload, gen_all, to_storage

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def widen(a, dt):
    """Stored values as float64."""
    a = np.asarray(a)
    if dt == "bf16":
        return (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return a.astype(np.float64)


# ----------------------------------------------------------------- rotary
def pair_axes(n_axes, sections, order):
    if order == "sections":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while sum(left):
        for a in range(n_axes):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def rope(x, positions, inv_freq, axes, pairing):
    """x [n][H][D] float64 turned by positions [axes][n] (integers) and inv_freq [R / 2]; the
    angles in extended precision."""
    y = x.copy()
    half = len(axes)
    for i in range(half):
        a, b = (i, i + half) if pairing == "halves" else (2 * i, 2 * i + 1)
        w = positions[axes[i]].astype(np.longdouble) * np.longdouble(inv_freq[i])
        c, s = np.cos(w).astype(np.float64)[:, None], np.sin(w).astype(np.float64)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


# -------------------------------------------------------------- attention
def step_case(cache, qkv, B, Hq, Hkv, D, Lmax, lens, T=1, bias=0.1, seed=31):
    w = Workload("ops", B=B, Hq=Hq, Hkv=Hkv, D=D, Lmax=Lmax, qkv_dtype=qkv, cache_dtype=cache, bias_std=bias,
                 seed=seed, q_len=T)
    return w, gen_all(w, seed=seed, seq_lens=np.array(lens, np.int32), fill_beyond="nan")


def cache_rows(w, cache, scales, plane, b, n):
    """The first n rows of slot b as float64 [Hkv][n][D] (INT8: codes times scales)."""
    x = widen(cache[b, :, :n], w.cache_dtype)
    return x * scales[plane, b, :, :n, None].astype(np.float64) if scales is not None else x


def queries(w, inp, b):
    """q + bias of slot b, float64 [T][Hq][D] (a step with one token has no token axis)."""
    q = widen(inp["q"][b], w.qkv_dtype).reshape(-1, w.Hq, w.D)
    if inp.get("bias") is not None:
        q = q + widen(inp["bias"], w.qkv_dtype)[:w.Hq * w.D].reshape(w.Hq, w.D)
    return q


def weights(w, q, k, lo, hi):
    """Softmax weights [Hq][n] of one token's queries q [Hq][D] over rows k [Hkv][n][D], of which
    it sees lo <= t < hi, and the largest sum of |q_d k_d| behind a score."""
    g = w.Hq // w.Hkv
    kk = np.repeat(k, g, axis=0)  # [Hq][n][D]
    s = np.einsum("hd,hnd->hn", q, kk) / np.sqrt(w.D)
    s[:, :lo] = -np.inf
    s[:, hi:] = -np.inf
    p = np.exp(s - s.max(axis=1, keepdims=True))
    mass = np.einsum("hd,hnd->hn", np.abs(q), np.abs(kk))[:, lo:hi].max() / np.sqrt(w.D)
    return p / p.sum(axis=1, keepdims=True), mass


def appended_i8(w, inp, b, which):
    """Codes [Hkv][T][D] and scales [Hkv][T] of slot b's new rows: the scored step's quantiser in fp32."""
    x = np.asarray(widen(inp[which + "_new"][b], w.qkv_dtype), np.float32).reshape(-1, w.Hkv, w.D)
    if inp.get("bias") is not None:
        o = (w.Hq + (w.Hkv if which == "v" else 0)) * w.D
        x = x + np.asarray(widen(inp["bias"], w.qkv_dtype), np.float32)[o:o + w.Hkv * w.D].reshape(w.Hkv, w.D)
    x = x.transpose(1, 0, 2)
    top = np.abs(x).max(axis=-1)
    s = np.where(top == 0, np.float32(1), top * (np.float32(1) / np.float32(127))).astype(np.float32)
    return np.clip(np.rint(x / s[..., None]), -127, 127).astype(np.int8), s


def added_weights(w, inp, k_after, scales_after, b, window=0):
    """Sum over the query rows of each kv head of slot b's weights, [Hkv][L + T], and the largest mass."""
    L, T, g = int(inp["seq_lens"][b]), w.q_len, w.Hq // w.Hkv
    k = cache_rows(w, k_after, scales_after, 0, b, L + T)
    q = queries(w, inp, b)
    out, mass = np.zeros((w.Hkv, L + T)), 0.0
    for j in range(T):
        lo = max(0, L + j + 1 - window) if window else 0
        p, m = weights(w, q[j], k, lo, L + j + 1)
        out += p.reshape(w.Hkv, g, -1).sum(axis=1)
        mass = max(mass, m)
    return out, mass


def weight_tolerance(w, mass, bias):
    """Relative error of a weight.  A score is a dot product of D fp32 products, off by at most
    (D + 4) half steps of its mass (order of summation included); a 16-bit q with a bias is kept
    as two 16-bit parts, which leave at most 2^-18 (bf16) of it; INT8 rows add the rounding of
    their scales' products and of the three-level query.  A weight's relative error is its
    score's error, plus that of the row's maximum and sum (as much again), plus the exponential's
    and the products' few half steps."""
    rel = (w.D + 8) * 2.0 ** -24
    if bias and w.cache_dtype == "bf16":
        rel += 2.0 ** -18
    return 2.0 * mass * rel + 16 * 2.0 ** -24


def cross(w, q, bias, k, v, scales, mem_lens):
    """Cross attention in float64: q [B][T][Hq][D] storage, memories in the cache's storage."""
    B, T = q.shape[:2]
    g = w.Hq // w.Hkv
    out = np.zeros((B, T, w.Hq, w.D))
    for b in range(B):
        n = int(mem_lens[b])
        if not 0 < n <= w.Lmax:
            continue
        kk, vv = cache_rows(w, k, scales, 0, b, n), cache_rows(w, v, scales, 1, b, n)
        qq = widen(q[b], w.qkv_dtype)
        if bias is not None:
            qq = qq + widen(bias, w.qkv_dtype).reshape(w.Hq, w.D)
        for j in range(T):
            p, _ = weights(w, qq[j], kk, 0, n)
            out[b, j] = np.einsum("hn,hnd->hd", p, np.repeat(vv, g, axis=0))
    return out


# --------------------------------------------------------------- eviction
def evict_moves(acc, pos, L, next_pos, budget, recent, sinks):
    """(source, destination) rows for one kv head of a slot with L rows."""
    if L <= budget:
        return []
    order = []
    for t in range(L):
        safe = 0 <= pos[t] < sinks or (recent > 0 and pos[t] >= int(next_pos) - recent)
        a = float(acc[t])
        order.append((0 if safe else 1, (0.0 if safe else (float("inf") if np.isnan(a) else -a)), t))
    # NaN ranks behind every number, -inf included
    order.sort(key=lambda k: (k[0], np.isnan(acc[k[2]]) and k[0] == 1, k[1], k[2]))
    kept = {t for _, _, t in order[:budget]}
    holes = [t for t in range(budget) if t not in kept]
    movers = sorted(t for t in kept if t >= budget)
    return list(zip(movers, holes))


def evict(planes, acc, pos, lens, next_pos, budget, recent, sinks):
    """Moves rows of every array of planes ([B][Hkv][Lmax]...) in place; returns the new lengths."""
    new = np.array(lens).copy()
    Lmax = acc.shape[2]
    a0, p0 = acc.copy(), pos.copy()
    for b in range(acc.shape[0]):
        L = int(lens[b])
        if not budget < L <= Lmax:
            continue
        new[b] = budget
        for h in range(acc.shape[1]):
            for s, d in evict_moves(a0[b, h], p0[b, h], L, next_pos[b], budget, recent, sinks):
                for x in planes:
                    x[b, h, d] = x[b, h, s]
    return new


def store(x, dt):
    return to_storage(np.asarray(x, np.float32), dt)
