"""Paged FP8 attention step (oracle).

TEST INFRASTRUCTURE ONLY -- not part of the product path.

What the pages describe: a paged KV cache of 16-token blocks stored as E4M3
with one scale each for keys and values, restored inside the attention
("FP8 Quantization", D.4; "[vLLM] FP8", KV cache quantization; "Quantization
guide for serving: FP8, AWQ, GPTQ", KV-cache FP8 section).

What is computed here, in float64 from the definitions:
    slot map:  request r holds computed[r] tokens in ceil(computed / page)
               blocks and gets new[r] more; blocks come from the free list in
               request order; token at position p has slot
               block[p // page] * page + p % page.
    norm, rotation:  y = x / sqrt(mean x^2 + eps) * w, then the pairs (a, b)
               of the first rot values turn to (a c - b s, b c + a s).
    attention: softmax over the visible keys of scale * ks * <q, K>, times
               vs * V; key j of a query at position p is visible if j <= p and
               (window == 0 or p - j < window or j < sinks) and its page is
               mapped; a prefix's keys are visible to every query.  A row of no
               visible key is zeros, its log-sum-exp -inf.

Each comparison carries its own tolerance, derived from the roundings that
the definition leaves open: see ``attention_ref`` and ``norm_rope_ref``.
"""

import numpy as np

from . import e4m3


def slot_map_ref(computed, new, table, free, page, T):
    """(table, slots, positions, offsets, lens, taken), by handing out blocks one by one."""
    table = np.array(table, dtype=np.int32, copy=True)
    slots = np.full(T, -1, dtype=np.int64)
    positions = np.full(T, -1, dtype=np.int64)
    offsets, lens, taken, t = [0], [], 0, 0
    for r in range(len(computed)):
        c, n = max(0, int(computed[r])), max(0, int(new[r]))
        blocks = {i: int(table[r, i]) for i in range(min(-(-c // page), table.shape[1]))}
        for i in range(-(-c // page), -(-(c + n) // page)):
            b = int(free[taken]) if taken < len(free) else -1
            taken += 1
            if i < table.shape[1]:
                table[r, i] = b
                blocks[i] = b
        for p in range(c, c + n):
            if t < T:
                b = blocks.get(p // page, -1)
                positions[t] = p
                slots[t] = b * page + p % page if b >= 0 else -1
            t += 1
        offsets.append(t)
        lens.append(c + n)
    return table, slots, positions, np.array(offsets), np.array(lens), taken


def norm_rope_ref(x, w, eps, cos, sin, interleaved):
    """x [T, H, D], w [D], cos / sin [T, rot / 2], all float64 -> (result, tolerance before rounding).

    The tolerance covers the fp32 evaluation: the mean of squares is a sum of
    positive terms, at most 8 fused and 6 butterfly additions deep, so 14
    roundings of 2^-24, halved by the root; the root, the reciprocal, two
    products, the weight and cosine products and the final fused addition add
    8: under 16 half-ulps in relation to the magnitudes that enter, doubled
    here.  The tolerance is relative to |a c| + |b s|.
    """
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    rot = 2 * cos.shape[1]
    z, mag = y.copy(), np.abs(y)
    c, s = cos[:, None, :], sin[:, None, :]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    mag[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
    mag[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
    return z, mag * 32 * 2.0 ** -24


def key_slots(row, length, page, num_blocks):
    """Cache slot of each key 0 .. length - 1, -1 where no block is mapped."""
    j = np.arange(length)
    b = np.full(length, -1, dtype=np.int64)
    there = j // page < len(row)
    b[there] = np.asarray(row, dtype=np.int64)[j[there] // page]
    return np.where((b >= 0) & (b < num_blocks), b * page + j % page, -1)


def attention_ref(q, key_cache, value_cache, table, lens, offsets, scale, ks, vs, window=0, sinks=0,
                  prefix_row=None, prefix_len=0):
    """q [T, Hq, D] float64, caches uint8 [blocks, page, Hk, D].

    Returns (out, lse, tol, tol_lse, covered): tol bounds |kernel - out|
    including the bf16 rounding, from
      scores: D exact products summed in fp32: D 2^-24 sum |q k| |c|, and two
              roundings (the scale factor, its product) of the score itself;
      exp2:   the difference's rounding and the instruction's 1 ulp, 2^-22;
      P:      fp16, the row's largest at 2^10 or above: 2^-11 relative, 2^-35 of the
              largest absolute where it is subnormal;
      sums:   fp32 over L terms and the joins of parts, (L + 64) 2^-24;
      result: bf16, 2^-8 relative.
    """
    nb, page, Hk, D = key_cache.shape
    T, Hq, _ = q.shape
    G = Hq // Hk
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    tol, tol_lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    covered = np.zeros(T, dtype=bool)
    kd = e4m3.decode(key_cache).astype(np.float64).reshape(-1, Hk, D)
    vd = e4m3.decode(value_cache).astype(np.float64).reshape(-1, Hk, D)
    c = scale * ks
    for r in range(len(lens)):
        a, e = int(offsets[r]), int(offsets[r + 1])
        n, length = e - a, max(0, int(lens[r]))
        if n <= 0:
            continue
        covered[a:e] = True
        slots = key_slots(table[r], length, page, nb)
        j, p = np.arange(length)[None], (length - n + np.arange(n))[:, None]
        vis = (j <= p) & (slots >= 0)[None]
        if window > 0:
            vis &= (p - j < window) | (j < sinks)
        if prefix_row is not None:
            ps = key_slots(prefix_row, max(0, prefix_len), page, nb)
            slots = np.concatenate([ps, slots])
            vis = np.concatenate([np.broadcast_to((ps >= 0)[None], (n, len(ps))), vis], 1)
        if vis.shape[1] == 0:
            continue
        sl = np.where(slots >= 0, slots, 0)
        for h in range(Hk):
            k, v = kd[sl, h], vd[sl, h]
            vnan = np.isnan(v)
            v0 = np.where(vnan, 0.0, v)
            for g in range(h * G, (h + 1) * G):
                x = q[a:e, g]
                s = np.where(vis, (x @ k.T) * c, -np.inf)
                mag = np.where(vis, (np.abs(x) @ np.abs(k).T) * abs(c), 0.0)
                top = s.max(1, keepdims=True)
                base = np.where(np.isneginf(top), 0.0, top)
                w = np.exp(s - base)
                l = w.sum(1, keepdims=True)
                some = l > 0
                l1 = np.where(some | np.isnan(l), l, 1.0)
                o = np.where(some | np.isnan(l), (w @ v0) / l1 * vs, 0.0)
                o = np.where((vis.astype(float) @ vnan) > 0, np.nan, o)
                out[a:e, g] = o
                with np.errstate(divide="ignore"):
                    lse[a:e, g] = (np.log(l) + base)[:, 0]
                ds = (np.nanmax(mag, 1, keepdims=True) * D * 2.0 ** -24 +
                      np.nanmax(np.where(vis & np.isfinite(s), np.abs(s), 0), 1, keepdims=True) *
                      4 * 2.0 ** -24)
                sums = (vis.shape[1] + 64) * 2.0 ** -24
                absv = (w @ np.abs(v0)) / l1 * abs(vs)
                rel = 2.0 ** -11 + 2 * ds + 2 * 2.0 ** -22 + 2 * sums
                tol[a:e, g] = np.abs(np.where(np.isnan(o), 0, o)) * 2.0 ** -8 + absv * rel + \
                    (vis @ np.abs(v0)) / l1 * abs(vs) * 2.0 ** -35
                tol_lse[a:e, g] = (ds + sums + 2.0 ** -22)[:, 0] + \
                    np.abs(np.where(np.isfinite(lse[a:e, g]), lse[a:e, g], 0)) * 2.0 ** -22
    return out, lse, tol, tol_lse, covered
