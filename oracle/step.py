"""What a serving step runs around the linears and the attention (oracle).

TEST INFRASTRUCTURE ONLY -- not part of the product path.

In float64 from the definitions:
    norm:     r = bf16(x + residual); v = r / sqrt(mean r^2 + eps) * w.
    axes:     the cosines and sines of each pair, from its axis' position.
    4 bits:   out = sum_g s_g sum_{k in g} x_k (c_k - z_g), W4A16 with groups
              ("Quantization guide for serving: FP8, AWQ, GPTQ").
    log probabilities: z = scale x, lse = log sum exp z, z[token] - lse,
              -sum p log p, the largest k by (value, lower index).

Each comparison carries its own tolerance, derived from the roundings that
the definition leaves open.
"""

import numpy as np

from . import quant
from .kv_cache import bf16_rne_bits


def add_ref(x_bits, r_bits):
    """bf16(x + r) with the sum in fp32, as bits."""
    return bf16_rne_bits(quant.bf16_bits_to_f32(x_bits) + quant.bf16_bits_to_f32(r_bits))


def norm_ref(r_bits, w_bits, eps):
    """(v float64, tolerance of the fp32 evaluation).

    The mean is a sum of squares, positive terms: at most 64 fused additions
    of a lane's 8 chunks of 8 values, 6 across the wave and 16 across waves,
    86 roundings, halved by the root; the mean's product and eps, the root's
    reciprocal (1 ulp) and two products add 5: under 48 half-ulps of 2^-24.
    Doubled here.
    """
    r = quant.bf16_bits_to_f32(r_bits).astype(np.float64)
    w = quant.bf16_bits_to_f32(w_bits).astype(np.float64)
    v = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * w
    return v, np.abs(v) * 96 * 2.0 ** -24


def axes_ref(sections, in_turn):
    """Axis of each rotated pair, handed out one by one."""
    half, n = sum(sections), len(sections)
    if not in_turn:
        return [a for a in range(n) for _ in range(sections[a])]
    of, left = [], list(sections)
    for i in range(half):
        a = i % n
        if a and left[a]:
            left[a] -= 1
        else:
            a = 0
        of.append(a)
    assert not any(left[1:])
    return of


def int4_pack_ref(values):
    """uint8 values [N, K] -> packed [N, K / 2], by the layout's definition."""
    v = np.asarray(values, dtype=np.uint8).reshape(values.shape[0], -1, 8) & 15
    b = [v[..., 0] | v[..., 2] << 4, v[..., 4] | v[..., 6] << 4,
         v[..., 1] | v[..., 3] << 4, v[..., 5] | v[..., 7] << 4]
    return np.stack(b, -1).reshape(values.shape[0], -1)


def int4_quant_ref(w_bits, group, symmetric):
    """(values [N, K], scales [N, K / group] fp32, zeros) by groups, in fp32 steps."""
    f = np.float32
    w = quant.bf16_bits_to_f32(w_bits)
    g = w.reshape(w.shape[0], -1, group)
    lo = np.minimum(g.min(-1), f(0))
    hi = np.maximum(g.max(-1), f(0))
    s = np.maximum(-lo, hi) / f(7) if symmetric else (hi - lo) / f(15)
    some = s > 0
    div = np.where(some, s, f(1))
    z = np.full(s.shape, f(8)) if symmetric else \
        np.where(some, np.minimum(np.rint(-lo / div), f(15)), f(0))
    c = np.where(some[..., None], np.rint(g / div[..., None]) + z[..., None], z[..., None])
    return (np.clip(c, 0, 15).astype(np.uint8).reshape(w.shape), s.astype(f),
            None if symmetric else z.astype(np.uint8))


def int4_linear_ref(x_bits, values, scales, zeros):
    """(out float64 [M, N], tolerance before the result's rounding).

    Per group of G values the matrix unit sums x (16 + c) and x, exact
    products, in fp32: G additions (each at most 2^-23 of what has gathered,
    were they cut rather than rounded), G 2^-23 of the magnitudes' sum; taking one from the
    other and scaling rounds twice, K / G scaled groups and up to 16 waves'
    parts are added: (K / G + 20) 2^-24 of the scaled groups' magnitude.
    """
    x = quant.bf16_bits_to_f32(x_bits).astype(np.float64)
    (M, K), (N, groups) = x.shape, scales.shape
    G = K // groups
    z = np.full(scales.shape, 8.0) if zeros is None else zeros.astype(np.float64)
    s = scales.astype(np.float64)
    out, tol = np.zeros((M, N)), np.zeros((M, N))
    mag = np.zeros((M, N))
    for g in range(groups):
        xs = x[:, g * G:(g + 1) * G]
        c = values[:, g * G:(g + 1) * G].astype(np.float64)
        part = xs @ (c - z[:, g, None]).T * s[:, g]
        a = np.abs(xs)
        out += part
        tol += (a @ (16 + c).T + a.sum(1, keepdims=True) * (16 + z[:, g])) * np.abs(s[:, g]) * \
            (G * 2.0 ** -23)
        mag += a @ np.abs(c - z[:, g, None]).T * np.abs(s[:, g])
    return out, tol + mag * (groups + 20) * 2.0 ** -24


def logprobs_ref(x, tokens, k, scale):
    """x [T, V] float64 -> dict of outputs and `tol`, a tolerance per row.

    A weight 2^t carries the roundings of x - m, of c = scale log2(e) and of
    their product, 3 2^-24 |t|, and the exponential's ulp, 2^-23; S and D sum at
    most V / 512 + 64 of them one after the other (a thread's own, the wave's,
    the waves', up to 8192 / 64 parts', and the rescaling of each), and
    sum w |t| / S = log2 S - H_2, below 2^5 for any V here.  So log S, D / S and
    what is left of them are within (V / 512 + 256) 2^-24 of their magnitude
    plus 1, and a log probability within 4 2^-24 of its own magnitude on top.
    """
    T, V = x.shape
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        z = x * scale
        bad = np.isnan(x).any(1) | (x == np.inf).any(1)
        top = z.max(1)
        none = np.isneginf(top) & ~bad
        base = np.where(np.isfinite(top), top, 0.0)
        w = np.exp(z - base[:, None])
        S = w.sum(1)
        lse = np.where(bad, np.nan, np.log(S) + base)
        # from the maximum: next to a far lse the differences would be lost, in 64 bits, too
        logp = (z - base[:, None]) - np.log(S)[:, None]
        logp[none] = -np.inf
        entropy = np.where(bad, np.nan, np.where(none, 0.0, np.log(S) - np.where(
            w > 0, w * (z - base[:, None]), 0.0).sum(1) / S))
    given = (tokens >= 0) & (tokens < V)
    at = np.where(given, tokens, 0)
    rows = np.arange(T)
    logp[bad] = np.nan
    mine = np.where(given, logp[rows, at], 0.0)
    ranks = np.where(given & ~bad, (x > x[rows, at][:, None]).sum(1), -1)
    order = np.argsort(-np.where(bad[:, None], 0.0, x), axis=1, kind="stable")[:, :k]
    tops = np.take_along_axis(logp, order, 1)
    order = np.where(bad[:, None], -1, order)
    n = (V / 512 + 256) * 2.0 ** -24
    with np.errstate(invalid="ignore"):
        size = 1.0 + np.log(np.where(S > 0, S, 1.0))

    def tol(v):
        v = np.abs(np.where(np.isfinite(v), v, 0.0))
        return n * (size if v.ndim == 1 else size[:, None]) + 4 * 2.0 ** -24 * v

    return dict(logprobs=mine, ranks=ranks, entropy=entropy, lse=lse, top=tops, ids=order), tol
