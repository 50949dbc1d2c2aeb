"""Pins of the paged-attention oracle (CPU): every function against a direct
loop over the definition or a closed form."""

import math

import numpy as np
import pytest

from oracle import attention, e4m3


def test_slot_map_by_hand():
    table = np.full((3, 4), -1, dtype=np.int32)
    table[0, 0] = 9
    got = attention.slot_map_ref([3, 0, 0], [3, 0, 5], table, [4, 7, 2, 5], 4, 10)
    t, slots, pos, offs, lens, taken = got
    assert taken == 3                       # one more for request 0, two for request 2
    assert t.tolist() == [[9, 4, -1, -1], [-1] * 4, [7, 2, -1, -1]]
    assert slots.tolist() == [39, 16, 17, 28, 29, 30, 31, 8, -1, -1]
    assert pos.tolist() == [3, 4, 5, 0, 1, 2, 3, 4, -1, -1]
    assert offs.tolist() == [0, 3, 3, 8] and lens.tolist() == [6, 0, 5]


def test_slot_map_without_enough_blocks():
    table = np.full((2, 2), -1, dtype=np.int32)
    t, slots, pos, _, _, taken = attention.slot_map_ref([0, 0], [3, 5], table, [6], 2, 8)
    assert taken == 5                       # 2 and 3 blocks wanted, one there
    assert slots.tolist() == [12, 13, -1, -1, -1, -1, -1, -1]
    assert pos.tolist() == [0, 1, 2, 0, 1, 2, 3, 4]
    assert t.tolist() == [[6, -1], [-1, -1]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_angles(interleaved):
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((5, 2, 32)), np.ones(32)
    ang = rng.uniform(0, 6, (5, 8))
    z, tol = attention.norm_rope_ref(x, w, 0.0, np.cos(ang), np.sin(ang), interleaved)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True))
    assert np.allclose((z * z).mean(-1), 1.0)
    assert np.array_equal(z[..., 16:], y[..., 16:])      # not rotated
    for t in range(5):
        for i in range(8):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 8)
            u = complex(*y[t, 1, [a, b]]) * complex(math.cos(ang[t, i]), math.sin(ang[t, i]))
            assert np.allclose(z[t, 1, [a, b]], [u.real, u.imag])
    z0, _ = attention.norm_rope_ref(x, w, 0.0, np.ones((5, 8)), np.zeros((5, 8)), interleaved)
    assert np.array_equal(z0, y)                         # position 0 turns nothing
    assert (tol < 1e-4).all()


def brute(q, kc, vc, table, lens, offsets, scale, ks, vs, window, sinks, far=None, far_len=0):
    """One query, head and key at a time."""
    nb, page, Hk, D = kc.shape
    T, Hq, _ = q.shape
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -math.inf)

    def of(cache, row, j, h):
        if j // page >= len(row) or not 0 <= row[j // page] < nb:
            return None
        return [float(x) for x in e4m3.decode(cache[row[j // page], j % page, h])]

    for r in range(len(lens)):
        n = offsets[r + 1] - offsets[r]
        for i in range(n):
            t, p = offsets[r] + i, lens[r] - n + i
            for h in range(Hq):
                keys = [(far, j) for j in range(far_len)]
                keys += [(table[r], j) for j in range(max(0, p + 1))
                         if window == 0 or p - j < window or j < sinks]
                seen = []
                for row, j in keys:
                    k = of(kc, row, j, h * Hk // Hq)
                    if k is not None:
                        seen.append((scale * ks * sum(x * y for x, y in zip(q[t, h], k)),
                                     of(vc, row, j, h * Hk // Hq)))
                if seen:
                    top = max(s for s, _ in seen)
                    l = sum(math.exp(s - top) for s, _ in seen)
                    lse[t, h] = top + math.log(l)
                    for d in range(D):
                        out[t, h, d] = vs * sum(math.exp(s - top) * v[d] for s, v in seen) / l
    return out, lse


@pytest.mark.parametrize("window,sinks,prefix", [(0, 0, False), (3, 0, False), (3, 2, False),
                                                 (1, 9, False), (0, 0, True)])
def test_attention_against_loops(window, sinks, prefix):
    rng = np.random.default_rng(5)
    kc, vc = (rng.integers(0, 0x7f, (9, 3, 2, 4), dtype=np.uint8) & 0xbf for _ in range(2))
    kc |= rng.integers(0, 2, kc.shape, dtype=np.uint8) << 7
    q = rng.standard_normal((9, 4, 4))
    table = np.array([[4, 1, 7], [0, -1, 2], [8, 30, 3], [5, 6, 6]])
    lens, offsets = [8, 7, 0, 2], [0, 2, 5, 6, 9]       # the last request: more queries than tokens
    far = np.array([2, 5]) if prefix else None
    far_len = 5 if prefix else 0
    got = attention.attention_ref(q, kc, vc, table, lens, offsets, 0.3, 0.5, 2.0, window, sinks,
                                  far, far_len)
    want = brute(q, kc, vc, table, lens, offsets, 0.3, 0.5, 2.0, window, sinks, far, far_len)
    assert np.allclose(got[0], want[0], rtol=1e-12, atol=1e-12)
    assert np.array_equal(np.isneginf(got[1]), np.isneginf(want[1]))
    fine = np.isfinite(want[1])
    assert np.allclose(got[1][fine], want[1][fine], rtol=1e-12)
    assert got[4].all()


def test_nan_values_reach_only_rows_that_see_them():
    kc = np.zeros((1, 4, 1, 2), dtype=np.uint8)
    vc = np.zeros((1, 4, 1, 2), dtype=np.uint8)
    vc[0, 2, 0, 1] = 0x7f
    out = attention.attention_ref(np.ones((4, 1, 2)), kc, vc, np.array([[0]]), [4], [0, 4], 1.0, 1.0,
                                  1.0)[0]
    assert np.isnan(out[2:, 0, 1]).all() and not np.isnan(out[:2]).any()
    assert not np.isnan(out[..., 0]).any()
    kc[0, 3, 0, 0] = 0xff                               # a NaN key makes the whole row NaN
    out = attention.attention_ref(np.ones((4, 1, 2)), kc, vc, np.array([[0]]), [4], [0, 4], 1.0, 1.0,
                                  1.0)[0]
    assert np.isnan(out[3]).all() and not np.isnan(out[:2]).any()


def test_tolerance_is_tight():
    """The tolerance is of the order of the bf16 rounding: it would not hide a wrong key."""
    rng = np.random.default_rng(6)
    kc, vc = (rng.integers(0x20, 0x48, (20, 16, 1, 64), dtype=np.uint8) for _ in range(2))
    vc |= rng.integers(0, 2, vc.shape, dtype=np.uint8) << 7
    q = rng.standard_normal((1, 1, 64))
    args = (np.arange(20)[None], [300], [0, 1], 0.1, 0.5, 1.0)
    out, _, tol, _, _ = attention.attention_ref(q, kc, vc, *args)
    less = attention.attention_ref(q, kc, vc, np.arange(20)[None], [299], [0, 1], 0.1, 0.5, 1.0)[0]
    assert (np.abs(less - out) > tol).mean() > 0.3
