"""The step oracle against closed forms and brute force (CPU only)."""

import math

import numpy as np
import pytest

from oracle import quant, step
from workloads import synth


def bits(x):
    return synth.f32_to_bf16_bits(np.asarray(x, dtype=np.float32))


def test_norm_of_a_constant_row_and_of_one_value():
    v, tol = step.norm_ref(bits([[3.0] * 128, [0.0] * 64 + [2.0] + [0.0] * 63]), bits([0.5] * 128), 0.0)
    assert np.allclose(v[0], 0.5, atol=0, rtol=1e-15)
    assert math.isclose(v[1, 64], 0.5 * math.sqrt(128), rel_tol=1e-15) and np.count_nonzero(v[1]) == 1
    assert (tol >= 0).all()


def test_addition_rounds_to_even():
    a, b = bits([256.0, 256.0, 1.0]), bits([1.0, 3.0, -1.0])
    assert list(quant.bf16_bits_to_f32(step.add_ref(a, b))) == [256.0, 260.0, 0.0]


def test_axes():
    assert step.axes_ref([2, 1, 1], False) == [0, 0, 1, 2]
    assert step.axes_ref([2, 1, 1], True) == [0, 1, 2, 0]
    assert step.axes_ref([4, 1, 1], True) == [0, 1, 2, 0, 0, 0]
    assert step.axes_ref([3, 2, 0], True) == [0, 1, 0, 0, 1]
    # the rule as the header words it
    for s in ([24, 20, 20], [8], [5, 3], [10, 2, 2, 2], [7, 1, 4]):
        half, n = sum(s), len(s)
        want = [i % n if i % n and i < n * s[i % n] else 0 for i in range(half)]
        assert step.axes_ref(s, True) == want


def test_pack_layout():
    v = np.arange(16, dtype=np.uint8)[None]
    got = step.int4_pack_ref(v)[0]
    assert list(got) == [0x20, 0x64, 0x31, 0x75, 0xa8, 0xec, 0xb9, 0xfd]
    dword = int.from_bytes(bytes(got[:4]), "little")
    assert [dword >> 4 * i & 15 for i in range(8)] == [0, 2, 4, 6, 1, 3, 5, 7]


@pytest.mark.parametrize("symmetric", [False, True])
def test_quantization_error_and_codes(symmetric):
    rng = np.random.default_rng(3)
    w = bits(rng.standard_normal((5, 256)))
    w[2, :64] = 0
    w[3, :64] = np.abs(quant.bf16_bits_to_f32(w[3, :64])).view(np.uint32) >> 16   # one sign only
    c, s, z = step.int4_quant_ref(w, 64, symmetric)
    zero = np.full(s.shape, 8.0) if symmetric else z.astype(np.float64)
    back = (c.reshape(5, 4, 64) - zero[..., None]) * s[..., None]
    off = np.abs(back.reshape(5, 256) - quant.bf16_bits_to_f32(w))
    # half a step, and half a step more where the zero point was rounded at an end
    assert (off.reshape(5, 4, 64) <= s[..., None] * (0.5 if symmetric else 1.0) * (1 + 1e-6)).all()
    assert (s[2, 0] == 0) and c.max() == 15 and (c.min() == 1 if symmetric else c.min() == 0)


def test_int4_product_by_loops():
    rng = np.random.default_rng(4)
    x, c = bits(rng.standard_normal((2, 128))), rng.integers(0, 16, (3, 128))
    s, z = rng.random((3, 4)).astype(np.float32), rng.integers(0, 16, (3, 4)).astype(np.uint8)
    got, tol = step.int4_linear_ref(x, c, s, z)
    xf = quant.bf16_bits_to_f32(x)
    for m in range(2):
        for n in range(3):
            want = math.fsum(float(xf[m, k]) * float(s[n, k // 32]) * (int(c[n, k]) - int(z[n, k // 32]))
                             for k in range(128))
            assert math.isclose(got[m, n], want, rel_tol=1e-12, abs_tol=1e-12)
    # 32 additions to a group of magnitude (31 + 31) sum |x|, scales below 1; 24 roundings of 2^-24
    # of at most 15 sum |x|
    most = np.abs(xf).sum(1, keepdims=True) * (32 * 62 * 2.0 ** -23 + 15 * 24 * 2.0 ** -24)
    assert (tol > 0).all() and (tol <= most).all()


def test_logprobs_closed_forms():
    x = np.array([[0.0, 0.0, 0.0, 0.0], [math.log(3), 0.0, -math.inf, -math.inf],
                  [-math.inf] * 4, [math.nan, 0, 0, 0], [math.inf, 0, 0, 0]])
    got, tol = step.logprobs_ref(x, np.array([2, 1, 0, 1, -1]), 3, 1.0)
    assert np.allclose(got["logprobs"][:2], [-math.log(4)] * 2)
    assert got["logprobs"][2] == -math.inf and np.isnan(got["logprobs"][3]) and got["logprobs"][4] == 0
    assert list(got["ranks"]) == [0, 1, 0, -1, -1]
    assert np.allclose(got["entropy"][:3], [math.log(4), math.log(4) - 0.75 * math.log(3), 0])
    assert got["ids"].tolist() == [[0, 1, 2], [0, 1, 2], [0, 1, 2], [-1] * 3, [-1] * 3]
    assert got["lse"][2] == -math.inf and np.isnan(got["lse"][3:]).all()
    assert (tol(got["lse"]) > 0).all()
