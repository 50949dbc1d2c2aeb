"""fp8_add_rms_norm_quant against the oracle (needs a gfx950 GPU).

The residual bit for bit; the norm within half a bf16 step and the tolerance
of its fp32 evaluation; scales within that tolerance; codes between the codes of
the float64 value moved down and up by it."""

import numpy as np
import pytest
import torch

from oracle import e4m3, quant, step
from workloads import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_w8a8_block_amd as fp8


def dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def normal(rng, *shape):
    return synth.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def wide(bits, extra):
    """The rows as a slice of wider ones."""
    t = torch.full((bits.shape[0], bits.shape[1] + extra), 9.0, dtype=torch.bfloat16, device="cuda")
    t[:, :bits.shape[1]] = dev(bits)
    return t[:, :bits.shape[1]]


def check_codes(codes, scales, v, tol, per):
    """Dynamic codes and scales of float64 values v, `per` to a scale."""
    T, H = v.shape
    g = np.abs(v).reshape(T, -1, per).max(-1) / 448
    slack = tol.reshape(T, -1, per).max(-1) / 448 + g * 2.0 ** -23
    s = scales.cpu().numpy().astype(np.float64).reshape(T, -1)
    assert (np.abs(s - g) <= slack).all()
    s = np.repeat(s, per, 1)
    check_quotients(codes, np.divide(v, s, out=v * 0, where=s > 0),
                    np.divide(tol, s, out=tol * 0, where=s > 0))


def check_quotients(codes, z, tol):
    """Codes between those of z moved down and up (decoded: codes are monotone)."""
    got = e4m3.decode(codes.cpu().numpy()).astype(np.float64)
    lo, hi = (e4m3.decode(e4m3.encode((z + f * (tol + np.abs(z) * 2.0 ** -22)).astype(np.float32)))
              .astype(np.float64) for f in (-1, 1))
    assert ((got >= lo) & (got <= hi)).all()


def check(r_bits, w, eps, mode, out, q, scales, static=None):
    v, tol = step.norm_ref(r_bits, w, eps)
    if out is not None:
        f = quant.bf16_bits_to_f32(bits_of(out)).astype(np.float64)
        assert (np.abs(f - v) <= np.abs(v) * 2.0 ** -8 + 2 * tol).all()
    if mode == "tensor":
        check_quotients(q, v / static, tol / static)
    elif mode is not None:
        check_codes(q, scales, v, tol, 128 if mode == "block" else v.shape[1])


# T, H, mode, residual, bf16 output, extra columns of the rows
CASES = {
    "one_token": (1, 4096, "block", True, False, 0),
    "one_group": (3, 128, "block", True, True, 8),
    "odd_groups": (5, 128 * 3, "block", True, False, 0),
    "a_wave": (7, 512, "row", True, False, 0),
    "past_a_wave": (7, 640, "row", True, True, 16),
    "past_four_waves": (2, 2176, "block", False, True, 0),
    "wide": (9, 7168, "row", True, True, 32),
    "wider": (3, 16384, "block", True, False, 0),
    "wider_odd": (2, 8320, "tensor", True, True, 0),
    "widest": (2, 65536, "block", True, False, 0),
    "widest_row": (2, 65536 - 128, "row", True, False, 0),
    "static": (33, 1024, "tensor", True, False, 8),
    "no_codes": (17, 3968, None, True, True, 8),
    "no_residual": (4, 256, None, False, True, 0),
    "many": (1500, 1152, "block", True, True, 24),
    "many_wide": (1030, 4096, "row", False, False, 0),
}


@pytest.mark.parametrize("case", list(CASES))
def test_against_oracle(case):
    T, H, mode, res, both, extra = CASES[case]
    print(case, flush=True)
    rng = np.random.default_rng([T, H])
    x, r, w = normal(rng, T, H), normal(rng, T, H), normal(rng, H)
    r[:, rng.integers(0, H, 3)] = normal(rng, T, 3) + np.uint16(5 << 7)          # 32 times as large
    tx, tr, tw = wide(x, extra), wide(r, extra) if res else None, dev(w)
    out = wide(np.zeros_like(x), extra) if both else None
    ro = torch.empty((T, H), dtype=torch.bfloat16, device="cuda") if res else None
    if mode is None:
        fp8.add_rms_norm(tx, tw, residual=tr, eps=1e-5, out=out, residual_out=ro)
        q = scales = static = None
    else:
        static = np.float32(0.03) if mode == "tensor" else None
        q, scales = fp8.add_rms_norm_quant(
            tx, tw, residual=tr, eps=1e-5, scale_mode=mode, out=out, residual_out=ro,
            scale=None if static is None else torch.tensor([static], device="cuda"))
    torch.cuda.synchronize()
    total = step.add_ref(x, r) if res else x
    if res:
        assert np.array_equal(bits_of(ro), total) and np.array_equal(bits_of(tr), r)
    check(total, w, 1e-5, mode, out, q, scales, static)
    for t in (tx, tr, out):
        if t is not None and extra:                    # what lies between the rows
            behind = t.as_strided((T, extra), (H + extra, 1), t.storage_offset() + H)
            assert (behind == 9.0).all()


def test_in_place_and_into_rows_apart():
    rng = np.random.default_rng(5)
    T, H = 6, 384
    x, r, w = normal(rng, T, H), normal(rng, T, H), dev(normal(rng, H))
    q0, s0 = fp8.add_rms_norm_quant(dev(x), w, residual=(stream := dev(r)))
    assert np.array_equal(bits_of(stream), step.add_ref(x, r))
    q = torch.full((T, H + 16), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((T, 7), -1.0, device="cuda")
    q1, s1 = fp8.add_rms_norm_quant(dev(x), w, residual=dev(r), q=q[:, :H], scales=s[:, 2:5])
    assert torch.equal(q0, q[:, :H]) and torch.equal(s0, s[:, 2:5])
    assert (q[:, H:] == 0x55).all() and (s[:, :2] == -1).all() and (s[:, 5:] == -1).all()
    rows = torch.full((T, 2), -1.0, device="cuda")
    _, s2 = fp8.add_rms_norm_quant(dev(x), w, residual=dev(r), scale_mode="row", scales=rows[:, 0])
    assert (rows[:, 1] == -1).all() and (rows[:, 0] > 0).all()


def test_codes_feed_the_gemm():
    """The codes and scales are what block_gemm takes: the product of what they stand for."""
    rng = np.random.default_rng(6)
    x, r = normal(rng, 5, 512), normal(rng, 5, 512)
    wq, ws = fp8.quant_weight_block(dev(normal(rng, 256, 512)))
    q, s = fp8.add_rms_norm_quant(dev(x), dev(normal(rng, 512)), residual=dev(r))
    out = fp8.block_gemm(q, s, wq, ws).double().cpu()
    a = q.view(torch.float8_e4m3fn).cpu().double() * s.cpu().double().repeat_interleave(128, 1)
    b = wq.view(torch.float8_e4m3fn).cpu().double() * ws.cpu().double().repeat_interleave(
        128, 1).repeat_interleave(128, 0)
    want = a @ b.t()
    assert (out - want).norm() <= 2.0 ** -8 * want.norm()       # half a bf16 step each at most


def test_far_values():
    """Rows whose squares overflow or vanish in fp32, zero rows, no eps."""
    H, huge, tiny = 256, 2.0 ** 120, 2.0 ** -120
    rng = np.random.default_rng(7)
    base = rng.standard_normal((6, H)).astype(np.float32)
    x = synth.f32_to_bf16_bits(base * np.array([1, huge, tiny, 1e-20, 1e18, 0], np.float32)[:, None])
    w = normal(rng, H)
    for mode in ("block", "row"):
        for eps in (0.0, 1e-6):
            out = torch.empty((6, H), dtype=torch.bfloat16, device="cuda")
            q, s = fp8.add_rms_norm_quant(dev(x), dev(w), eps=eps, scale_mode=mode, out=out)
            n = 6 if eps else 5
            check(x[:n], w, np.float64(np.float32(eps)), mode, out[:n], q[:n], s[:n])
            if not eps:                                  # 0 / 0
                assert torch.isnan(out[5]).all()
            else:
                assert (out[5] == 0).all() and (s[5] == 0).all() and ((q[5] & 0x7f) == 0).all()


def test_groups_below_the_scales_resolution():
    """Maxima of 2^-149 .. 2^-124: amax / 448 has few bits or none, quotients pass 448 and saturate.

    The product of r and the reciprocal root is rounded to 2^-149 there, 2^-150 off at
    most, that with the weight 1 is exact; the scale is 2^-150 off at most.  2^-149
    bounds each with the float64 value's own tolerance."""
    rng = np.random.default_rng(9)
    T, H, quantum = 20, 384, 2.0 ** -149
    x = rng.standard_normal((T, H)) * 2.0 ** np.arange(-3, 17)[:, None]     # rms of 2^-3 .. 2^16
    x[:, 128:256] = rng.integers(-127, 128, (T, 128)) * 2.0 ** -133         # bf16 subnormals
    x = synth.f32_to_bf16_bits(x.astype(np.float32))
    for mode, ordinary in (("block", 1.0), ("row", 0.0)):
        w = np.full(H, ordinary, np.float32)
        w[128:256] = 1.0
        w = synth.f32_to_bf16_bits(w)
        q, s = fp8.add_rms_norm_quant(dev(x), dev(w), eps=1e-6, scale_mode=mode)
        v, tol = step.norm_ref(x, w, 1e-6)
        v, tol, q = v[:, 128:256], tol[:, 128:256] + quantum, q[:, 128:256]
        s = (s[:, 1] if mode == "block" else s).cpu().numpy().astype(np.float64)[:, None]
        g = np.abs(v).max(-1, keepdims=True) / 448
        assert (np.abs(s - g) <= quantum + g * 2.0 ** -16).all()
        assert (s == 0).any() and (g > 1.05 * s).any()        # the sizes meant: none, rounded far down
        assert ((q & 0x7f) != 0x7f).all()
        check_quotients(q, np.divide(v, s, out=v * 0, where=s > 0),
                        np.divide(tol, s, out=tol * 0, where=s > 0))


@pytest.mark.parametrize("mode", ["block", "row"])
def test_roots_beyond_the_types_range(mode):
    """Rows whose 1 / rms fp32 does not hold, without eps: one far value, subnormals only."""
    rng = np.random.default_rng(10)
    for H, values in ((65536, [2.0 ** -122]), (65536, [2.0 ** -133]), (65408, [3 * 2.0 ** -133]),
                      (1024, [-2.0 ** -133, 2.0 ** -126]), (128, [5 * 2.0 ** -133] * 128),
                      (256, rng.integers(-127, 128, 256) * 2.0 ** -133),
                      (4096, rng.standard_normal(4096) * 2.0 ** -127)):
        x = np.zeros((2, H), np.float32)
        x[0, rng.permutation(H)[:len(values)]] = values
        x[1] = -x[0]
        x, w = synth.f32_to_bf16_bits(x), normal(rng, H)
        for residual in (None, dev(x * 0)):
            out = torch.empty((2, H), dtype=torch.bfloat16, device="cuda")
            q, s = fp8.add_rms_norm_quant(dev(x), dev(w), residual=residual, eps=0.0, scale_mode=mode,
                                          out=out)
            check(x, w, 0.0, mode, out, q, s)


def test_nan_and_infinity_stay_in_their_rows():
    rng = np.random.default_rng(8)
    T, H = 8, 1024
    x, r, w = normal(rng, T, H), normal(rng, T, H), dev(normal(rng, H))
    out0, out1 = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q0, s0 = fp8.add_rms_norm_quant(dev(x), w, residual=dev(r), out=out0)
    x[2, 5], x[6, 900] = 0x7fc0, 0x7f80
    q1, s1 = fp8.add_rms_norm_quant(dev(x), w, residual=dev(r), out=out1)
    keep = [0, 1, 3, 4, 5, 7]
    assert torch.equal(q0[keep], q1[keep]) and torch.equal(s0[keep], s1[keep])
    assert torch.equal(out0[keep].view(torch.int16), out1[keep].view(torch.int16))
    assert torch.isnan(out1[2]).all() and torch.isnan(s1[2]).all()
    assert torch.isnan(out1[6, 900]) and (out1[6, :900] == 0).all() and torch.isnan(s1[6, 7])


def test_empty_and_refusals():
    x = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    q, s = fp8.add_rms_norm_quant(x, w, residual=x.clone())
    assert q.shape == (0, 256) and s.shape == (0, 2)
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, device="cuda")

    def go(x=x, w=w, **more):
        fp8.add_rms_norm_quant(x, w, **more)

    go()
    for bad, err in ((dict(x=x.float()), TypeError), (dict(x=x[:, :200]), ValueError),
                     (dict(x=x.t()), ValueError), (dict(w=w[:128]), ValueError),
                     (dict(residual=x[:3].clone()), ValueError), (dict(residual=x), ValueError),
                     (dict(residual_out=x.clone()), ValueError), (dict(scale=one), ValueError),
                     (dict(scale_mode="tensor"), ValueError), (dict(scale_mode=5), ValueError),
                     (dict(scale_mode="tensor", scale=one, scales=one), ValueError),
                     (dict(scales=torch.zeros((4, 1), device="cuda")), ValueError),
                     (dict(scale_mode="row", scales=torch.zeros((4, 1), device="cuda")), ValueError),
                     (dict(out=x), ValueError), (dict(out=x[:2].clone()), ValueError),
                     (dict(q=x.view(torch.uint8)), ValueError), (dict(eps=-1.0), ValueError),
                     (dict(w=w.cpu()), ValueError)):
        with pytest.raises(err):
            go(**bad)
