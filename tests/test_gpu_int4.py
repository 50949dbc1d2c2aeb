"""4-bit weights (needs a gfx950 GPU): packing and quantization bit for bit, the
product against the float64 definition with the tolerance of its fp32 sums and
half a bf16 step of the result."""

import numpy as np
import pytest
import torch

from oracle import quant, step
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


@pytest.mark.parametrize("N, K, extra", [(1, 128, 0), (5, 384, 0), (300, 1024, 24), (129, 14336, 0)])
def test_pack(N, K, extra):
    rng = np.random.default_rng([N, K])
    v = rng.integers(0, 256, (N, K + extra), dtype=np.uint8)
    got = fp8.int4_pack(torch.from_numpy(v).cuda()[:, :K])
    assert np.array_equal(got.cpu().numpy(), step.int4_pack_ref(v[:, :K] & 15))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [False, True])
def test_quant_weight(group, symmetric):
    rng = np.random.default_rng(group)
    w = normal(rng, 37, 640)
    w[3, :200] = 0
    w[4, :128] &= 0x7fff                                   # no negative value
    w[5, :128] |= 0x8000
    w[6, 0] = 0x0001                                       # a subnormal alone in its group
    w[6, 1:128] = 0
    w[7] = synth.f32_to_bf16_bits(np.float32(2.0 ** 100))
    wide = torch.zeros((37, 648), dtype=torch.bfloat16, device="cuda")
    wide[:, :640] = dev(w)
    codes, scales, zeros = fp8.int4_quant_weight(wide[:, :640], group, symmetric)
    c, s, z = step.int4_quant_ref(w, group, symmetric)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), step.int4_pack_ref(c))
    assert zeros is None if symmetric else np.array_equal(zeros.cpu().numpy(), z)


def weights(rng, N, K, group, zeros):
    c = rng.integers(0, 16, (N, K), dtype=np.uint8)
    s = (rng.random((N, K // group)) + 0.5).astype(np.float32) * np.float32(0.01)
    z = rng.integers(0, 16, s.shape, dtype=np.uint8) if zeros else None
    return c, s, z


def run(x, c, s, z, out=None):
    return fp8.int4_linear(x, torch.from_numpy(step.int4_pack_ref(c)).cuda(), torch.from_numpy(s).cuda(),
                           None if z is None else torch.from_numpy(z).cuda(), out=out)


def check(out, x_bits, c, s, z):
    want, tol = step.int4_linear_ref(x_bits, c, s, z)
    f = quant.bf16_bits_to_f32(bits_of(out)).astype(np.float64)
    off = np.abs(f - want) - (np.abs(want) * 2.0 ** -8 + tol * (1 + 2.0 ** -8))
    assert (off <= 0).all(), (off.max(), np.unravel_index(off.argmax(), off.shape))
    # each result at most half a bf16 step off, were the sums exact
    assert np.linalg.norm(f - want) <= 2.0 ** -8 * np.linalg.norm(want) * 1.125 + np.linalg.norm(tol) / 16


# M, N, K, group, zeros, extra columns of x, of out
CASES = {
    "one_token": (1, 256, 512, 128, False, 0, 0),
    "one_block": (1, 16, 128, 128, True, 0, 0),
    "one_column": (3, 1, 256, 64, True, 0, 0),
    "odd_columns": (2, 77, 384, 32, True, 8, 0),
    "many_blocks": (1, 48, 11008, 128, False, 0, 3),
    "two_rows": (2, 300, 1408, 64, False, 0, 0),
    "sixteen": (16, 128, 640, 32, False, 0, 0),
    "seventeen": (17, 130, 640, 128, True, 16, 5),
    "thirty_one": (31, 65, 256, 64, True, 0, 0),
    "thirty_three": (33, 129, 256, 128, False, 0, 0),
    "sixty_four": (64, 64, 1152, 32, True, 0, 0),
    "sixty_five": (65, 200, 512, 64, True, 0, 0),
    "prompt": (200, 333, 768, 128, True, 8, 1),
    "prompt_small_groups": (130, 256, 512, 32, False, 0, 0),
    "prompt_middle_groups": (257, 272, 1024, 64, False, 0, 0),
    "wide": (3, 20000, 128, 128, False, 0, 0),
    "wider": (5, 70001, 128, 64, True, 0, 0),
    "few_tall": (4, 40000, 256, 64, True, 0, 0),
    "some_columns": (9, 6500, 256, 64, True, 0, 0),
    "more_columns": (6, 9000, 256, 128, False, 0, 0),
    "runs_of_a_batch": (16, 2048, 16384, 128, True, 0, 0),
    "runs_odd_columns": (24, 515, 8192, 64, False, 8, 3),
    "runs_of_a_prompt": (100, 301, 4096, 32, True, 0, 0),
    "runs_even_columns": (70, 300, 4096, 128, False, 0, 0),
    "chunks_of_groups": (3, 20001, 40960, 32, True, 0, 0),
    "chunks_of_few_columns": (2, 100, 40960, 32, True, 0, 0),
    "chunks_of_eight_waves": (1, 64, 65536, 64, False, 0, 0),
    "a_batch_of_a_head": (13, 66001, 256, 64, True, 0, 0),
    "large_tiles": (700, 1601, 512, 128, True, 8, 3),
    "large_tiles_no_zeros": (650, 1700, 384, 128, False, 0, 0),
    "large_tiles_middle": (1030, 1030, 256, 64, True, 0, 0),
    "large_tiles_middle_no_zeros": (1030, 1030, 384, 64, False, 0, 0),
    "large_tiles_small": (520, 2100, 256, 32, True, 0, 0),
    "large_tiles_small_no_zeros": (520, 2100, 128, 32, False, 0, 0),
    "large_tiles_in_runs": (600, 1800, 2048, 128, True, 0, 0),
    "wider_batch": (20, 66000, 128, 32, True, 0, 0),
}


@pytest.mark.parametrize("case", list(CASES))
def test_against_oracle(case):
    M, N, K, group, zeros, ex, eo = CASES[case]
    print(case, flush=True)
    rng = np.random.default_rng([M, N, K])
    x = normal(rng, M, K)
    x[:, rng.integers(0, K, 2)] = normal(rng, M, 2) + np.uint16(4 << 7)
    c, s, z = weights(rng, N, K, group, zeros)
    wide = torch.full((M, K + ex), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = dev(x)
    out = torch.full((M, N + eo), 7.0, dtype=torch.bfloat16, device="cuda")
    run(wide[:, :K], c, s, z, out[:, :N])
    check(out[:, :N], x, c, s, z)
    assert (out[:, N:] == 7.0).all()


@pytest.mark.parametrize("M", [1, 13, 40, 150, 1000])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_each_value_finds_its_weight(M, group):
    """One value of x at a time: the codes come out exactly, so no value meets another's weight."""
    K, N = 256, 80 if M < 1000 else 1100
    rng = np.random.default_rng(M)
    c, s, z = weights(rng, N, K, group, True)
    s[:] = np.float32(0.25)
    for k0 in range(0, K, M):
        x = np.zeros((M, K), dtype=np.uint16)
        ks = np.arange(k0, min(K, k0 + M))
        x[np.arange(len(ks)), ks] = 0x3f80                        # 1.0
        out = run(dev(x), c, s, z).float().cpu().numpy()
        want = (c[:, ks].astype(int) - z[:, ks // group].astype(int)).T * 0.25
        assert np.array_equal(out[:len(ks)], want)
        if k0 > 64:
            break


# M, N, K: few rows, each tile, runs of K
FAR = [(1, 80, 512), (4, 37, 384), (13, 80, 512), (9, 5000, 256), (6, 9000, 256), (9, 66000, 128),
       (24, 515, 8192), (40, 130, 256), (100, 301, 4096), (700, 1601, 256)]


@pytest.mark.parametrize("M, N, K", FAR)
@pytest.mark.parametrize("group, zeros", [(32, True), (64, False), (128, True), (128, False)])
def test_values_near_the_types_end(M, N, K, group, zeros):
    """x (16 + code) or its sums leave fp32's range where the result does not: right all the same."""
    rng = np.random.default_rng([M, N, group])
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[::3] = np.clip(x[::3], -1.9, 1.9) * np.float32(2.0 ** 127)
    x[1::3, ::5] *= np.float32(2.0 ** 118)
    x = synth.f32_to_bf16_bits(x)
    c, s, z = weights(rng, N, K, group, zeros)
    s *= np.float32(2.0 ** -30)
    if zeros:
        z[::2] = rng.integers(0, 256, z[::2].shape)
    out = run(dev(x), c, s, z)
    want, tol = step.int4_linear_ref(x, c, s, z)
    f = quant.bf16_bits_to_f32(bits_of(out)).astype(np.float64)
    assert np.isfinite(f).all()
    assert (np.abs(f - want) <= np.abs(want) * 2.0 ** -8 + tol * (1 + 2.0 ** -8)).all()
    # a result beyond the type is an infinity with its sign, a row with a NaN or infinity is NaN
    s *= np.float32(2.0 ** 60)
    x[-1, K - 1] = 0x7f80
    f = quant.bf16_bits_to_f32(bits_of(run(dev(x), c, s, z))).astype(np.float64)
    want, tol = (a[:-1] * 2.0 ** 60 for a in (want, tol))
    far = np.abs(want) > 2.0 ** 129 + 2 * tol
    assert np.array_equal(f[:-1][far], np.sign(want[far]) * np.inf) and np.isnan(f[-1]).all()
    near = np.abs(want) < 2.0 ** 127 - 2 * tol
    assert (np.abs(f[:-1] - want)[near] <= (np.abs(want) * 2.0 ** -8 + tol * (1 + 2.0 ** -8))[near]).all()


@pytest.mark.parametrize("M", [1, 4, 13, 40, 150, 1000])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_each_place_finds_its_weight(M, group):
    """Each place of two blocks of 128 values, as many of them a call as there are rows."""
    K, N = 256, 80 if M < 1000 else 1100
    rng = np.random.default_rng(M)
    c, s, z = weights(rng, N, K, group, True)
    s[:] = np.float32(0.25)
    d = [torch.from_numpy(a).cuda() for a in (step.int4_pack_ref(c), s, z)]
    want = (c.astype(int) - np.repeat(z, group, 1).astype(int)).T * 0.25
    for k0 in range(0, K, M):
        x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
        ks = torch.arange(k0, min(K, k0 + M), device="cuda")
        x[torch.arange(len(ks), device="cuda"), ks] = 1.0
        out = fp8.int4_linear(x, *d)[:len(ks)].float().cpu().numpy()
        assert np.array_equal(out, want[k0:k0 + M]), k0


@pytest.mark.parametrize("M, N, K", FAR)
@pytest.mark.parametrize("group, zeros", [(32, False), (64, True), (128, True)])
def test_subnormal_values(M, N, K, group, zeros):
    """Subnormal values of x keep their part in both of the sums."""
    rng = np.random.default_rng([M, N, group, 1])
    x = rng.integers(0, 128, (M, K)).astype(np.uint16)
    x |= (rng.integers(0, 2, (M, K)) << 15).astype(np.uint16)
    c, s, z = weights(rng, N, K, group, zeros)
    s *= np.float32(2.0 ** 100)
    check(run(dev(x), c, s, z), x, c, s, z)


@pytest.mark.parametrize("M, N, K", [(24, 515, 8192), (100, 300, 4096)])
def test_workspaces(M, N, K):
    """A call without the workspace, or with a part of it, does not cut K."""
    rng = np.random.default_rng([M, N])
    c, s, z = weights(rng, N, K, 64, True)
    x = normal(rng, M, K)
    d = [dev(x), torch.from_numpy(step.int4_pack_ref(c)).cuda(), torch.from_numpy(s).cuda(),
         torch.from_numpy(z).cuda()]
    n = fp8.int4_workspace_bytes(M, N, K)
    assert n > 0 and fp8.int4_workspace_bytes(1, N, K) == 0
    store = torch.full((n + 32,), 0x55, dtype=torch.uint8, device="cuda")
    for size in (n, n - 16, 0):
        ws = store[16:16 + size]
        check(fp8.int4_linear(*d, workspace=ws), x, c, s, z)
        assert (store[:16] == 0x55).all() and (store[16 + size:] == 0x55).all()
        store.fill_(0x55)
    with pytest.raises(ValueError):
        fp8.int4_linear(*d, workspace=store[1:])                   # not aligned


def test_rows_of_one_sign():
    """The offset's part of the sums is largest where x has one sign: still within tolerance."""
    rng = np.random.default_rng(12)
    x = normal(rng, 9, 4096) & np.uint16(0x7fff)
    c, s, z = weights(rng, 64, 4096, 128, True)
    check(run(dev(x), c, s, z), x, c, s, z)


def test_rows_do_not_depend_on_their_neighbours():
    """A NaN or infinity stays in its row; far zero points and negative scales are taken as they are."""
    rng = np.random.default_rng(13)
    for M in (16, 70, 140):
        x = normal(rng, M, 256)
        c, s, z = weights(rng, 96, 256, 64, True)
        z[3], s[4] = 200, -s[4]
        a = run(dev(x), c, s, z)
        check(a, x, c, s, z)
        x[5, 17], x[8, 200] = 0x7fc0, 0xff80
        b = run(dev(x), c, s, z)
        keep = [m for m in range(M) if m not in (5, 8)]
        assert torch.equal(a[keep].view(torch.int16), b[keep].view(torch.int16))
        assert torch.isnan(b[[5, 8]]).all()


def test_repeats_are_equal_and_empty_calls():
    rng = np.random.default_rng(14)
    c, s, z = weights(rng, 500, 2048, 128, True)
    x = dev(normal(rng, 90, 2048))
    first = run(x, c, s, z)
    for _ in range(3):
        assert torch.equal(first, run(x, c, s, z))
    assert run(x[:0], c, s, z).shape == (0, 500)


def test_refusals():
    rng = np.random.default_rng(15)
    c, s, z = weights(rng, 32, 256, 64, True)
    x, codes = dev(normal(rng, 4, 256)), torch.from_numpy(step.int4_pack_ref(c)).cuda()
    s, z = torch.from_numpy(s).cuda(), torch.from_numpy(z).cuda()

    def go(x=x, codes=codes, s=s, z=z, out=None):
        fp8.int4_linear(x, codes, s, z, out=out)

    go()
    for bad, err in ((dict(x=x.float()), TypeError), (dict(x=x[:, :128]), ValueError),
                     (dict(codes=codes[:, :64]), ValueError), (dict(codes=codes[:16]), ValueError),
                     (dict(s=s[:, :3].contiguous()), ValueError), (dict(s=s.double()), TypeError),
                     (dict(s=s[:, :1].contiguous(), z=None), ValueError),       # groups of 256
                     (dict(z=z[:, :2].contiguous()), ValueError), (dict(z=z.int()), TypeError),
                     (dict(out=x), ValueError), (dict(codes=codes.cpu()), ValueError),
                     (dict(x=x[:, 1:129], codes=codes[:, :64].contiguous()), ValueError)):
        with pytest.raises(err):
            go(**bad)
    w = dev(normal(rng, 4, 256))
    for bad in (dict(w=w, group=16), dict(w=w, group=0), dict(w=w[:, :192], group=64)):
        with pytest.raises(ValueError):
            fp8.int4_quant_weight(**bad)
    with pytest.raises(TypeError):
        fp8.int4_quant_weight(w.float())
    with pytest.raises(ValueError):
        fp8.int4_pack(torch.zeros((4, 100), dtype=torch.uint8, device="cuda"))
