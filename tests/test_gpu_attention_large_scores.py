"""Scores so large that fp32 holds no fraction of them, in both attention kernels
(needs a gfx950 GPU).

A row's softmax is then 1 at its largest score, wherever that leads the others by
more than the products' rounding, and 0 elsewhere: the result is that key's value,
the log-sum-exp its score."""

import numpy as np
import pytest
import torch

from oracle import attention, e4m3, quant
from workloads import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_w8a8_block_amd as fp8


@pytest.mark.parametrize("power", [16, 18, 20, 24, 27, 31, 60, 100])
@pytest.mark.parametrize("D,requests", [(64, [(1, 300), (1, 700), (2, 40)]), (64, [(150, 400)]),
                                        (128, [(1, 300), (1, 2000)]), (128, [(150, 400), (60, 60)]),
                                        (256, [(1, 300), (20, 90)])])
@pytest.mark.parametrize("below", [False, True])
def test_one_key_wins(power, D, requests, below):
    rng = np.random.default_rng([power, D, len(requests)])
    Hq, Hk, page, ks, vs = 4, 2, 16, 0.5, 0.25
    scale = 0.75 if not below else -0.75
    new, lens = [n for n, _ in requests], [l for _, l in requests]
    T, offsets = sum(new), np.cumsum([0] + new)
    blocks = [-(-l // page) for l in lens]
    kc, vc = (rng.integers(0x20, 0x58, (sum(blocks), page, Hk, D), dtype=np.uint8)
              for _ in range(2))
    vc |= rng.integers(0, 2, vc.shape, dtype=np.uint8) << 7
    q = rng.standard_normal((T, Hq, D))
    if below:                                      # positive products, a negative scale:
        q = np.abs(q)                              # every score lies far below 0
    else:
        kc |= rng.integers(0, 2, kc.shape, dtype=np.uint8) << 7
    q_bits = synth.f32_to_bf16_bits((q * 2.0 ** power).astype(np.float32))
    table = np.full((len(lens), max(blocks)), -1, dtype=np.int32)
    first = np.cumsum([0] + blocks)
    for r, n in enumerate(blocks):
        table[r, :n] = np.arange(first[r], first[r] + n)

    def dev(x, dtype):
        return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")

    lse = torch.empty((T, Hq), device="cuda")
    out = fp8.paged_attention(
        torch.from_numpy(q_bits.view(np.int16)).cuda().view(torch.bfloat16),
        torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), dev(table, torch.int32),
        dev(lens, torch.int32), dev(offsets, torch.int32), dev([ks], torch.float32),
        dev([vs], torch.float32), scale=scale, lse=lse).double().cpu().numpy()
    lse = lse.double().cpu().numpy()

    q = quant.bf16_bits_to_f32(q_bits).astype(np.float64)
    kd, vd = (e4m3.decode(c).astype(np.float64).reshape(-1, Hk, D) for c in (kc, vc))
    clear = 0
    for r in range(len(lens)):
        slots = attention.key_slots(table[r], lens[r], page, len(kc))
        for i in range(new[r]):
            seen = slots[:lens[r] - new[r] + i + 1]
            for h in range(Hq):
                x, k = q[offsets[r] + i, h], kd[seen, h // 2]
                s = k @ x * (scale * ks)
                # D exact products summed in fp32, the factor's rounding and its product's
                err = (D + 4) * 2.0 ** -24 * (np.abs(k) @ np.abs(x)).max() * abs(scale * ks)
                best = int(s.argmax())
                assert abs(lse[offsets[r] + i, h] - s[best]) <= err + np.log(len(s)) + 2, (r, i, h)
                if len(s) > 1 and s[best] - np.delete(s, best).max() < 2 * err + 60:
                    assert np.isfinite(out[offsets[r] + i, h]).all(), (r, i, h)
                    continue
                clear += 1
                # P in fp16 (2^-11), the result in bf16 (half a step, 2^-8): P's is
                # below half a step of a value of 4 bits, which comes out exact
                assert np.array_equal(out[offsets[r] + i, h], vd[seen[best], h // 2] * vs), (r, i, h)
    assert clear > 0.75 * T * Hq


@pytest.mark.parametrize("n", [1, 60])                 # tokens per request: either kernel
@pytest.mark.parametrize("power", [22, 29, 90])
def test_one_key_wins_behind_a_prefix(n, power):
    """Head 0's largest score is in the shared prefix, head 1's among a request's own keys."""
    rng = np.random.default_rng([n, power])
    B, D, page, far, own = 5, 64, 16, 333, 77
    shared, mine = -(-far // page), -(-own // page)
    kc = np.zeros((shared + mine, page, 2, D), dtype=np.uint8)
    kc[..., 0] = 0x38                                  # 1, but 16 at the two that win
    vc = rng.integers(0x20, 0x58, kc.shape, dtype=np.uint8)
    kc[200 // page, 200 % page, 0, 0] = kc[shared, 5, 1, 0] = 0x58
    q = torch.zeros((B * n, 2, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0 ** power

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    lse = torch.empty((B * n, 2), device="cuda")
    out = fp8.prefix_attention(
        q, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), i32(list(range(shared))),
        i32([far]), i32([list(range(shared, shared + mine))] * B), i32([own] * B),
        i32(list(range(0, B * n + 1, n))), torch.ones(1, device="cuda"),
        torch.ones(1, device="cuda"), scale=0.3, lse=lse).float().cpu()
    for h, at in ((0, (200 // page, 200 % page, 0)), (1, (shared, 5, 1))):
        want = torch.from_numpy(e4m3.decode(vc[at]).astype(np.float32))
        assert torch.equal(out[:, h], want.expand(B * n, D)), h
    top = float(np.float32(0.3)) * 16 * 2.0 ** power
    assert torch.allclose(lse.cpu().double(), torch.tensor(top, dtype=torch.float64), rtol=2.0 ** -21)
