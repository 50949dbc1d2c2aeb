"""Softmax weights far below a row's largest one, in both attention kernels
(needs a gfx950 GPU).

One key that every query sees scores `nats` above all the others and its values
are zeros, so that a result is what the others' small weights leave.  Requests
share one table row, and there are as many as workgroups (a multiple of them for
the 16-row kernel), so that no share cuts an item and one base serves all of its
keys."""

import numpy as np
import pytest
import torch

from oracle import attention

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_w8a8_block_amd as fp8

D, PAGE = 64, 64
ZERO, ONE, TOP = 0x00, 0x38, 0x58                      # codes of 0, 1 and 16


def caches(keys, top_at):
    """Keys 0 and values 1 (their sign by value), but key top_at: 16 and 0."""
    blocks = -(-keys // PAGE)
    kc = np.zeros((blocks, PAGE, 1, D), dtype=np.uint8)
    vc = np.full((blocks, PAGE, 1, D), ONE, dtype=np.uint8)
    vc[..., 1::2] |= 0x80
    kc[top_at // PAGE, top_at % PAGE, 0, 0] = TOP
    vc[top_at // PAGE, top_at % PAGE] = ZERO
    return kc, vc


@pytest.mark.parametrize("n", [1, 64])                 # the 16-row kernel, the 256-row one
@pytest.mark.parametrize("keys,top_at", [(65536, 0), (131071, 3), (131071, 70000)])
def test_small_weights_count(n, keys, top_at):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    B = 2 * cus if n == 1 else cus
    nats = [15.0, 16.0, 17.0, 17.25, 17.5, 20.0]
    kc, vc = caches(keys, top_at)
    few = np.zeros((len(nats) * n, 1, D))
    few[:, 0, 0] = np.repeat(nats, n) / 8              # 16 ks q = nats, exact in bf16
    of = np.arange(B) % len(nats)
    q = few.reshape(len(nats), n, 1, D)[of].reshape(B * n, 1, D)
    lse = torch.empty((B * n, 1), device="cuda")
    out = fp8.paged_attention(
        torch.tensor(q, dtype=torch.bfloat16, device="cuda"), torch.from_numpy(kc).cuda(),
        torch.from_numpy(vc).cuda(),
        torch.arange(len(kc), dtype=torch.int32, device="cuda").expand(B, -1).contiguous(),
        torch.full((B,), keys, dtype=torch.int32, device="cuda"),
        torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda"),
        torch.full((1,), 0.5, device="cuda"), torch.ones(1, device="cuda"), scale=1.0, lse=lse)
    ref, ref_lse, tol, tol_lse, _ = attention.attention_ref(
        few, kc, vc, np.arange(len(kc))[None].repeat(len(nats), 0), [keys] * len(nats),
        np.arange(len(nats) + 1) * n, 1.0, 0.5, 1.0)
    out = out.double().cpu().numpy().reshape(B, n, D)
    lse = lse.double().cpu().numpy().reshape(B, n)
    ref, tol = ref.reshape(-1, n, D)[of], tol.reshape(-1, n, D)[of]
    off = np.abs(out - ref) - tol
    assert (off <= 0).all(), [(nats[i], float(out[i, 0, 0]), float(ref[i, 0, 0]))
                              for i in range(len(nats))]
    assert (np.abs(lse - ref_lse.reshape(-1, n)[of]) <= tol_lse.reshape(-1, n)[of]).all()
