"""What the reader of tensor arguments returns for GPU tensors (needs a gfx950 GPU)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp8_w8a8_block_amd import _tensor_args as args


def test_pointers_and_shapes():
    dev = torch.device("cuda", torch.cuda.current_device())
    i = torch.zeros(12, dtype=torch.int32, device=dev)
    assert args.vector(i, torch.int32, dev, 12) == i.data_ptr() == args.vector(i, torch.int32, dev, -1)
    for bad in (args.vector(i, torch.int32, dev, 11), args.vector(i, torch.int64, dev, 12),
                args.vector(i[::2], torch.int32, dev, 6), args.vector(i.view(3, 4), torch.int32, dev, 12),
                args.vector(i, torch.int32, torch.device("cuda", dev.index + 1), 12),
                args.vector(i, torch.int32, torch.device("cpu"), 12)):
        assert bad is None
    assert args.vector(i[:0], torch.int32, dev, 0) == i[:0].data_ptr()
    m = i.view(3, 4)
    assert args.matrix(m, torch.int32, dev) == (m.data_ptr(), 3, 4)
    assert args.matrix(m[:, :2], torch.int32, dev) is None
    assert args.table(m, dev, 3) == (m.data_ptr(), 4, 4)
    assert args.table(m[:, 1:3], dev, 3) == (m[:, 1:].data_ptr(), 4, 2)
    assert args.table(m[:1, :2], dev, 1) == (m.data_ptr(), 2, 2)
    assert args.table(m, dev, 2) is None and args.table(m.t(), dev, 4) is None
    x = torch.zeros((5, 6, 8), dtype=torch.bfloat16, device=dev)
    assert args.heads(x, dev) == (x.data_ptr(), 5, 6, 8, 48)
    assert args.heads(x[:, 2:4], dev) == (x[:, 2:].data_ptr(), 5, 2, 8, 48)
    assert args.heads(x[:1, :3], dev) == (x.data_ptr(), 1, 3, 8, 24)
    for bad in (x[:, ::2], x[..., :4], x[:0], x[0], x.half()):
        assert args.heads(bad, dev) is None
    k = torch.zeros((3, 4, 2, 16), dtype=torch.uint8, device=dev)
    v = torch.zeros_like(k)
    assert args.caches(k, v, dev) == (k.data_ptr(), v.data_ptr(), 3, 4, 2, 16)
    for a, b in ((k, v[:2]), (k[..., :8], v[..., :8]), (k[0], v[0]), (k, v.int())):
        assert args.caches(a, b, dev) is None
