"""The reader of tensor arguments refuses what is not a GPU tensor of the wanted
form by giving None (the binding's checks then say why), and what is no call at
all by a TypeError."""

import numpy as np
import pytest
import torch

import fp8_w8a8_block_amd as fp8
from fp8_w8a8_block_amd import _attention

fp8.lib()
GPU = torch.device("cuda", 0)                      # a name; no GPU is needed here


def args():
    return _attention._tensor_args


@pytest.mark.parametrize("device", [torch.device("cpu"), GPU])
def test_host_tensors_and_other_objects_give_none(device):
    i = torch.zeros(4, dtype=torch.int32)
    c = torch.zeros((2, 4, 1, 16), dtype=torch.uint8)
    for t in (i, None, 3, "x", np.zeros(4, dtype=np.int32)):
        assert args().vector(t, torch.int32, device, 4) is None
        assert args().heads(t, device) is None
        assert args().table(t, device, 4) is None
        assert args().matrix(t, torch.int32, device) is None
        assert args().caches(t, c, device) is None
        assert args().caches(c, t, device) is None
    assert args().vector(i, torch.int32, None, 4) is None


@pytest.mark.parametrize("call", [
    lambda a: a.vector(), lambda a: a.vector(1, 2, 3, 4), lambda a: a.heads(1),
    lambda a: a.table(1, 2), lambda a: a.matrix(1, 2, 3), lambda a: a.caches(1, 2),
    lambda a: a.vector(None, torch.int32, GPU, "n"), lambda a: a.table(None, GPU, "n"),
])
def test_no_call_at_all(call):
    with pytest.raises(TypeError):
        call(args())


def test_calls_say_what_is_wrong():
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="query must be a device tensor"):
        fp8.paged_attention(x, *[None] * 7)
    with pytest.raises(TypeError, match="computed_lens must be a tensor"):
        fp8.kv_slot_map([1], None, None, None, 16, 1)
