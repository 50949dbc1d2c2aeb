"""fp8_kv_slot_map against the oracle (needs a gfx950 GPU): every output and
the whole table, exactly, over batches of one to thousands of requests."""

import numpy as np
import pytest
import torch

from oracle import attention

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_w8a8_block_amd as fp8


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def check(computed, new, page, width, free, T, ld=None, seed=0):
    rng = np.random.default_rng(seed)
    B = len(computed)
    table = np.full((B, width), -1, dtype=np.int32)
    for r in range(B):
        have = min(width, -(-max(0, int(computed[r])) // page))
        table[r, :have] = rng.integers(0, 1 << 20, have)
    wide = i32(np.full((B, ld or width), 77))
    wide[:, :width] = i32(table)
    got = fp8.kv_slot_map(i32(computed), i32(new), wide[:, :width], i32(free), page, T)
    slots, pos, offs, lens, taken = (x.cpu().numpy() for x in got)
    want = attention.slot_map_ref(computed, new, table, free, page, T)
    assert np.array_equal(wide[:, :width].cpu().numpy(), want[0])
    assert (wide[:, width:].cpu().numpy() == 77).all()
    assert np.array_equal(pos, want[2])
    assert np.array_equal(slots, want[1])
    assert np.array_equal(offs, want[3]) and np.array_equal(lens, want[4])
    assert taken[0] == want[5]


@pytest.mark.parametrize("B", [1, 2, 255, 257, 1023, 1025, 2500])
@pytest.mark.parametrize("page", [1, 7, 16])
def test_decode_steps(B, page):
    rng = np.random.default_rng([B, page])
    computed = rng.integers(0, 300, B)
    new = (rng.random(B) < 0.9).astype(int)
    check(computed, new, page, 320 // page + 2, rng.permutation(4000)[:B], int(new.sum()) + 3)


@pytest.mark.parametrize("lens", [[1], [511], [512], [513], [0, 0, 1024, 0, 1], [5000, 3, 0, 2000],
                                  [1] * 40 + [700] * 5])
@pytest.mark.parametrize("page", [16, 5])
def test_prefill(lens, page):
    rng = np.random.default_rng([len(lens), page])
    computed = rng.integers(0, 50, len(lens))
    T = sum(lens)
    check(computed, lens, page, 6000 // page, rng.permutation(9000), T, ld=6000 // page + 3)
    check(computed, lens, page, 6000 // page, rng.permutation(9000), T + 700)     # padded
    check(computed, lens, page, 6000 // page, rng.permutation(9000), max(1, T // 2))  # cut short


def test_edges():
    check([], [], 16, 4, [1, 2], 5)                        # no request
    check([0, 0], [0, 0], 16, 4, [1, 2], 0)                # no token
    check([-5, 3], [2, -1], 4, 3, [8], 4)                  # negative lengths are none
    check([10, 0], [30, 9], 4, 4, [8, 9, 1, 2, 3, 4, 5, 6, 7, 11, 12, 13], 39)   # table too narrow
    check([0, 7], [9, 9], 4, 8, [3], 18)                   # free list too short
    check([0, 7], [9, 9], 4, 8, [], 18)
    check([4, 8], [1, 1], 1 << 20, 1, [5], 2)              # one huge page


def test_unmapped_pages_and_huge_lengths():
    table = i32([[3, -1, 9]])
    got = fp8.kv_slot_map(i32([6]), i32([1]), table, i32([]), 4, 1)
    assert got[0].tolist() == [-1] and got[1].tolist() == [6]
    big = (1 << 31) - 1
    table = i32(np.full((2, 1), -1))
    got = fp8.kv_slot_map(i32([big, big]), i32([big, 5]), table, i32([0]), 1 << 20, 4)
    assert got[3].tolist() == [big, big]                   # saturated
    assert got[2].tolist() == [0, big, big]
    assert got[1].tolist() == [big + i for i in range(4)]
    assert got[0].tolist() == [-1] * 4


def test_lengths_that_no_table_holds():
    """Blocks behind a row's end are counted, not walked: 2^31 of them in each of 300 rows."""
    big, B, width = (1 << 31) - 1, 300, 4
    free = np.arange(50, 60)
    table = i32(np.full((B, width), 7))
    got = fp8.kv_slot_map(i32([1] * B), i32([2] + [big] * (B - 1)), table, i32(free), 1, 6)
    want = np.full((B, width), 7)                          # entry 0 was there
    want[0, 1:3] = free[:2]
    want[1, 1:] = free[2:5]
    want[2:, 1:] = -1                                      # the list ended in the row before
    assert np.array_equal(table.cpu().numpy(), want)
    assert got[0].tolist() == [50, 51, 52, 53, 54, -1] and got[1].tolist() == [1, 2, 1, 2, 3, 4]
    assert int(got[4]) == big


def test_refusals():
    x, t = i32([1, 2]), i32([[0], [0]])
    with pytest.raises(TypeError):
        fp8.kv_slot_map(x.long(), x, t, x, 16, 2)
    with pytest.raises(ValueError):
        fp8.kv_slot_map(x, x[:1], t, x, 16, 2)
    with pytest.raises(ValueError):
        fp8.kv_slot_map(x, x, t[:1], x, 16, 2)
    with pytest.raises(ValueError, match="shape"):
        fp8.kv_slot_map(x, x, t, x, 0, 2)
    with pytest.raises(ValueError):
        fp8.kv_slot_map(x, x, t, x, 16, -1)
    with pytest.raises(ValueError, match="overlaps"):
        fp8.kv_slot_map(x, x, t, x, 16, 2, seq_lens=x)
