"""fp8_token_logprobs against the float64 definition (needs a gfx950 GPU): whole
numbers equal, the rest within the tolerance of fp32 sums."""

import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_w8a8_block_amd as fp8

NAMES = ("logprobs", "ranks", "entropy", "lse", "top", "ids")


def logits(rng, T, V, bf16, ld=None, offset=0):
    """Device logits [T, V] in rows of ld, starting `offset` values into their storage."""
    ld = V if ld is None else ld
    store = torch.full((offset + T * ld,), 1e30, dtype=torch.bfloat16 if bf16 else torch.float32,
                       device="cuda")
    x = store.as_strided((T, V), (ld, 1), offset)
    x.copy_(torch.from_numpy((rng.standard_normal((T, V)) * 3).astype(np.float32)))
    return x


def check(x, tokens, k, scale=1.0, **buffers):
    got = fp8.token_logprobs(x, torch.as_tensor(tokens, device="cuda"), k=k, scale=scale, **buffers)
    torch.cuda.synchronize()
    got = {n: v.cpu().numpy() for n, v in zip(NAMES, got)}
    want, tol = step.logprobs_ref(x.float().cpu().numpy().astype(np.float64), np.asarray(tokens), k,
                                  float(np.float32(scale)))
    assert np.array_equal(got["ranks"], want["ranks"])
    assert np.array_equal(got["ids"], want["ids"])
    for n in ("logprobs", "entropy", "lse", "top"):
        g, w = got[n].astype(np.float64), want[n]
        # fp32 holds nothing beyond 2^128 - 2^104: from half a step above it on, 2^103, a
        # value's nearest is infinity (two logits can be 2^129 apart)
        with np.errstate(invalid="ignore"):
            w = np.where(np.abs(w) >= 2.0 ** 128 - 2.0 ** 103, np.sign(w) * np.inf, w)
        assert np.array_equal(np.isnan(g), np.isnan(w)) and np.array_equal(np.isneginf(g), np.isneginf(w)), n
        ok = np.isfinite(w)
        off = np.where(ok, np.abs(np.where(ok, g, 0) - np.where(ok, w, 0)) - tol(w), 0)
        assert (off <= 0).all(), (n, off.max())
    return got


# T, V, k, bf16, row stride beyond V, first value
CASES = {
    "one_token": (1, 128000, 20, True, 0, 0),
    "one_token_f32": (1, 100003, 64, False, 0, 0),
    "one_logit": (3, 1, 1, True, 0, 0),
    "few_logits": (5, 7, 7, False, 1, 3),
    "below_a_segment": (4, 63, 5, True, 0, 1),
    "a_segment": (4, 64, 64, True, 0, 0),
    "past_a_segment": (4, 65, 3, True, 0, 7),
    "a_sweep": (3, 4096, 20, True, 0, 0),
    "past_a_sweep": (3, 4097, 20, True, 0, 5),
    "a_batch": (3, 16384, 2, True, 0, 0),
    "past_a_batch_f32": (3, 8193, 33, False, 2, 1),
    "no_alternatives": (9, 5000, 0, True, 0, 0),
    "odd_rows": (61, 32001, 5, True, 0, 0),
    "odd_rows_f32": (37, 20011, 5, False, 0, 2),
    "apart": (11, 30000, 8, True, 13, 9),
    "a_workgroup_each": (1100, 2001, 20, True, 0, 0),
    "a_workgroup_each_f32": (1030, 3333, 7, False, 0, 0),
    "long_rows_each": (1024, 24000, 1, True, 0, 0),
    "many_segments": (2, 600000, 64, False, 0, 0),
    "many_segments_of_many_rows": (260, 300001, 3, True, 0, 0),
    "sixteen_sweeps": (5, 65000, 40, True, 2, 0),
    "past_sixteen_sweeps": (5, 65601, 40, True, 3, 5),
    "parts": (37, 70001, 20, False, 0, 2),
    "parts_of_batches": (130, 120001, 33, False, 0, 0),
    "parts_of_batches_bf16": (140, 140000, 5, True, 1, 0),
    "a_workgroup_for_each_unit": (256, 70000, 5, True, 0, 3),
}


@pytest.mark.parametrize("case", list(CASES))
def test_against_oracle(case):
    T, V, k, bf16, more, offset = CASES[case]
    print(case, flush=True)
    rng = np.random.default_rng([T, V])
    x = logits(rng, T, V, bf16, V + more, offset)
    tokens = rng.integers(0, V, T)
    if T > 2:
        tokens[:3] = [0, V - 1, -1]
    if T > 4:
        tokens[4] = V
    check(x, tokens, k, scale=0.7)


@pytest.mark.parametrize("T, V", [(3, 9000), (1030, 9000), (3, 80000)])
@pytest.mark.parametrize("bf16", [True, False])
def test_equal_logits(T, V, bf16):
    """Rows of one value, of few values, and with the ties at the end: the lowest indexes first."""
    rng = np.random.default_rng(2)
    x = logits(rng, T, V, bf16)
    x[0] = 1.5
    x[1] = torch.from_numpy(rng.integers(0, 3, V).astype(np.float32)).cuda()
    x[2] = -2.0
    x[2, -30:] = 4.0
    x[2, 100:110] = 5.0
    x[-1, ::2] = 0.0
    x[-1, 1::2] = -0.0                                          # equal to 0
    tokens = rng.integers(0, V, T)
    for k in (1, 20, 64):
        check(x, tokens, k)


@pytest.mark.parametrize("T, V", [(4, 10007), (1030, 10007), (4, 80007)])
@pytest.mark.parametrize("bf16", [True, False])
def test_masks(T, V, bf16):
    """Masked rows: a few logits left, fewer than k, one, none; masks of the lowest value."""
    rng = np.random.default_rng(3)
    x = logits(rng, T, V, bf16)
    low = torch.finfo(x.dtype).min
    x[0] = -torch.inf
    keep = rng.permutation(V)[:40]
    x[1, [i for i in range(V) if i not in set(keep)]] = -torch.inf
    x[2] = -torch.inf
    x[2, 777] = -3.0
    x[3, 5000:] = low
    x[-1] = low
    tokens = rng.integers(0, V, T)
    tokens[:4] = [5, keep[0], 777, 6000]
    for k in (1, 64):
        check(x, tokens, k, scale=0.5)


def test_mask_of_the_lowest_value_everywhere_at_scale_one():
    x = torch.full((2, 5000), torch.finfo(torch.float32).min, device="cuda")
    x[1, 3] = 2.0
    check(x, [1, 3], 4)


@pytest.mark.parametrize("T, V", [(5, 9001), (1030, 9001), (5, 80001)])
def test_no_distribution(T, V):
    """NaN and +inf make their row NaN and -1, wherever they stand, and no other row."""
    rng = np.random.default_rng(4)
    x = logits(rng, T, V, False)
    x[0, 0], x[1, V - 1], x[2, 4500] = torch.nan, torch.nan, torch.inf
    x[3] = torch.nan
    x[4] = -torch.inf
    x[4, 5] = torch.nan
    x[0, 1] = 1e30                                              # the NaN's thread is far below
    got = check(x, rng.integers(0, V, T), 6)
    assert (got["ids"][:5] == -1).all() and (got["ids"][5:] >= 0).all()


@pytest.mark.parametrize("T, V", [(4, 5000), (300, 5000), (4, 80000)])
@pytest.mark.parametrize("bf16", [True, False])
def test_the_types_ends(T, V, bf16):
    """Differences beyond the type's largest value: weights of 0, and no NaN."""
    x = logits(np.random.default_rng(8), T, V, bf16)
    low = torch.finfo(x.dtype).min
    x[0] = low
    x[0, 77] = -low
    x[1, ::3], x[1, 5], x[1, V - 1] = low, -low, -low
    x[2, :V // 2], x[2, V // 2:] = -torch.inf, low
    x[3] = -low
    tokens = np.zeros(T, dtype=np.int64)
    tokens[:4] = [77, 5, V - 1, 9]
    check(x, tokens, 9)


def test_far_logits():
    """Large logits keep their differences; the scale is applied once."""
    rng = np.random.default_rng(5)
    x = logits(rng, 3, 20000, False)
    x[0] += 30000.0
    x[1] *= 1e4
    x[2] *= 1e-20
    for scale in (1.0, 0.01, 30.0):
        check(x, [7, 8, 9], 10, scale=scale)


FAR_SCALES = (float(torch.finfo(torch.float32).max), 2.5e38, 2.0 ** 126)


@pytest.mark.parametrize("T, V", [(5, 7001), (300, 7001), (5, 90001)])
@pytest.mark.parametrize("bf16", [True, False])
def test_largest_scales(T, V, bf16):
    """Scales up to the type's largest (a temperature of 0, cut there): the largest logits
    share the probability, and logits that small have a distribution of their own."""
    x = logits(np.random.default_rng(9), T, V, bf16)
    store = x.clone()
    tokens = np.zeros(T, dtype=np.int64)
    for scale in FAR_SCALES:
        x.copy_(store)
        x[1, 5], x[1, V - 2] = 40.0, 40.0                      # two equal maxima
        x[2] = 3.0
        x[3, 7:] = -torch.inf
        x[-1] = 0.0
        tokens[:5] = [int(x[0].float().argmax()), 5, 9, 8, V - 1]
        got = check(x, tokens, 5, scale=scale)
        assert (got["logprobs"][0] == 0) == ((x[0] == x[0].max()).sum().item() == 1)
        x.copy_(store * (1.0 / scale))                         # subnormal values
        check(x, tokens, 5, scale=scale)


@pytest.mark.parametrize("T, V", [(4, 5000), (300, 5000), (4, 80000)])
@pytest.mark.parametrize("bf16", [True, False])
def test_smallest_scales(T, V, bf16):
    """Logits up to the type's ends under scales that bring them back: their differences pass
    fp32's range, scale times them does not."""
    x = logits(np.random.default_rng(10), T, V, bf16)
    low = torch.finfo(x.dtype).min
    x.copy_((x.float().clamp(-9, 9) * 3.7e37).to(x.dtype))
    x[0, 3], x[0, 4] = low, -low
    x[1, ::2], x[1, 1::2] = low, -low
    x[2, 100:] = -torch.inf
    tokens = np.arange(T, dtype=np.int64) % V
    tokens[:3] = [3, 2, 50]
    for scale in (1e-38, 2e-38, 1e-37, 1e-44, 2.0 ** -100, 7e-31, 1e-20, 0.3):
        check(x, tokens, 9, scale=scale)


@pytest.mark.parametrize("V, bf16", [(128000, True), (100003, False), (600000, True)])
def test_one_workspace_for_a_falling_number_of_rows(V, bf16):
    """Its size is not one of the largest batch: the largest over all row counts serves each."""
    rng = np.random.default_rng(11)
    x = logits(rng, 300, V, bf16)
    tokens = rng.integers(0, V, 300)
    n = max(fp8.logprobs_workspace_bytes(T, V, 3, x.dtype) for T in [*range(1, 257), 300])
    store = torch.full((n + 64,), 0xff, dtype=torch.uint8, device="cuda")
    given = torch.as_tensor(tokens, device="cuda")
    for T in (300, 256, 255, 64, 1):
        got = fp8.token_logprobs(x[:T], given[:T], k=3, workspace=store[16:16 + n])
        want = fp8.token_logprobs(x[:T], given[:T], k=3)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (store[:16] == 0xff).all() and (store[16 + n:] == 0xff).all()
    check(x[:3], tokens[:3], 3, workspace=store[16:16 + n])


def test_buffers_are_written_whole_and_nothing_else():
    rng = np.random.default_rng(6)
    T, V, k = 6, 90000, 3
    x = logits(rng, T, V, True)
    n = fp8.logprobs_workspace_bytes(T, V, k)
    assert n > 0
    store = torch.full((n + 64,), 0xff, dtype=torch.uint8, device="cuda")
    f, i = (torch.full((T + 2,), 9, dtype=d, device="cuda") for d in (torch.float32, torch.int32))
    e, l = f.clone(), f.clone()
    top, ids = (torch.full((T + 2, k), 9, dtype=d, device="cuda") for d in (torch.float32, torch.int32))
    check(x, rng.integers(0, V, T), k, logprobs=f[1:-1], ranks=i[1:-1], entropy=e[1:-1], lse=l[1:-1],
          top_logprobs=top[1:-1], top_ids=ids[1:-1], workspace=store[16:16 + n])
    for t in (f, i, e, l, top, ids):
        assert (t[0] == 9).all() and (t[-1] == 9).all()
    assert (store[:16] == 0xff).all() and (store[16 + n:] == 0xff).all()


def test_empty_and_refusals():
    x = torch.zeros((4, 3000), dtype=torch.bfloat16, device="cuda")
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    assert fp8.token_logprobs(x[:0], tok[:0], k=2)[4].shape == (0, 2)
    n = fp8.logprobs_workspace_bytes(1, 128000, 1)
    wide, ws = torch.zeros((1, 128000), dtype=torch.bfloat16, device="cuda"), torch.zeros(
        n - 1, dtype=torch.uint8, device="cuda")

    def go(x=x, tok=tok, **more):
        fp8.token_logprobs(x, tok, **more)

    go()
    for bad, err in ((dict(x=x.half()), TypeError), (dict(x=x[0]), ValueError),
                     (dict(x=x.t()), ValueError), (dict(tok=tok[:3]), ValueError),
                     (dict(tok=tok.int()), TypeError), (dict(k=65), ValueError), (dict(k=-1), ValueError),
                     (dict(x=x[:, :2].contiguous(), k=3), ValueError), (dict(scale=0.0), ValueError),
                     (dict(scale=float("nan")), ValueError), (dict(logprobs=tok), TypeError),
                     (dict(ranks=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
                     (dict(k=2, top_ids=torch.zeros((4, 3), dtype=torch.int32, device="cuda")), ValueError),
                     (dict(x=wide, tok=tok[:1], workspace=ws), ValueError),
                     (dict(tok=tok.cpu()), ValueError)):
        with pytest.raises(err):
            go(**bad)
