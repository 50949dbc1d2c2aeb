"""fp8_paged_attention and fp8_prefix_attention against the float64 oracle
(needs a gfx950 GPU).

Each output element is held to the oracle's derived tolerance (bf16 half step
of the result, the fp16 rounding of the softmax weights, fp32 sums).  Every
cache place that no request maps holds NaN codes, so a read of what should be
masked shows."""

import numpy as np
import pytest
import torch

from oracle import attention, quant
from workloads import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_w8a8_block_amd as fp8

NAN = 0x7f


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def codes(rng, *shape):
    """E4M3 codes of values around 1/32 .. 16, no NaN."""
    c = rng.integers(0x10, 0x5c, shape, dtype=np.uint8)
    return c | (rng.integers(0, 2, shape, dtype=np.uint8) << 7)


class Batch:
    """A ragged batch; requests are (new tokens, length) pairs."""

    def __init__(self, seed, requests, Hq, Hk, D, page=16, far=0, pad=0, spare=0, q_scale=0.15):
        rng = np.random.default_rng(seed)
        self.rng, self.page, self.far = rng, page, far
        new, self.lens = [r[0] for r in requests], [r[1] for r in requests]
        self.offsets = np.cumsum([0] + new)
        T = int(self.offsets[-1]) + pad
        need = [-(-max(0, n) // page) for n in self.lens]
        shared = -(-far // page)
        nb = max(1, shared + sum(need) + 3)
        order = rng.permutation(nb)
        self.far_row = order[:shared].astype(np.int32)
        self.kc = np.full((nb, page, Hk, D), NAN, dtype=np.uint8)
        self.vc = np.full((nb, page, Hk, D), NAN, dtype=np.uint8)
        self.fill(self.far_row, far)
        self.table = np.full((len(requests), max(need + [1]) + spare), -1, dtype=np.int32)
        at = shared
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            self.fill(order[at:at + n], self.lens[r])
            at += n
        q = (rng.standard_normal((T, Hq, D)) * q_scale).astype(np.float32)
        self.q_bits = synth.f32_to_bf16_bits(q)
        self.ks, self.vs = np.float32(0.5), np.float32(0.25)
        self.shape = (T, Hq, Hk, D)

    def fill(self, blocks, length):
        for i, b in enumerate(blocks):
            n = min(self.page, length - i * self.page)
            self.kc[b, :n] = codes(self.rng, n, *self.kc.shape[2:])
            self.vc[b, :n] = codes(self.rng, n, *self.vc.shape[2:])

    def want(self, scale, window=0, sinks=0):
        q = quant.bf16_bits_to_f32(self.q_bits).astype(np.float64)
        extra = (self.far_row, self.far) if self.far else (None, 0)
        return attention.attention_ref(q, self.kc, self.vc, self.table, self.lens, self.offsets,
                                       scale, float(self.ks), float(self.vs), window, sinks, *extra)

    def run(self, scale=None, window=0, sinks=0, prefix=None, wide=False, workspace=None):
        T, Hq, Hk, D = self.shape
        q = bf16(self.q_bits)
        out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        table = i32(self.table)
        if wide:                                   # rows inside wider ones
            q = torch.cat([q, q.flip(0)], 1)[:, :Hq]
            out = torch.full((T, Hq + 3, D), 7.0, dtype=torch.bfloat16, device="cuda")[:, :Hq]
            table = torch.cat([table, table.flip(0)], 1)[:, :self.table.shape[1]]
        lse = torch.full((T, Hq), 7.0, device="cuda")
        kc, vc = torch.from_numpy(self.kc).cuda(), torch.from_numpy(self.vc).cuda()
        ks, vs = torch.tensor([self.ks], device="cuda"), torch.tensor([self.vs], device="cuda")
        args = (table, i32(self.lens), i32(self.offsets), ks, vs)
        if (self.far > 0) if prefix is None else prefix:
            fp8.prefix_attention(q, kc, vc, i32(self.far_row), i32([self.far]), *args, scale=scale,
                                 out=out, lse=lse, workspace=workspace)
        else:
            fp8.paged_attention(q, kc, vc, *args, scale=scale, window=window, sinks=sinks, out=out,
                                lse=lse, workspace=workspace)
        torch.cuda.synchronize()
        return out, lse

    def check(self, scale=None, window=0, sinks=0, prefix=None, wide=False):
        out, lse = self.run(scale, window, sinks, prefix, wide)
        close(f64(out), lse.cpu().numpy().astype(np.float64),
              self.want(self.shape[3] ** -0.5 if scale is None else scale, window, sinks))


def close(out, lse, want):
    ref, ref_lse, tol, tol_lse, covered = want
    assert (out[~covered] == 7.0).all() and (lse[~covered] == 7.0).all(), "rows of no request"
    out, lse, ref, ref_lse = (x[covered] for x in (out, lse, ref, ref_lse))
    tol, tol_lse = tol[covered], tol_lse[covered]
    assert np.array_equal(np.isnan(out), np.isnan(ref)), \
        (int(np.isnan(out).sum()), int(np.isnan(ref).sum()))
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref_lse))
    fine = ~np.isnan(ref)
    off = np.abs(out - ref)[fine] - tol[fine]
    assert (off <= 0).all(), (off.max(), np.argwhere((np.abs(out - ref) > tol) & fine)[:4].tolist())
    fine = np.isfinite(ref_lse)
    off = np.abs(lse[fine] - ref_lse[fine]) - tol_lse[fine]
    assert (off <= 0).all(), off.max()


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 257, 600]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 4, 7, 16, 20])
def test_single_tokens(D, G):
    Batch([D, G], [(1, n) for n in LENGTHS], 2 * G, 2, D).check()


@pytest.mark.parametrize("page", [1, 3, 16, 64, 1000])
def test_pages(page):
    Batch(page, [(1, n) for n in LENGTHS] + [(40, 70)], 8, 2, 64, page=page).check()


def test_empty_rows_and_requests():
    """No keys, no queries, more queries than tokens, tokens behind the last request."""
    b = Batch(1, [(0, 50), (1, 0), (2, 1), (0, 0), (1, 40), (5, 3), (0, 9)], 8, 2, 128, pad=3)
    b.check()
    b = Batch(2, [(0, 0)], 4, 4, 64, pad=2)
    b.check()
    b = Batch(3, [(60, 20), (0, 5), (200, 0), (80, 130)], 8, 2, 64, pad=9)
    b.check()
    b.lens[3] = -7                                    # a negative length is none
    b.check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("requests", [[(2, 2)], [(3, 130), (3, 40), (3, 3)], [(33, 33)],
                                      [(128, 128)], [(129, 400), (7, 9), (1, 300)],
                                      [(64, 64), (200, 263)]])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (3, 1)])
def test_several_tokens(D, requests, heads):
    Batch([D, len(requests)], requests, *heads, D).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (5, 3), (100, 4), (128, 1), (17, 200),
                                          (1000, 4), (64, 64), (0, 5)])
def test_window_and_sinks(window, sinks):
    few = [(1, n) for n in LENGTHS + [1500]]
    Batch(window, few, 8, 2, 64).check(window=window, sinks=sinks)
    Batch(window, [(2, 300), (1, 700), (3, 3), (2, 1)], 8, 2, 128).check(window=window, sinks=sinks)
    Batch(window, [(150, 150), (90, 500), (1, 800)], 4, 1, 64).check(window=window, sinks=sinks)
    Batch(window, [(70, 300)], 4, 2, 128).check(window=window, sinks=sinks)


def test_widest_window():
    """A window and sinks of the largest number, with queries before position 0."""
    big = (1 << 31) - 1
    for D in (64, 128):
        b = Batch(D, [(1, 40), (3, 1), (1, 0), (70, 9)], 8, 2, D)
        b.check(window=big)
        b.check(window=big, sinks=big)
    b = Batch(7, [(90, 20), (200, 131)], 8, 2, 64)
    b.check(window=big, sinks=3)


@pytest.mark.parametrize("n", [1, 70])
def test_longest_requests(n):
    """A request of 2^31 - 65536 keys in repeated blocks of 2^20, seen through a
    window, against its last block alone; and a length that passes that."""
    page, D, most = 1 << 20, 64, 0x7fff0000
    rng = np.random.default_rng(n)
    kc, vc = (torch.from_numpy(codes(rng, 2, page, 1, D)).cuda() for _ in range(2))
    one = torch.ones(1, device="cuda")
    q = bf16(synth.f32_to_bf16_bits((rng.standard_normal((n, 4, D)) * 0.15).astype(np.float32)))
    table = np.zeros((1, 2048), dtype=np.int32)
    table[0, 2047] = 1
    offs = i32([0, n])
    far = fp8.paged_attention(q, kc, vc, i32(table), i32([most]), offs, one, one, window=300)
    near = fp8.paged_attention(q, kc, vc, i32([[1]]), i32([most - 2047 * page]), offs, one, one,
                               window=300)
    assert torch.isfinite(far.float()).all()
    assert torch.equal(far.view(torch.int16), near.view(torch.int16))
    out = fp8.paged_attention(q, kc, vc, i32(table), i32([(1 << 31) - 1]), offs, one, one,
                              window=300)
    assert (out == 0).all()                        # nothing of their windows is there


def test_long_context():
    """One request over many shares, and a batch of more requests than a scan pass."""
    Batch(1, [(1, 20011)], 4, 1, 64).check()
    Batch(2, [(1, 9001)], 32, 8, 128).check()
    rng = np.random.default_rng(3)
    many = [(int(rng.integers(0, 2)), int(rng.integers(0, 60))) for _ in range(700)]
    Batch(4, many, 4, 2, 64).check()
    Batch(5, [(n + 30, s + n + 30) for n, s in many[:300]], 4, 4, 64).check()


def test_large_scores():
    """Softmaxes of one key and of many, where the running maximum moves a lot."""
    Batch(1, [(1, n) for n in LENGTHS], 8, 2, 128, q_scale=8.0).check()
    Batch(2, [(150, 300)], 8, 2, 128, q_scale=8.0).check()
    Batch(3, [(1, 300), (1, 33)], 8, 2, 64, q_scale=1.0).check(scale=-0.7)


def test_strides():
    Batch(1, [(1, n) for n in LENGTHS], 8, 2, 128, spare=2).check(wide=True)
    Batch(2, [(150, 300), (1, 9)], 8, 2, 64, spare=2).check(wide=True)
    Batch(3, [(1, n) for n in LENGTHS], 8, 2, 64, far=77, spare=2).check(wide=True)


@pytest.mark.parametrize("requests", [[(1, 200), (1, 100), (1, 64)], [(90, 200), (60, 100), (9, 64)]])
def test_bad_tables(requests):
    """Entries outside the cache and tables that end early hide their keys."""
    b = Batch(1, requests, 8, 2, 64)
    b.table[0, 2], b.table[0, 5], b.table[1, 1:] = -1, 1 << 20, -5
    b.table[2, 3] = b.kc.shape[0]
    b.check()
    b.table = b.table[:, :4].copy()                  # 64 tokens fit
    b.check()
    b.table = b.table[:, :0].copy()
    b.check()


@pytest.mark.parametrize("requests,window", [([(1, 150), (1, 40)], 0), ([(3, 150), (2, 40)], 0),
                                             ([(100, 150)], 0), ([(100, 400), (2, 200)], 30),
                                             ([(1, 150), (2, 140)], 20)])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_codes(requests, window, D):
    """A NaN code reaches the rows that see it, and no other."""
    b = Batch(D, requests, 8, 2, D)
    page = b.page
    for r, (n, length) in enumerate(requests):
        for j, cache in ((length - 1, b.vc), (max(0, length - n // 2 - 1), b.vc),
                         (max(0, length - 40), b.vc), (max(0, length - 3), b.kc)):
            cache[b.table[r, j // page], j % page, r % 2, (7 * j) % D] = 0xff if j % 2 else 0x7f
    b.check(window=window)
    b.check(window=window, sinks=2)


def test_infinite_queries():
    b = Batch(1, [(1, 50), (1, 60)], 4, 2, 64)
    b.q_bits[0, 0, 0] = 0x7fc0                       # NaN: its row alone
    out, lse = b.run()
    o = f64(out)
    assert np.isnan(o[0, 0]).all() and np.isfinite(o[0, 1:]).all() and np.isfinite(o[1]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("far", [1, 15, 64, 200, 1003])
def test_prefix(D, far):
    Batch([D, far], [(1, n) for n in LENGTHS], 8, 2, D, far=far).check()


@pytest.mark.parametrize("requests,heads", [([(1, 1)], (4, 1)), ([(1, 5), (1, 700)], (2, 2)),
                                            ([(2, 30)] * 20, (8, 2)), ([(60, 60), (9, 200)], (8, 2)),
                                            ([(0, 4), (1, 0), (3, 1), (0, 0)], (8, 2)),
                                            ([(1, 9)] * 300, (4, 2))])
def test_prefix_batches(requests, heads):
    Batch(len(requests), requests, *heads, 64, far=333, pad=2).check()
    Batch(len(requests), requests, *heads, 128, page=7, far=40, pad=1).check()


def test_prefix_of_nothing_and_bad_prefixes():
    b = Batch(1, [(1, 40), (3, 9), (1, 0)], 8, 2, 64, far=50, pad=2)
    b.far = 0
    b.far_row = b.far_row[:0]
    b.check(prefix=True)
    b = Batch(2, [(1, 40), (30, 90), (1, 0)], 8, 2, 64, far=100)
    b.far_row[[0, 3]] = [-1, 1 << 20]
    b.check()
    b.far_row = b.far_row[:2]                        # 32 of 100 tokens in the table
    b.check()
    b.kc[b.far_row[1], 3, 1, 5] = NAN                # seen by every query of its head
    b.check()


def test_prefix_equals_joined_requests():
    """The same tokens as one request each, up to the order of the sums."""
    b = Batch(1, [(1, n) for n in LENGTHS], 8, 2, 128, page=16, far=160)
    out, lse = b.run()
    rows = [np.concatenate([b.far_row, row]) for row in b.table]
    joined = Batch(1, [(1, n) for n in LENGTHS], 8, 2, 128, page=16, far=160)
    joined.table = np.stack(rows)
    joined.lens = [n + 160 for n in LENGTHS]
    joined.far = 0
    joined.check()
    o2, l2 = joined.run()
    assert torch.allclose(out.float(), o2.float(), rtol=2 ** -7, atol=1e-4)
    assert torch.allclose(lse, l2, rtol=1e-5, atol=1e-5)


def test_far_places_in_a_large_cache():
    """Places of the cache behind 4 GiB."""
    page, Hk, D, nb = 16, 8, 128, 300000
    b = Batch(1, [(1, 500), (3, 40), (1, 17)], 16, Hk, D, page=page)
    small = b.kc.shape[0]
    shift = nb - small
    kc, vc = (torch.zeros((nb, page, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    kc[shift:], vc[shift:] = torch.from_numpy(b.kc).cuda(), torch.from_numpy(b.vc).cuda()
    table = np.where(b.table >= 0, b.table + shift, -1)
    T, Hq = b.shape[:2]
    for _ in range(2):                               # few rows, then many
        lse = torch.full((b.shape[0], Hq), 7.0, device="cuda")
        out = fp8.paged_attention(bf16(b.q_bits), kc, vc, i32(table), i32(b.lens), i32(b.offsets),
                                  torch.tensor([b.ks], device="cuda"),
                                  torch.tensor([b.vs], device="cuda"), lse=lse)
        close(f64(out), lse.cpu().numpy().astype(np.float64), b.want(D ** -0.5))
        b = Batch(2, [(100, 500)], 16, Hk, D, page=page)
        kc[nb - b.kc.shape[0]:] = torch.from_numpy(b.kc).cuda()
        vc[nb - b.vc.shape[0]:] = torch.from_numpy(b.vc).cuda()
        table = np.where(b.table >= 0, b.table + nb - b.kc.shape[0], -1)


def test_repeats_are_bit_identical():
    b = Batch(1, [(1, n) for n in LENGTHS] + [(50, 3000)], 8, 2, 128, far=2000)
    for prefix in (False, True):
        first = b.run(prefix=prefix)
        # another workspace content and address
        ws = torch.full((fp8.attention_workspace_bytes(*b.shape[:1], len(b.lens), *b.shape[1:],
                                                       shared_prefix=prefix) + 64,), 0xff,
                        dtype=torch.uint8, device="cuda")
        again = b.run(prefix=prefix, workspace=ws)
        for x, y in zip(first, again):
            assert torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                               y.view(torch.int16 if y.dtype == torch.bfloat16 else torch.int32))


def test_refusals():
    b = Batch(1, [(1, 40), (1, 9)], 8, 2, 64)
    T, Hq, Hk, D = b.shape
    q, kc, vc = bf16(b.q_bits), torch.from_numpy(b.kc).cuda(), torch.from_numpy(b.vc).cuda()
    one = torch.ones(1, device="cuda")

    def go(q=q, kc=kc, table=i32(b.table), lens=i32(b.lens), offs=i32(b.offsets), ks=one, **kw):
        return fp8.paged_attention(q, kc, vc, table, lens, offs, ks, one, **kw)

    go()
    out = torch.empty_like(q)
    for bad, err in ((dict(q=q.half()), TypeError), (dict(q=q[..., :32].contiguous()), ValueError),
                     (dict(kc=kc[..., :32]), ValueError), (dict(kc=kc[:2]), ValueError),
                     (dict(table=i32(b.table).long()), TypeError),
                     (dict(table=i32(b.table)[:1]), ValueError),
                     (dict(lens=i32(b.lens)[:1]), ValueError), (dict(offs=i32([0, 1])), ValueError),
                     (dict(ks=one.double()), TypeError), (dict(window=-1), ValueError),
                     (dict(sinks=-1), ValueError), (dict(scale=float("nan")), ValueError),
                     (dict(out=q), ValueError), (dict(out=out[:1]), ValueError),
                     (dict(lse=torch.empty((T, 3), device="cuda")), ValueError),
                     (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), ValueError),
                     (dict(q=q[:, :3].contiguous()), ValueError)):
        with pytest.raises(err):
            go(**bad)
    with pytest.raises(TypeError):
        fp8.prefix_attention(q, kc, vc, i32([0]), None, i32(b.table), i32(b.lens), i32(b.offsets),
                             one, one)
    with pytest.raises(TypeError):
        fp8.prefix_attention(q, kc, vc, i32([0]).long(), i32([1]), i32(b.table), i32(b.lens),
                             i32(b.offsets), one, one)


def test_prefix_of_many_rows():
    """More rows than waves of one grid: 2^26 and some, against slices of them.

    Prefix and own keys are one key tile each, so that no share cuts a row's sums
    and slices have the same bits."""
    T, Hq, D, page, far, own, part = (1 << 21) + 1, 32, 64, 16, 40, 3, 1000
    rng = np.random.default_rng(8)
    kc, vc = (torch.from_numpy(codes(rng, 4, page, Hq, D)).cuda() for _ in range(2))
    one = torch.ones(1, device="cuda")
    q = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    for a in range(0, T, 1 << 17):
        q[a:a + (1 << 17)] = torch.randn(q[a:a + (1 << 17)].shape, generator=g, device="cuda") * 0.15

    def go(q, length):
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        out = torch.full_like(q, 7.0)
        fp8.prefix_attention(q, kc, vc, i32([2, 0, 1]), i32([far]), i32([[3]]), i32([length]),
                             i32([0, len(q)]), one, one, out=out, lse=lse)
        return out, lse

    out, lse = go(q, own)
    edge = (1 << 26) // Hq
    # the last three tokens are the ones that see own keys
    for a in (0, edge // 16 - part // 2, edge // 3, edge - part - own, T - part):
        o, l = go(q[a:a + part], own if a + part == T else 0)
        assert torch.equal(out[a:a + part].view(torch.int16), o.view(torch.int16)), a
        assert torch.equal(lse[a:a + part], l), a
    assert torch.isfinite(lse).all() and not (lse == 7.0).any()


@pytest.mark.parametrize("requests", [[(2, 1), (3, 2), (1, 0), (1, 4)],
                                      [(60, 59), (70, 90), (1, 0), (90, 90)]])
def test_prefix_equals_joined_requests_with_few_own_tokens(requests):
    """All but one of a request's queries among its own tokens: still the joined form."""
    far = 160
    b = Batch(9, requests, 8, 2, 64, far=far)
    b.check()
    split = b.want(64 ** -0.5)
    b.table = np.concatenate([b.far_row[None].repeat(len(requests), 0), b.table], 1)
    b.lens, b.far = [n + far for n in b.lens], 0
    b.check()
    joined = b.want(64 ** -0.5)
    for x, y in zip(split[:2], joined[:2]):          # one definition, in 64 bits
        assert np.allclose(x, y, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("requests", [[(2, 0), (4, 1), (1, 1)], [(60, 20), (70, 3)]])
def test_queries_inside_the_prefix_see_all_of_it(requests):
    """Fewer own tokens than that: the first queries see what all others see of the prefix."""
    b = Batch(10, requests, 8, 2, 64, far=100)
    b.check()
    out, lse = b.run()
    b.lens = [0] * len(requests)                     # the prefix alone
    o2, l2 = b.run()
    for r, (n, length) in enumerate(requests):
        first = slice(int(b.offsets[r]), int(b.offsets[r]) + n - length)
        assert torch.equal(out[first].view(torch.int16), o2[first].view(torch.int16))
        assert torch.equal(lse[first], l2[first])


@pytest.mark.parametrize("heads,D", [((4, 1), 64), ((8, 2), 128)])
def test_more_requests_than_a_scan_pass_of_the_large_tiles(heads, D):
    """Requests behind the 512th and the 1024th of the 256-row kernel's shares, some
    without queries or keys; one of several row tiles behind them."""
    rng = np.random.default_rng(D)
    many = [(int(n), int(max(0, n + s))) for n, s in
            zip(rng.integers(0, 40, 1100), rng.integers(-20, 60, 1100))]
    many[1030] = (300, 700)
    assert sum(n for n, _ in many) * heads[0] // heads[1] > 48 * len(many)
    Batch(D, many, *heads, D, pad=5).check()
    Batch(D + 1, many[:700], *heads, D, far=150).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("shared", [False, True])
def test_one_workspace_serves_any_number_of_requests(D, shared):
    """Sized for all tokens in one request, it is large enough for fewer and for any batch."""
    def need(T, B):
        return fp8.attention_workspace_bytes(T, B, 8, 2, D, shared_prefix=shared)

    sizes = [1, 3, 12, 13, 64, 500, 4000]
    for T in sizes:
        for B in (1, 2, 5, 40, 400):
            assert need(T, B) <= need(T, 1), (T, B)
            assert all(need(t, B) <= need(T, B) for t in sizes if t <= T), (T, B)
    ws = torch.empty(need(600, 1), dtype=torch.uint8, device="cuda")
    for requests in ([(1, 40)] * 50, [(300, 300), (2, 9)]):
        b = Batch(D, requests, 8, 2, D, far=70 if shared else 0)
        out, lse = b.run(workspace=ws)
        close(f64(out), lse.cpu().numpy().astype(np.float64), b.want(D ** -0.5))
