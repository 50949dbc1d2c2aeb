"""The operators around the linears as a served step runs them: norm with FP8
codes, the QKV product, positions on three axes, attention, the output linear,
norm, a 4-bit head, log probabilities -- eager, captured and replayed, on another
stream, two at once; and each of them where offsets pass 32 bits (needs a gfx950
GPU).

Each operator's output is held to the oracle on what the operator before it left
on the device."""

import numpy as np
import pytest
import torch

from oracle import attention, e4m3, quant, step
from workloads import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_w8a8_block_amd as fp8

EPS = 1e-6
SECTIONS = (24, 20, 20)
REACH = 200


def bf16(x):
    bits = synth.f32_to_bf16_bits(np.asarray(x, dtype=np.float32))
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def same(x, y):
    return torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


class Layer:
    """A layer and a head over it, with all buffers of a step of T tokens, some of them padding."""

    def __init__(self, seed, T=37, B=5, H=512, Hq=4, Hk=2, D=128, V=5003, k=6, page=16, width=4):
        self.rng = rng = np.random.default_rng(seed)
        self.T, self.B, self.H, self.Hq, self.Hk, self.D, self.V, self.k = T, B, H, Hq, Hk, D, V, k
        self.page = page
        dev, n = "cuda", Hq + 2 * Hk
        self.w1, self.w2 = bf16(rng.uniform(0.5, 1.5, H)), bf16(rng.uniform(0.5, 1.5, H))
        self.qw, self.kw = bf16(rng.uniform(0.5, 1.5, D)), bf16(rng.uniform(0.5, 1.5, D))
        self.wqkv = fp8.quant_weight_block(bf16(rng.standard_normal((n * D, H)) / H ** 0.5))
        self.wo = fp8.quant_weight_block(bf16(rng.standard_normal((H, Hq * D)) / (Hq * D) ** 0.5))
        self.head = fp8.int4_quant_weight(bf16(rng.standard_normal((V, H)) / H ** 0.5), 64)
        ang = np.arange(REACH)[:, None] * (1e4 ** (-np.arange(D // 2) / (D // 2)))[None]
        self.cs = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)
                                   .astype(np.float32)).cuda()
        self.ks, self.vs = torch.tensor([0.0625], device=dev), torch.tensor([0.03125], device=dev)
        nb = B * width
        self.free = torch.tensor(rng.permutation(nb), dtype=torch.int32, device=dev)
        self.kc = torch.full((nb, page, Hk, D), 0x7f, dtype=torch.uint8, device=dev)
        self.vc = torch.full((nb, page, Hk, D), 0x7f, dtype=torch.uint8, device=dev)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        self.computed = torch.zeros(B, dtype=torch.int32, device=dev)
        self.new = torch.zeros(B, dtype=torch.int32, device=dev)
        self.slots = torch.empty(T, dtype=torch.int64, device=dev)
        self.pos = torch.empty(T, dtype=torch.int64, device=dev)
        self.offsets = torch.empty(B + 1, dtype=torch.int32, device=dev)
        self.lens = torch.empty(B, dtype=torch.int32, device=dev)
        self.taken = torch.empty(1, dtype=torch.int32, device=dev)
        self.shift = torch.tensor(rng.integers(0, 100, (3, T)), device=dev)
        self.x = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.res0 = torch.empty_like(self.x)
        self.res, self.res2 = torch.empty_like(self.x), torch.empty_like(self.x)
        self.xq = torch.empty((T, H), dtype=torch.uint8, device=dev)
        self.xs = torch.empty((T, H // 128), device=dev)
        self.qkv = torch.empty((T, n * D), dtype=torch.bfloat16, device=dev)
        self.q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
        self.o = torch.full((T, Hq, D), 0.0, dtype=torch.bfloat16, device=dev)
        self.ws = torch.empty(fp8.attention_workspace_bytes(T, B, Hq, Hk, D), dtype=torch.uint8,
                              device=dev)
        self.h = torch.empty_like(self.x)
        self.y = torch.empty_like(self.x)
        self.last = torch.empty((B, H), dtype=torch.bfloat16, device=dev)
        self.logits = torch.empty((B, V), dtype=torch.bfloat16, device=dev)
        self.tokens = torch.empty(B, dtype=torch.int64, device=dev)
        self.probs = [torch.empty(B, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                      torch.empty(B, device=dev), torch.empty(B, device=dev),
                      torch.empty((B, k), device=dev),
                      torch.empty((B, k), dtype=torch.int32, device=dev)]

    def feed(self, new):
        rng = self.rng
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.x.copy_(bf16(rng.standard_normal((self.T, self.H))))
        self.res0.copy_(bf16(rng.standard_normal((self.T, self.H)) * 3))
        self.tokens.copy_(torch.tensor(rng.integers(0, self.V, self.B)))

    def step(self):
        T, Hq, Hk, D = self.T, self.Hq, self.Hk, self.D
        fp8.add_rms_norm_quant(self.x, self.w1, residual=self.res0, eps=EPS, q=self.xq, scales=self.xs,
                               residual_out=self.res)
        fp8.block_gemm(self.xq, self.xs, *self.wqkv, out=self.qkv)
        fp8.kv_slot_map(self.computed, self.new, self.table, self.free, self.page, T, self.slots, self.pos,
                        self.offsets, self.lens, self.taken)
        self.pos3 = torch.where(self.pos >= 0, self.pos + self.shift, self.pos)
        x = self.qkv.view(T, Hq + 2 * Hk, D)
        fp8.qk_norm_mrope_cache(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], self.qw, self.kw, self.cs,
                                self.pos3, SECTIONS, self.slots, self.kc, self.vc, self.ks, self.vs,
                                eps=EPS, in_turn=True, query_out=self.q)
        fp8.paged_attention(self.q, self.kc, self.vc, self.table, self.lens, self.offsets, self.ks, self.vs,
                            out=self.o, workspace=self.ws)
        fp8.linear(self.o.view(T, Hq * D), *self.wo, out=self.h)
        fp8.add_rms_norm(self.h, self.w2, residual=self.res, eps=EPS, out=self.y, residual_out=self.res2)
        torch.index_select(self.y, 0, self.offsets[1:].long() - 1, out=self.last)
        fp8.int4_linear(self.last, *self.head, out=self.logits)
        fp8.token_logprobs(self.logits, self.tokens, k=self.k, logprobs=self.probs[0], ranks=self.probs[1],
                           entropy=self.probs[2], lse=self.probs[3], top_logprobs=self.probs[4],
                           top_ids=self.probs[5])

    def advance(self):
        self.free.copy_(torch.roll(self.free, -int(self.taken)))
        self.computed.copy_(self.lens)

    STATE = ("kc", "vc", "table", "xq", "xs", "res", "qkv", "q", "o", "h", "y", "res2", "logits")

    def state(self):
        return {**{n: getattr(self, n).clone() for n in self.STATE},
                **{f"probs{i}": t.clone() for i, t in enumerate(self.probs)}}


def check_norm(x, residual, w, res):
    """The residual bit for bit -> (norm float64, its tolerance)."""
    total = step.add_ref(bits_of(x), bits_of(residual))
    assert np.array_equal(bits_of(res), total)
    return step.norm_ref(total, bits_of(w), EPS)


def check_layer(s):
    v, tol = check_norm(s.x, s.res0, s.w1, s.res)
    scale = np.repeat(f64(s.xs), 128, 1)
    off = np.abs(e4m3.decode(s.xq.cpu().numpy()).astype(np.float64) * scale - v)
    # half a step: 2^-4 of the value, of subnormals 2^-10 of the scale; the scale's own rounding
    assert (off <= np.abs(v) * (2.0 ** -4 + 2.0 ** -20) + scale * 2.0 ** -10 + 2 * tol).all()
    T, Hq, Hk, D = s.T, s.Hq, s.Hk, s.D
    pos = s.pos3.cpu().numpy()
    live = (pos >= 0).all(0)
    axis = np.array(step.axes_ref(SECTIONS, True))
    at, cs = np.where(live, pos, 0)[axis].T, s.cs.cpu().numpy().astype(np.float64)
    cos, sin = cs[at, np.arange(D // 2)], cs[at, D // 2 + np.arange(D // 2)]
    z, tol = attention.norm_rope_ref(f64(s.qkv).reshape(T, -1, D)[:, :Hq], f64(s.qw), EPS, cos, sin, False)
    assert (np.abs(f64(s.q) - z)[live] <= (np.abs(z) * 2.0 ** -8 + 2 * tol)[live]).all()
    v, tol = check_norm(s.h, s.res, s.w2, s.res2)
    assert (np.abs(f64(s.y) - v) <= np.abs(v) * 2.0 ** -8 + 2 * tol).all()
    codes, scales, zeros = (t.cpu().numpy() for t in s.head)
    b = codes.reshape(s.V, -1, 4)
    values = np.stack([b[..., 0] & 15, b[..., 2] & 15, b[..., 0] >> 4, b[..., 2] >> 4,
                       b[..., 1] & 15, b[..., 3] & 15, b[..., 1] >> 4, b[..., 3] >> 4], -1)
    values = values.reshape(s.V, -1)
    assert np.array_equal(step.int4_pack_ref(values), codes)
    want, tol = step.int4_linear_ref(bits_of(s.last), values, scales, zeros)
    assert (np.abs(f64(s.logits) - want) <= np.abs(want) * 2.0 ** -8 + tol * (1 + 2.0 ** -8)).all()
    want, tol = step.logprobs_ref(f64(s.logits), s.tokens.cpu().numpy(), s.k, 1.0)
    got = dict(zip(("logprobs", "ranks", "entropy", "lse", "top", "ids"), s.probs))
    for n in ("ranks", "ids"):
        assert np.array_equal(got[n].cpu().numpy(), want[n])
    for n in ("logprobs", "entropy", "lse", "top"):
        assert (np.abs(f64(got[n]) - want[n]) <= tol(want[n])).all(), n


STEPS = ([9, 1, 17, 3, 5], [1, 1, 1, 1, 1], [1, 16, 1, 2, 1])


def test_steps_against_oracle():
    s = Layer(1)
    for new in STEPS:
        s.feed(new)
        before = s.state()
        s.step()
        torch.cuda.synchronize()
        check_layer(s)
        for n in ("q", "o"):                              # padding's rows as they were
            assert same(getattr(s, n)[sum(new):], before[n][sum(new):])
        s.advance()


def test_captured_steps():
    """One captured step, replayed with other lengths and rows, with eager steps between."""
    def run(captured):
        s, other, states, graph = Layer(2), Layer(3), [], None
        for i, new in enumerate(STEPS + STEPS[1:]):
            s.feed(new)
            if captured and graph is None:
                warm = torch.cuda.Stream()
                warm.wait_stream(torch.cuda.current_stream())
                before = {n: getattr(s, n).clone() for n in ("kc", "vc", "table")}
                with torch.cuda.stream(warm):
                    s.step()
                torch.cuda.current_stream().wait_stream(warm)
                for n, t in before.items():
                    getattr(s, n).copy_(t)
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    s.step()
            if captured:
                graph.replay()
                other.feed([1] * 5)
                other.step()
            else:
                s.step()
            torch.cuda.synchronize()
            states.append(s.state())
            s.advance()
        return states

    for a, b in zip(run(False), run(True)):
        for n in a:
            assert same(a[n], b[n]), n


def test_two_at_once_on_other_streams():
    def run(streams):
        layers = [Layer(4), Layer(5, V=70001)]
        out = []
        for new in STEPS:
            for s, stream in zip(layers, streams):
                s.feed(new)
            torch.cuda.synchronize()
            for _ in range(3):                              # the same step again: same results
                for s, stream in zip(layers, streams):
                    with torch.cuda.stream(stream):
                        s.step()
            torch.cuda.synchronize()
            out += [s.state() for s in layers]
            for s in layers:
                s.advance()
        return out

    here = torch.cuda.current_stream()
    for a, b in zip(run((here, here)), run((torch.cuda.Stream(), torch.cuda.Stream()))):
        for n in a:
            assert same(a[n], b[n]), n


def test_graphs_that_share_a_workspace():
    """4-bit products cut into runs and rows' parts of log probabilities, all in one workspace."""
    rng = np.random.default_rng(6)
    jobs = []
    for M, N, K, V in ((24, 256, 8192, 130000), (100, 301, 4096, 90001)):
        x = bf16(rng.standard_normal((M, K)))
        w = fp8.int4_quant_weight(bf16(rng.standard_normal((N, K))), 64)
        lo = bf16(rng.standard_normal((4, V)))
        n = (fp8.int4_workspace_bytes(M, N, K), fp8.logprobs_workspace_bytes(4, V, 20))
        assert min(n) > 0
        jobs.append((x, w, lo, torch.tensor([0, 1, 2, V - 1], device="cuda"), max(n)))
    ws = torch.empty(max(j[-1] for j in jobs), dtype=torch.uint8, device="cuda")

    def run(job, workspace):
        x, w, lo, tokens, _ = job
        return [fp8.int4_linear(x, *w, workspace=workspace),
                *fp8.token_logprobs(lo, tokens, k=20, workspace=workspace)]

    want = [run(j, None) for j in jobs]
    graphs = []
    for job in jobs:
        run(job, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(job, ws)
        graphs.append((g, out))
    for _ in range(4):
        for (g, out), w, job in zip(graphs, want, jobs):
            for t in out:
                t.fill_(3)
            g.replay()
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(out, w))
            ws.fill_(0xff)
            assert all(same(a, b) for a, b in zip(run(job, None), w))


# ---- offsets past 32 bits

@pytest.fixture(autouse=True)
def memory_back():
    yield
    torch.cuda.empty_cache()


def rows_apart(bits, ld):
    """The rows ld values apart in their storage, which is not filled between them."""
    T, H = bits.shape
    store = torch.empty((T - 1) * ld + H, dtype=torch.bfloat16, device="cuda")
    t = store.as_strided((T, H), (ld, 1))
    t.copy_(torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16))
    return t


def normal(rng, *shape):
    return synth.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


@pytest.mark.parametrize("mode", ["block", "row"])
def test_norm_rows_far_apart(mode):
    rng, T, H, ld = np.random.default_rng(7), 5, 1152, 2 ** 30 + 8
    x, r, w = normal(rng, T, H), normal(rng, T, H), bf16(rng.uniform(0.5, 1.5, H))
    a, b, o, ro = (rows_apart(t, ld) for t in (x, r, x * 0, x * 0))
    q, s = fp8.add_rms_norm_quant(a, w, residual=b, scale_mode=mode, out=o, residual_out=ro)
    near = [torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q2, s2 = fp8.add_rms_norm_quant(a.contiguous(), w, residual=b.contiguous(), scale_mode=mode, out=near[0],
                                    residual_out=near[1])
    assert same(q, q2) and same(s, s2) and same(o, near[0]) and same(ro, near[1])
    check_norm(a, b, w, ro)


def test_norm_of_many_rows():
    """More than 2^32 values: the last rows are the ones they are alone."""
    T, H = 4190000, 1152
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    q, s = fp8.add_rms_norm_quant(x, w)
    for rows in (slice(0, 3), slice(T // 2, T // 2 + 3), slice(T - 3, T)):
        q1, s1 = fp8.add_rms_norm_quant(x[rows].contiguous(), w)
        assert same(q[rows], q1) and same(s[rows], s1)


def test_axes_far_apart():
    """Rows, caches and axes of positions far apart."""
    rng, T, Hq, Hk, D = np.random.default_rng(8), 4, 3, 2, 128
    ld, page = 3 * 2 ** 29, 16
    row = normal(rng, T, (Hq + 2 * Hk) * D)
    ang = np.arange(REACH)[:, None] * (1e4 ** (-np.arange(D // 2) / (D // 2)))[None]
    cs = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    w, one = bf16(rng.uniform(0.5, 1.5, D)), torch.tensor([0.05], device="cuda")
    nb = 2 ** 33 // (page * Hk * D)
    kc, vc = (torch.empty((nb, page, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    pos = torch.tensor(rng.integers(0, REACH, (3, T)), device="cuda")
    apart = torch.empty(2 * 2 ** 29 + T, dtype=torch.int64, device="cuda").as_strided((3, T), (2 ** 29, 1))
    apart.copy_(pos)
    slots = torch.tensor([nb * page - 1, 3, 2 ** 24 + 5, nb * page // 2], device="cuda")

    def run(x, pos, slots, kc, vc, out):
        x = x.as_strided((T, Hq + 2 * Hk, D), (x.stride(0), D, 1))
        return fp8.qk_norm_mrope_cache(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], w, w, cs, pos,
                                       SECTIONS, slots, kc, vc, one, one, query_out=out)

    far = rows_apart(row, ld)
    out = torch.empty((T - 1) * ld + Hq * D, dtype=torch.bfloat16, device="cuda")
    out = out.as_strided((T, Hq, D), (ld, D, 1))
    run(far, apart, slots, kc, vc, out)
    kn, vn = (torch.zeros((1, page, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    want = run(far.contiguous(), pos, torch.arange(T, device="cuda"), kn, vn, None)
    assert same(out, want)
    for big, small in ((kc, kn), (vc, vn)):
        assert same(big.view(-1, Hk, D)[slots], small.view(-1, Hk, D)[:T])


def tail_products(x, codes, scales, zeros, out, rows):
    """out's columns `rows` against the float64 definition."""
    b = codes[rows].cpu().numpy().reshape(len(rows), -1, 4)
    values = np.stack([b[..., 0] & 15, b[..., 2] & 15, b[..., 0] >> 4, b[..., 2] >> 4,
                       b[..., 1] & 15, b[..., 3] & 15, b[..., 1] >> 4, b[..., 3] >> 4], -1)
    want, tol = step.int4_linear_ref(bits_of(x), values.reshape(len(rows), -1), scales[rows].cpu().numpy(),
                                     zeros[rows].cpu().numpy())
    assert (np.abs(f64(out[:, rows]) - want) <= np.abs(want) * 2.0 ** -8 + tol * (1 + 2.0 ** -8)).all()


# M, N, K
FAR = {"few": (1, 32768, 2 ** 18 + 128), "few_rows": (3, 32768, 2 ** 18 + 128),
       "batch": (13, 140000, 65536), "batch_few_columns": (16, 4096, 2 ** 21 + 256),
       "middle": (20, 140000, 65536), "many": (70, 140000, 65536)}


@pytest.mark.parametrize("case", list(FAR))
def test_int4_of_a_large_weight(case):
    """Codes past 4 GiB."""
    M, N, K = FAR[case]
    print(case, flush=True)
    assert N * K // 2 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(M)
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda").random_(generator=g)
    scales = torch.rand((N, K // 128), device="cuda", generator=g) * 0.01
    zeros = torch.randint(0, 16, scales.shape, dtype=torch.uint8, device="cuda", generator=g)
    x = torch.randn((M, K), device="cuda", generator=g).to(torch.bfloat16)
    out = fp8.int4_linear(x, codes, scales, zeros)
    rows = [0, 1, N // 2, N - 17, N - 16, N - 1]
    tail_products(x, codes, scales, zeros, out, rows)


def test_int4_pack_and_quantization_of_large_weights():
    """Packed codes past 4 GiB: the rows there are the ones they are alone."""
    N, K = 33000, 2 ** 18 + 128
    assert N * K // 2 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(2)
    values = torch.empty((N, K), dtype=torch.uint8, device="cuda").random_(generator=g)
    codes = fp8.int4_pack(values)
    parts = [slice(0, 2), slice(N // 2, N // 2 + 2), slice(N - 2, N)]
    for rows in parts:
        assert np.array_equal(codes[rows].cpu().numpy(), step.int4_pack_ref(values[rows].cpu().numpy() & 15))
    del values, codes
    w = torch.empty((N, K), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    for group, symmetric in ((32, False), (128, True)):
        codes, scales, zeros = fp8.int4_quant_weight(w, group, symmetric)
        for rows in parts:
            c, s, z = step.int4_quant_ref(bits_of(w[rows]), group, symmetric)
            assert np.array_equal(codes[rows].cpu().numpy(), step.int4_pack_ref(c))
            assert np.array_equal(scales[rows].cpu().numpy().view(np.uint32), s.view(np.uint32))
            assert zeros is None if symmetric else np.array_equal(zeros[rows].cpu().numpy(), z)


def test_int4_rows_far_apart():
    rng, N, K = np.random.default_rng(9), 200, 256
    w = fp8.int4_quant_weight(bf16(rng.standard_normal((N, K))), 32)
    for M in (3, 9, 20, 70):
        ld = 2 ** 32 // M                               # the last rows' bytes past 2^32
        ld += 8 - ld % 8
        x = rows_apart(normal(rng, M, K), ld)
        store = torch.empty((M - 1) * ld + N, dtype=torch.bfloat16, device="cuda")
        out = fp8.int4_linear(x, *w, out=store.as_strided((M, N), (ld, 1)))
        assert same(out, fp8.int4_linear(x.contiguous(), *w))
        del x, store, out
        torch.cuda.empty_cache()


def test_int4_of_many_rows():
    """More than 2^32 results."""
    M, N, K = 40000, 110000, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda").random_(generator=g)
    scales = torch.rand((N, 1), device="cuda", generator=g)
    zeros = torch.randint(0, 16, scales.shape, dtype=torch.uint8, device="cuda", generator=g)
    x = torch.randn((M, K), device="cuda", generator=g).to(torch.bfloat16)
    out = fp8.int4_linear(x, codes, scales, zeros)
    rows = [0, N // 2, N - 1]
    for m in (0, M // 2, M - 4):
        tail_products(x[m:m + 4], codes, scales, zeros, out[m:m + 4], rows)


@pytest.mark.parametrize("T, V, ld", [(5, 9001, 2 ** 30 + 5), (1100, 4100000, None), (250, 18000000, None)])
def test_logprobs_past_32_bits(T, V, ld):
    g = torch.Generator(device="cuda").manual_seed(T)
    if ld is None:
        x = torch.randn((T, V), device="cuda", generator=g, dtype=torch.bfloat16)
    else:
        x = torch.empty((T - 1) * ld + V, device="cuda").as_strided((T, V), (ld, 1))
        x.normal_(generator=g)
    assert (T - 1) * x.stride(0) > 2 ** 32 or ld
    tokens = torch.randint(0, V, (T,), device="cuda", generator=g)
    tokens[-1] = V - 1
    got = [t[-2:].cpu().numpy() for t in fp8.token_logprobs(x, tokens, k=5)]
    want, tol = step.logprobs_ref(f64(x[-2:]), tokens[-2:].cpu().numpy(), 5, 1.0)
    for n, v in zip(("logprobs", "ranks", "entropy", "lse", "top", "ids"), got):
        if n in ("ranks", "ids"):
            assert np.array_equal(v, want[n]), n
        else:
            assert (np.abs(v.astype(np.float64) - want[n]) <= tol(want[n])).all(), n


def test_logprobs_of_rows_in_parts_and_in_one_launch():
    """A row's whole results do not depend on how many rows are with it."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((1100, 80000), device="cuda", generator=g, dtype=torch.bfloat16)
    tokens = torch.randint(0, 80000, (1100,), device="cuda", generator=g)
    for k in (0, 1, 20, 33, 64):
        assert fp8.logprobs_workspace_bytes(1100, 80000, k) == 0 < fp8.logprobs_workspace_bytes(7, 80000, k)
        a = fp8.token_logprobs(x, tokens, k=k)
        b = fp8.token_logprobs(x[:7], tokens[:7], k=k)
        assert torch.equal(a[1][:7], b[1]) and torch.equal(a[5][:7], b[5])
        for i in (0, 2, 3, 4):
            assert torch.allclose(a[i][:7], b[i], rtol=2.0 ** -18, atol=2.0 ** -18)
