"""The paged attention step as it is served: slot map, norm and rotation into the
cache, attention, one after the other over several steps -- eager, captured
and replayed, on other streams, two at once (needs a gfx950 GPU).

Each operator's output is held to the oracle on the inputs that the operator
before it left on the device, so an error names its operator and none hides
behind the roundings of another."""

import numpy as np
import pytest
import torch

from oracle import attention, quant
from workloads import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_w8a8_block_amd as fp8

EPS = 1e-6


def bf16(x):
    bits = synth.f32_to_bf16_bits(np.asarray(x, dtype=np.float32))
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def same(x, y):
    return torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


class Server:
    """Requests with their caches and all buffers of a step of T tokens."""

    def __init__(self, seed, B, T, Hq, Hk, D, page=16, width=12, far=0, window=0, sinks=0):
        self.rng = rng = np.random.default_rng(seed)
        self.B, self.T, self.Hq, self.Hk, self.D, self.page = B, T, Hq, Hk, D, page
        self.far, self.window, self.sinks = far, window, sinks
        shared = -(-far // page)
        nb = B * width + shared
        order = rng.permutation(nb).astype(np.int32)
        self.far_table, self.far_len = i32(order[:shared]), i32([far])
        self.free = i32(order[shared:])
        dev = "cuda"
        self.kc = torch.full((nb, page, Hk, D), 0x7f, dtype=torch.uint8, device=dev)
        self.vc = torch.full((nb, page, Hk, D), 0x7f, dtype=torch.uint8, device=dev)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        self.computed = torch.zeros(B, dtype=torch.int32, device=dev)
        self.new = torch.zeros(B, dtype=torch.int32, device=dev)
        self.qkv = torch.empty((T, Hq + 2 * Hk, D), dtype=torch.bfloat16, device=dev)
        self.slots = torch.empty(T, dtype=torch.int64, device=dev)
        self.positions = torch.empty(T, dtype=torch.int64, device=dev)
        self.offsets = torch.empty(B + 1, dtype=torch.int32, device=dev)
        self.lens = torch.empty(B, dtype=torch.int32, device=dev)
        self.taken = torch.empty(1, dtype=torch.int32, device=dev)
        self.q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
        self.out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
        self.lse = torch.full((T, Hq), 7.0, device=dev)
        self.qw, self.kw = bf16(rng.uniform(0.5, 1.5, D)), bf16(rng.uniform(0.5, 1.5, D))
        ang = np.arange(4096)[:, None] * (1e4 ** (-np.arange(D // 2) / (D // 2)))[None]
        self.cs = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)
                                   .astype(np.float32)).cuda()
        self.ks, self.vs = torch.tensor([0.0625], device=dev), torch.tensor([0.03125], device=dev)
        self.ws = torch.empty(fp8.attention_workspace_bytes(T, B, Hq, Hk, D, far > 0),
                              dtype=torch.uint8, device=dev)
        if far:                                    # the prefix's tokens, by the same operators
            x = bf16(rng.standard_normal((far, Hq + 2 * Hk, D)))
            taken = i32([0])
            slots, pos, *_ = fp8.kv_slot_map(i32([0]), i32([far]), self.far_table.clone()[None],
                                             self.far_table, page, far, blocks_taken=taken)
            self.store(x, pos, slots)
            assert int(taken) == shared

    def store(self, x, positions, slots, q=None):
        Hq, Hk = self.Hq, self.Hk
        return fp8.qk_norm_rope_cache(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], self.qw, self.kw,
                                      self.cs, positions, slots, self.kc, self.vc, self.ks, self.vs,
                                      eps=EPS, query_out=q)

    def feed(self, new):
        """This step's lengths and rows, into the buffers that a step reads."""
        self.new.copy_(i32(new))
        self.qkv.copy_(bf16(self.rng.standard_normal(tuple(self.qkv.shape))))

    def step(self):
        """The operators of a step; every length stays on the device."""
        fp8.kv_slot_map(self.computed, self.new, self.table, self.free, self.page, self.T,
                        self.slots, self.positions, self.offsets, self.lens, self.taken)
        pos = self.positions
        if self.far:
            pos = torch.where(pos >= 0, pos + self.far, pos)
        self.store(self.qkv, pos, self.slots, self.q)
        batch = (self.table, self.lens, self.offsets, self.ks, self.vs)
        if self.far:
            fp8.prefix_attention(self.q, self.kc, self.vc, self.far_table, self.far_len, *batch,
                                 out=self.out, lse=self.lse, workspace=self.ws)
        else:
            fp8.paged_attention(self.q, self.kc, self.vc, *batch, window=self.window,
                                sinks=self.sinks, out=self.out, lse=self.lse, workspace=self.ws)

    def advance(self):
        """Takes the step's blocks off the free list and its tokens into the lengths."""
        self.free = self.free[int(self.taken):].clone()
        self.computed.copy_(self.lens)

    STATE = ("kc", "vc", "table", "computed", "new", "qkv", "q", "out", "lse", "slots", "positions",
             "offsets", "lens", "taken")

    def state(self):
        return {n: getattr(self, n).clone() for n in self.STATE}

    def restore(self, state):
        for n, t in state.items():
            getattr(self, n).copy_(t)

    def check(self, before):
        """What step() left against the oracle; before: state() in front of it."""
        host = {n: t.cpu().numpy() for n, t in before.items()
                if t.dtype in (torch.int32, torch.int64, torch.uint8)}
        table, slots, pos, offs, lens, taken = attention.slot_map_ref(
            host["computed"], host["new"], host["table"], self.free.cpu().numpy(), self.page, self.T)
        for got, want in ((self.table, table), (self.slots, slots), (self.positions, pos),
                          (self.offsets, offs), (self.lens, lens)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert int(self.taken) == taken
        live = pos >= 0
        Hq, Hk, D = self.Hq, self.Hk, self.D
        # queries; padded rows as they were
        cs = self.cs.cpu().numpy().astype(np.float64)[np.where(live, pos + self.far, 0)]
        z, tol = attention.norm_rope_ref(f64(self.qkv)[:, :Hq], f64(self.qw), EPS,
                                         cs[:, :D // 2], cs[:, D // 2:], False)
        off = np.abs(f64(self.q) - z)[live] - (np.abs(z) * 2.0 ** -8 + tol * 2)[live]
        assert off.size == 0 or (off <= 0).all(), off.max()
        pad = torch.from_numpy(~live).cuda()
        assert same(self.q[pad], before["q"][pad]) and same(self.out[pad], before["out"][pad])
        assert same(self.lse[pad], before["lse"][pad])
        # values as the plain cache write stores them
        kc, vc = before["kc"].clone(), before["vc"].clone()
        x = self.qkv
        fp8.kv_cache_write(x[:, Hq:Hq + Hk].contiguous(), x[:, Hq + Hk:].contiguous(), self.slots,
                           kc, vc, self.ks, self.vs)
        assert same(vc, self.vc)
        untouched = torch.ones(kc.shape[0] * self.page, dtype=torch.bool, device="cuda")
        untouched[self.slots[self.slots >= 0]] = False
        assert same(self.kc.flatten(0, 1)[untouched], before["kc"].flatten(0, 1)[untouched])
        # attention, on what the device holds
        far = (self.far_table.cpu().numpy(), self.far) if self.far else (None, 0)
        out, lse, tol, tol_lse, covered = attention.attention_ref(
            f64(self.q), self.kc.cpu().numpy(), self.vc.cpu().numpy(), table, lens, offs,
            D ** -0.5, float(self.ks), float(self.vs), self.window, self.sinks, *far)
        assert np.array_equal(covered, live)
        got = f64(self.out)
        assert not np.isnan(got[live]).any()
        assert (np.abs(got - out)[live] <= tol[live]).all()
        got = self.lse.cpu().numpy().astype(np.float64)[live]
        lse, tol_lse = lse[live], tol_lse[live]
        some = np.isfinite(lse)                    # -inf: rows that see no key
        assert np.array_equal(np.isneginf(got), ~some)
        assert (np.abs(got[some] - lse[some]) <= tol_lse[some]).all()


SERVERS = {
    "paged": dict(B=5, T=96, Hq=8, Hk=2, D=128),
    "window": dict(B=5, T=96, Hq=8, Hk=1, D=64, window=24, sinks=2, page=8, width=24),
    "wide_heads": dict(B=5, T=96, Hq=4, Hk=2, D=256),
    "large_tiles": dict(B=2, T=330, Hq=8, Hk=2, D=128, width=40),
    "prefix": dict(B=5, T=96, Hq=8, Hk=2, D=64, far=83),
    "prefix_large_tiles": dict(B=5, T=400, Hq=8, Hk=2, D=128, far=200, width=40),
}
# new tokens of each request in turn: prompts, single tokens, a mixture, a step of none
STEPS = [[40, 1, 33, 0, 17], [1, 1, 1, 1, 1], [1, 0, 50, 20, 1], [0, 0, 0, 0, 0], [1, 1, 1, 0, 1]]


def steps_of(s):
    for i, new in enumerate(STEPS):
        new = [n * s.T // 96 if n > 1 else n for n in new][:s.B]
        yield i, new


@pytest.mark.parametrize("name", list(SERVERS))
def test_steps(name):
    s = Server(1, **SERVERS[name])
    for _, new in steps_of(s):
        s.feed(new)
        before = s.state()
        s.step()
        torch.cuda.synchronize()
        s.check(before)
        s.advance()


@pytest.mark.parametrize("name", list(SERVERS))
def test_captured_steps(name):
    """One captured step replayed over changing lengths, each replay against an
    eager step from the same state, with eager work between the replays."""
    s = Server(2, **SERVERS[name])
    s.feed([0] * s.B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()                                   # a step without tokens, to load the kernels
    torch.cuda.current_stream().wait_stream(side)
    free = s.free.clone()                          # the graph reads this buffer
    s.free = free
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for i, new in steps_of(s):
        s.feed(new)
        before = s.state()
        graph.replay()
        torch.cuda.synchronize()
        replayed = s.state()
        s.restore(before)
        s.ws.fill_(0xff)                           # what it held is of no account
        s.step()
        torch.cuda.synchronize()
        for n, t in s.state().items():
            assert same(t, replayed[n]), (i, n)
        s.check(before)
        torch.randn(1000, device="cuda").sum().item()
        s.computed.copy_(s.lens)                   # blocks taken go to the list's end
        free.copy_(torch.roll(free, -int(s.taken)))


def test_graphs_that_share_a_workspace():
    """Two captured graphs, one workspace, replayed in turn."""
    a, b = Server(3, **SERVERS["paged"]), Server(4, **SERVERS["prefix"])
    n = max(a.ws.numel(), b.ws.numel())
    a.ws = b.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, want = [], []
    for s in (a, b):
        s.feed([9, 1, 40, 0, 1])
        start = s.state()
        s.step()
        torch.cuda.synchronize()
        want.append(s.state())
        s.restore(start)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step()
        graphs.append((s, g, start))
    for _ in range(4):
        for (s, g, start), w in zip(graphs, want):
            s.restore(start)
            g.replay()
            torch.cuda.synchronize()
            for n, t in s.state().items():
                assert same(t, w[n]), n


@pytest.mark.parametrize("names", [("paged", "prefix"), ("large_tiles", "prefix_large_tiles")])
def test_two_streams_at_once(names):
    """Steps of two servers on streams of their own, against the same steps alone."""
    servers = [Server(5 + i, **SERVERS[n]) for i, n in enumerate(names)]
    want, start = [], []
    for s in servers:
        s.feed([n * s.T // 96 for n in [30, 1, 40, 0, 20]][:s.B])
        start.append(s.state())
        s.step()
        torch.cuda.synchronize()
        want.append(s.state())
        s.restore(start[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in servers]
    for _ in range(8):
        for s, st, x in zip(servers, streams, start):
            with torch.cuda.stream(st):
                s.restore(x)
                s.step()
    torch.cuda.synchronize()
    for s, w in zip(servers, want):
        for n, t in s.state().items():
            assert same(t, w[n]), n


def test_free_blocks_run_out():
    """Tokens without a block are not stored and not seen."""
    s = Server(7, **SERVERS["paged"])
    s.free = s.free[:4].clone()
    s.feed([40, 1, 33, 0, 17])
    before = s.state()
    s.step()
    torch.cuda.synchronize()
    assert int(s.taken) == 9
    s.check(before)
