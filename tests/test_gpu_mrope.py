"""fp8_qk_norm_mrope_cache against the oracle (needs a gfx950 GPU): the angles of
each pair are picked by axis on the host, then held to the one-axis oracle."""

import numpy as np
import pytest
import torch

from oracle import attention, e4m3, kv_cache, quant, step
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


REACH = 300


def inputs(seed, T, Hq, Hk, D, rot, page, axes):
    rng = np.random.default_rng(seed)
    nb = T // page + 2
    ang = np.arange(REACH)[:, None] * (1e4 ** (-np.arange(rot // 2) / max(1, rot // 2)))[None]
    d = dict(row=normal(rng, T, Hq + 2 * Hk, D), qw=normal(rng, D), kw=normal(rng, D),
             cs=np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32),
             pos=rng.integers(0, REACH, (axes, T)), slots=rng.permutation(nb * page)[:T].astype(np.int64),
             k0=rng.integers(0, 256, (nb, page, Hk, D), dtype=np.uint8),
             v0=rng.integers(0, 256, (nb, page, Hk, D), dtype=np.uint8))
    d["pos"][:, ::3] = d["pos"][0, ::3]                  # text: one position on all axes
    return d


KS, VS = np.float32(0.021), np.float32(0.5)


def call(d, Hq, Hk, sections, in_turn, inter, out, gap=0):
    """gap: columns between the axes' rows of positions."""
    x, (A, T) = dev(d["row"]), d["pos"].shape
    kc, vc = (torch.from_numpy(d[n].copy()).cuda() for n in ("k0", "v0"))
    pos = torch.full((A, T + gap), -5, dtype=torch.int64, device="cuda")
    pos[:, :T] = torch.from_numpy(d["pos"]).cuda()
    got = fp8.qk_norm_mrope_cache(
        x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], dev(d["qw"]), dev(d["kw"]),
        torch.from_numpy(d["cs"]).cuda(), pos[:, :T], sections, torch.from_numpy(d["slots"]).cuda(), kc,
        vc, torch.tensor([KS], device="cuda"), torch.tensor([VS], device="cuda"), in_turn=in_turn,
        interleaved=inter, query_out=out)
    torch.cuda.synchronize()
    return bits_of(got), kc.cpu().numpy(), vc.cpu().numpy()


def check(d, Hq, Hk, sections, in_turn, inter, got, kc, vc, out0):
    T, _, D = d["row"].shape
    half = d["cs"].shape[1] // 2
    live = ((d["pos"] >= 0) & (d["pos"] < REACH)).all(0)
    axis = np.array(step.axes_ref(sections, in_turn), dtype=np.int64)
    pos = np.where(live, d["pos"], 0)[axis].T if half else np.zeros((T, 0), dtype=np.int64)
    cos = d["cs"][pos, np.arange(half)].astype(np.float64)
    sin = d["cs"][pos, half + np.arange(half)].astype(np.float64)
    x = quant.bf16_bits_to_f32(d["row"]).astype(np.float64)
    qw, kw = (quant.bf16_bits_to_f32(d[n]).astype(np.float64) for n in ("qw", "kw"))
    z, tol = attention.norm_rope_ref(x[:, :Hq], qw, 1e-6, cos, sin, inter)
    f = quant.bf16_bits_to_f32(got).astype(np.float64)
    assert (np.abs(f - z)[live] <= (np.abs(z) * 2.0 ** -8 + tol * 2)[live]).all()
    assert np.array_equal(got[~live], out0[~live])
    slots = np.where(live, d["slots"], -1)
    assert np.array_equal(vc, kv_cache.kv_write_ref(d["row"][:, Hq + Hk:], slots, d["v0"], VS))
    z, tol = attention.norm_rope_ref(x[:, Hq:Hq + Hk], kw, 1e-6, cos, sin, inter)
    lo, hi = ((z + s * (tol + np.abs(z) * 2.0 ** -23)) / np.float64(KS) for s in (-1, 1))
    lo, hi = (e4m3.decode(e4m3.encode(v.astype(np.float32))).astype(np.float64) for v in (lo, hi))
    flat, k0 = kc.reshape(-1, Hk, D), d["k0"].reshape(-1, Hk, D)
    touched = np.zeros(len(flat), dtype=bool)
    for t in range(T):
        if 0 <= slots[t] < len(flat):
            touched[slots[t]] = True
            v = e4m3.decode(flat[slots[t]]).astype(np.float64)
            assert ((v >= np.minimum(lo[t], hi[t])) & (v <= np.maximum(lo[t], hi[t]))).all(), t
    assert np.array_equal(flat[~touched], k0[~touched])


# T, Hq, Hk, D, rot, sections, in turn, neighbours paired, page
CASES = {
    "one_token": (1, 32, 8, 128, 128, (16, 24, 24), False, False, 16),
    "in_turn": (40, 4, 2, 128, 128, (24, 20, 20), True, False, 16),
    "uneven_sections": (33, 6, 3, 128, 96, (5, 20, 23), False, False, 7),
    "neighbours": (33, 4, 1, 64, 64, (11, 11, 10), False, True, 16),
    "neighbours_in_turn": (33, 4, 1, 80, 48, (10, 8, 6), True, True, 16),
    "two_axes": (21, 2, 2, 64, 32, (9, 7), True, False, 16),
    "four_axes": (21, 2, 2, 256, 256, (32, 32, 32, 32), True, False, 32),
    "four_sections": (21, 2, 2, 256, 128, (1, 62, 0, 1), False, False, 32),
    "an_empty_first": (12, 2, 1, 64, 64, (0, 16, 16), False, False, 16),
    "widest": (6, 2, 1, 512, 512, (100, 78, 78), True, False, 16),
    "no_rotation": (9, 2, 1, 64, 0, (0, 0), False, False, 16),
    "many_heads": (2300, 64, 2, 128, 64, (12, 10, 10), True, False, 16),
    "many": (1700, 8, 2, 128, 128, (24, 20, 20), True, False, 16),
}


@pytest.mark.parametrize("case", list(CASES))
def test_against_oracle(case):
    T, Hq, Hk, D, rot, sections, turn, inter, page = CASES[case]
    print(case, flush=True)
    d = inputs([T, D], T, Hq, Hk, D, rot, page, len(sections))
    if T > 8:
        d["slots"][[1, 4]] = [-1, d["k0"].shape[0] * page]
        d["pos"][-1, 5], d["pos"][0, 7], d["pos"][1, 2] = REACH, -1, 2 ** 40
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out0 = bits_of(out)
    got = call(d, Hq, Hk, sections, turn, inter, out, gap=3)
    check(d, Hq, Hk, sections, turn, inter, *got, out0)


@pytest.mark.parametrize("inter", [False, True])
def test_one_position_on_all_axes_is_the_plain_call(inter):
    T, Hq, Hk, D = 50, 4, 2, 128
    d = inputs(9, T, Hq, Hk, D, 128, 16, 3)
    d["pos"][:] = d["pos"][0]
    a = call(d, Hq, Hk, (24, 20, 20), True, inter, None)
    one = {**d, "pos": d["pos"][:1]}
    b = call(one, Hq, Hk, (64,), False, inter, None)
    x = dev(d["row"])
    kc, vc = (torch.from_numpy(d[n].copy()).cuda() for n in ("k0", "v0"))
    q = fp8.qk_norm_rope_cache(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], dev(d["qw"]), dev(d["kw"]),
                               torch.from_numpy(d["cs"]).cuda(), torch.from_numpy(d["pos"][0].copy()).cuda(),
                               torch.from_numpy(d["slots"]).cuda(), kc, vc,
                               torch.tensor([KS], device="cuda"), torch.tensor([VS], device="cuda"),
                               interleaved=inter)
    for g in (a, b):
        assert np.array_equal(g[0], bits_of(q)) and np.array_equal(g[1], kc.cpu().numpy())
        assert np.array_equal(g[2], vc.cpu().numpy())


@pytest.mark.parametrize("sections, inter", [((64,), False), ((24, 20, 20), False), ((24, 20, 20), True)])
def test_heads_whose_squares_leave_the_range(sections, inter):
    """Heads of values whose squares overflow or vanish in fp32, next to ordinary ones; without eps."""
    rng = np.random.default_rng(11)
    T, Hq, Hk, D = 24, 6, 3, 128
    d = inputs(12, T, Hq, Hk, D, D, 16, len(sections))
    x = rng.standard_normal((T, Hq + 2 * Hk, D))
    scale = 2.0 ** rng.choice([0, 55, 64, 90, 120, -38, -60, -80, -120, -128], x.shape[:2])
    scale[0] = 1.0
    x[1, :, 0], x[1, :, 1:] = 1.5, 0                            # one value alone
    d["row"] = synth.f32_to_bf16_bits((x * scale[..., None]).astype(np.float32))
    d["row"][2, :, 5] = synth.f32_to_bf16_bits(np.float32(3.0))
    row = dev(d["row"])
    kc, vc = (torch.from_numpy(d[n].copy()).cuda() for n in ("k0", "v0"))
    got = fp8.qk_norm_mrope_cache(
        row[:, :Hq], row[:, Hq:Hq + Hk], row[:, Hq + Hk:], dev(d["qw"]), dev(d["kw"]),
        torch.from_numpy(d["cs"]).cuda(), torch.from_numpy(d["pos"]).cuda(), sections,
        torch.from_numpy(d["slots"]).cuda(), kc, vc, torch.tensor([KS], device="cuda"),
        torch.tensor([VS], device="cuda"), eps=0.0, in_turn=len(sections) > 1, interleaved=inter)
    torch.cuda.synchronize()
    axis = np.array(step.axes_ref(sections, len(sections) > 1))
    half, pos = np.arange(D // 2), d["pos"][axis].T
    cos, sin = (d["cs"][pos, half + i].astype(np.float64) for i in (0, D // 2))
    x = quant.bf16_bits_to_f32(d["row"]).astype(np.float64)
    qw, kw = (quant.bf16_bits_to_f32(d[n]).astype(np.float64) for n in ("qw", "kw"))
    z, tol = attention.norm_rope_ref(x[:, :Hq], qw, 0.0, cos, sin, inter)
    f = quant.bf16_bits_to_f32(bits_of(got)).astype(np.float64)
    assert (np.abs(f - z) <= np.abs(z) * 2.0 ** -8 + tol * 2).all()
    z, tol = attention.norm_rope_ref(x[:, Hq:Hq + Hk], kw, 0.0, cos, sin, inter)
    lo, hi = ((z + s * (tol + np.abs(z) * 2.0 ** -23)) / np.float64(KS) for s in (-1, 1))
    lo, hi = (e4m3.decode(e4m3.encode(v.astype(np.float32))).astype(np.float64) for v in (lo, hi))
    v = e4m3.decode(kc.cpu().numpy().reshape(-1, Hk, D)[d["slots"]]).astype(np.float64)
    assert ((v >= lo) & (v <= hi)).all()


def test_refusals():
    d = inputs(5, 4, 2, 1, 64, 64, 16, 3)
    x, w, one = dev(d["row"]), dev(d["qw"]), torch.ones(1, device="cuda")
    kc, vc = (torch.from_numpy(d[n]).cuda() for n in ("k0", "v0"))
    cs, slots = torch.from_numpy(d["cs"]).cuda(), torch.from_numpy(d["slots"]).cuda()
    pos = torch.from_numpy(d["pos"]).cuda()

    def go(p=pos, sections=(12, 10, 10), turn=True, v=x[:, 3:], out=None):
        fp8.qk_norm_mrope_cache(x[:, :2], x[:, 2:3], v, w, w, cs, p, sections, slots, kc, vc, one, one,
                                in_turn=turn, query_out=out)

    go()
    for bad, err in ((dict(p=pos[0]), ValueError), (dict(p=pos[:2]), ValueError),
                     (dict(p=pos.int()), TypeError), (dict(p=pos[:, :3]), ValueError),
                     (dict(p=pos.cpu()), ValueError), (dict(sections=(12, 10, 9)), ValueError),
                     (dict(sections=(10, 11, 11)), ValueError), (dict(sections=(40, -4, -4)), ValueError),
                     (dict(v=x[:3, 3:]), ValueError), (dict(out=x[:, :2]), ValueError)):
        with pytest.raises(err):
            go(**bad)
