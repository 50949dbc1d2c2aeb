"""fp8_qk_norm_rope_cache against the oracle (needs a gfx950 GPU).

Queries within half a bf16 step of the float64 result plus the tolerance of
the fp32 evaluation; key codes between the codes of the float64 result moved
down and up by that tolerance; value codes bit for bit those of the static
quantizer; everything not named left as it was."""

import numpy as np
import pytest
import torch

from oracle import attention, e4m3, kv_cache, quant
from workloads import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_w8a8_block_amd as fp8


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def normal(rng, *shape):
    return synth.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def inputs(seed, T, Hq, Hk, D, rot, page, nb, reach=500):
    rng = np.random.default_rng(seed)
    row = normal(rng, T, Hq + 2 * Hk, D)
    ang = np.arange(reach)[:, None] * (1e4 ** (-np.arange(rot // 2) / max(1, rot // 2)))[None]
    return dict(row=row, qw=normal(rng, D), kw=normal(rng, D),
                cs=np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32),
                pos=rng.integers(0, reach, T), slots=rng.permutation(nb * page)[:T].astype(np.int64),
                k0=rng.integers(0, 256, (nb, page, Hk, D), dtype=np.uint8),
                v0=rng.integers(0, 256, (nb, page, Hk, D), dtype=np.uint8))


def call(d, Hq, Hk, ks, vs, eps, inter, out, stride_heads=0):
    """The call on slices of one QKV row; returns (out bits, key cache, value cache)."""
    T, H, D = d["row"].shape
    wide = np.zeros((T, H + stride_heads, D), dtype=np.uint16)
    wide[:, :H] = d["row"]
    x = bf16(wide)
    kc, vc = (torch.from_numpy(d[n].copy()).cuda() for n in ("k0", "v0"))
    got = fp8.qk_norm_rope_cache(
        x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:H], bf16(d["qw"]), bf16(d["kw"]),
        torch.from_numpy(d["cs"]).cuda(), torch.from_numpy(d["pos"]).cuda(),
        torch.from_numpy(d["slots"]).cuda(), kc, vc, torch.tensor([ks], device="cuda"),
        torch.tensor([vs], device="cuda"), eps=eps, interleaved=inter, query_out=out)
    torch.cuda.synchronize()
    return bits_of(got), kc.cpu().numpy(), vc.cpu().numpy()


def check(d, Hq, Hk, ks, vs, eps, inter, got, kc, vc, out0):
    T, H, D = d["row"].shape
    x = quant.bf16_bits_to_f32(d["row"]).astype(np.float64)
    qw, kw = (quant.bf16_bits_to_f32(d[n]).astype(np.float64) for n in ("qw", "kw"))
    reach, rot = d["cs"].shape
    nb, page = d["k0"].shape[:2]
    live = (d["pos"] >= 0) & (d["pos"] < reach)
    pos = np.where(live, d["pos"], 0)
    cos, sin = (d["cs"][pos][:, s].astype(np.float64) for s in
                (slice(0, rot // 2), slice(rot // 2, rot)))
    z, tol = attention.norm_rope_ref(x[:, :Hq], qw, eps, cos, sin, inter)
    f = quant.bf16_bits_to_f32(got).astype(np.float64)
    off = np.abs(f - z)[live] - (np.abs(z) * 2.0 ** -8 + tol * 2)[live]
    assert (off <= 0).all(), off.max()
    assert np.array_equal(got[~live], out0[~live])
    # keys: codes are monotone in the value
    z, tol = attention.norm_rope_ref(x[:, Hq:Hq + Hk], kw, eps, cos, sin, inter)
    slots = np.where(live, d["slots"], -1)
    want_v = kv_cache.kv_write_ref(d["row"][:, Hq + Hk:], slots, d["v0"], vs)
    assert np.array_equal(vc, want_v)
    lo, hi = ((z + s * (tol + np.abs(z) * 2.0 ** -23)) / np.float64(np.float32(ks))
              for s in (-1, 1))
    lo, hi = (e4m3.decode(e4m3.encode(v.astype(np.float32))).astype(np.float64) for v in (lo, hi))
    lo, hi = np.minimum(lo, hi), np.maximum(lo, hi)
    flat, k0 = kc.reshape(nb * page, Hk, D), d["k0"].reshape(nb * page, Hk, D)
    touched = np.zeros(nb * page, dtype=bool)
    for t in range(T):
        s = int(slots[t])
        if 0 <= s < nb * page:
            touched[s] = True
            v = e4m3.decode(flat[s]).astype(np.float64)
            assert ((v >= lo[t]) & (v <= hi[t])).all(), t
    assert np.array_equal(flat[~touched], k0[~touched])


# T, Hq, Hk, D, rot, interleaved, page, extra heads in the row
CASES = {
    "one_token": (1, 32, 8, 128, 128, False, 16, 0),
    "neighbours": (3, 4, 2, 64, 64, True, 16, 0),
    "partial": (33, 16, 2, 256, 64, False, 16, 1),
    "partial_neighbours": (19, 6, 3, 128, 32, True, 7, 2),
    "no_rotation": (9, 2, 2, 64, 0, False, 16, 0),
    "odd_head": (21, 5, 5, 80, 48, False, 3, 0),
    "odd_head_neighbours": (21, 3, 1, 112, 112, True, 16, 0),
    "smallest_head": (50, 3, 1, 16, 16, False, 16, 0),
    "widest_head": (6, 2, 1, 512, 512, False, 16, 0),
    "many_tokens": (1500, 8, 2, 128, 128, False, 16, 3),
    "many_tokens_wide": (2111, 16, 2, 256, 64, True, 32, 0),
}


@pytest.mark.parametrize("case", list(CASES))
def test_against_oracle(case):
    T, Hq, Hk, D, rot, inter, page, extra = CASES[case]
    print(case, flush=True)
    d = inputs([T, D], T, Hq, Hk, D, rot, page, T // page + 3)
    if T > 8:
        d["slots"][[1, 4]] = [-1, d["k0"].shape[0] * page]          # not stored
        d["pos"][[3, 6]] = [-1, 500]                                # padding
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out0 = bits_of(out)
    got = call(d, Hq, Hk, np.float32(0.021), np.float32(0.5), 1e-6, inter, out, extra)
    check(d, Hq, Hk, np.float32(0.021), np.float32(0.5), 1e-6, inter, *got, out0)


def test_values_at_the_edges():
    """Zero heads, saturating keys, huge and tiny heads, NaN and infinity."""
    T, Hq, Hk, D = 7, 2, 2, 64
    d = inputs(3, T, Hq, Hk, D, 64, 16, 2)
    d["row"][0] = 0
    d["row"][1] = synth.f32_to_bf16_bits(np.float32(1e15))
    d["row"][2, ::2] = synth.f32_to_bf16_bits(np.float32(1e-15))
    d["row"][3, 1, 5] = 0x7fc0
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got, kc, vc = call(d, Hq, Hk, np.float32(1e-4), np.float32(1.0), 1e-6, False, out)
    f = quant.bf16_bits_to_f32(got)
    assert (f[0] == 0).all()
    assert np.isnan(f[3, 1]).all() and np.isfinite(f[3, 0]).all()
    keep = d["row"].copy()
    keep[3] = 0
    ok = np.array([0, 1, 2, 4, 5, 6])
    d2 = {**d, "row": keep}
    got2, kc2, vc2 = call(d2, Hq, Hk, np.float32(1e-4), np.float32(1.0), 1e-6, False, out)
    assert np.array_equal(got[ok], got2[ok])
    check(d2, Hq, Hk, np.float32(1e-4), np.float32(1.0), 1e-6, False, got2, kc2, vc2, got2)


def test_empty_cache_and_empty_step():
    d = inputs(4, 5, 2, 1, 64, 64, 16, 1)
    d["k0"], d["v0"] = d["k0"][:0], d["v0"][:0]
    out = torch.zeros((5, 2, 64), dtype=torch.bfloat16, device="cuda")
    got = call(d, 2, 1, np.float32(1), np.float32(1), 1e-6, False, out)[0]
    assert (got != 0).any()
    d = inputs(4, 0, 2, 1, 64, 64, 16, 1)
    call(d, 2, 1, np.float32(1), np.float32(1), 1e-6, False, None)


def test_refusals():
    d = inputs(5, 4, 2, 1, 64, 64, 16, 1)
    out = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    x = bf16(d["row"])
    kc, vc = (torch.from_numpy(d[n]).cuda() for n in ("k0", "v0"))
    one, w, cs = torch.ones(1, device="cuda"), bf16(d["qw"]), torch.from_numpy(d["cs"]).cuda()
    pos, slots = torch.from_numpy(d["pos"]).cuda(), torch.from_numpy(d["slots"]).cuda()

    def go(q=x[:, :2], k=x[:, 2:3], v=x[:, 3:], qw=w, table=cs, p=pos, key=kc, o=out, s=one):
        fp8.qk_norm_rope_cache(q, k, v, qw, w, table, p, slots, key, vc, s, one, query_out=o)

    go()
    for bad, err in ((dict(q=x[:, :2].float()), TypeError), (dict(v=x[:3, 3:]), ValueError),
                     (dict(qw=w[:32]), ValueError), (dict(table=cs[:, :24].contiguous()), ValueError),
                     (dict(table=cs[:, :32]), ValueError), (dict(p=pos.int()), TypeError),
                     (dict(key=kc[..., :32]), ValueError), (dict(o=out[:3]), ValueError),
                     (dict(o=x[:, :2]), ValueError), (dict(s=one.cpu()), ValueError),
                     (dict(key=vc), ValueError)):
        with pytest.raises(err):
            go(**bad)
