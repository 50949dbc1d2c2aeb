"""The paged attention step's C ABI on the host: the library exports what
fp8w8a8_attention.h declares, the binding's types are the header's, and every
argument error is reported before any device work (CPU only; only the
host-only validation entry points are called)."""

import ctypes
import math
import os
import re

import pytest

from fp8_w8a8_block_amd import _attention

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8w8a8_attention.h")

OK, NULL, SHAPE, STRIDE, ALIGN, WORKSPACE, ALIAS = 0, 1, 2, 3, 4, 7, 10

# fake, well-aligned addresses 2^40 apart: validation never dereferences
A = [(i + 1) << 40 for i in range(20)]


def signatures():
    text = re.sub(r"/\*.*?\*/|//[^\n]*", "", open(HEADER).read(), flags=re.S)
    got = {}
    for ret, name, params in re.findall(
            r"^\s*([A-Za-z_][A-Za-z0-9_]*)\s+(fp8_[a-z0-9_]+)\s*\(([^)]*)\)\s*;", text, flags=re.M):
        types = []
        for prm in params.split(","):
            m = re.fullmatch(r"([A-Za-z_][A-Za-z0-9_]*)\s*(\**)\s*\w+",
                             " ".join(prm.replace("const", " ").split()))
            assert m, (name, prm)
            types.append(m.group(1) + m.group(2))
        got[name] = (ret, types)
    return got


def test_exports_and_argument_types():
    c_of = {"int64_t": ctypes.c_int64, "int": ctypes.c_int, "size_t": ctypes.c_size_t,
            "float": ctypes.c_float, "fp8_status": ctypes.c_int}
    sigs, lib = signatures(), _attention.lib()
    assert sorted(sigs) == sorted(_attention._SIGS) and len(sigs) == 8
    for name, (ret, params) in sigs.items():
        assert hasattr(lib, name)
        b_ret, b_args = _attention._SIGS[name]
        assert b_ret is c_of[ret], name
        want = [ctypes.c_void_p if t.endswith("*") else c_of[t] for t in params]
        assert b_args == want, name


def slot_map(computed=A[0], new=A[1], B=4, bs=16, table=A[2], ld=8, width=8, free=A[3], nfree=9,
             slots=A[4], pos=A[5], T=50, offs=A[6], lens=A[7], taken=A[8]):
    return _attention.lib().fp8_validate_kv_slot_map(computed, new, B, bs, table, ld, width, free,
                                                     nfree, slots, pos, T, offs, lens, taken)


def test_slot_map_arguments():
    assert slot_map() == OK
    assert slot_map(B=0, computed=None, new=None, lens=None, table=None) == OK
    assert slot_map(T=0, slots=None, pos=None) == OK
    assert slot_map(nfree=0, free=None) == OK
    assert slot_map(width=0, ld=0, table=None) == OK
    for bad in (dict(B=-1), dict(T=-1), dict(bs=0), dict(bs=-4), dict(nfree=-1), dict(width=-1),
                dict(T=1 << 31), dict(B=1 << 31), dict(bs=1 << 31)):
        assert slot_map(**bad) == SHAPE, bad
    for name in ("computed", "new", "table", "free", "slots", "pos", "offs", "lens", "taken"):
        assert slot_map(**{name: None}) == NULL, name
        assert slot_map(**{name: A[9] + 2}) == ALIGN, name
    assert slot_map(slots=A[4] + 4) == ALIGN
    assert slot_map(ld=7) == STRIDE
    assert slot_map(ld=1 << 60) == STRIDE
    assert slot_map(slots=A[5]) == ALIAS
    assert slot_map(lens=A[0]) == ALIAS
    assert slot_map(free=A[2] + 4 * 31) == ALIAS          # the table's last entry
    assert slot_map(free=A[2] + 4 * 32) == OK
    assert slot_map(offs=A[1] - 4 * 4) == ALIAS           # B + 1 offsets


def rope(q=A[0], ld_q=512, k=A[1], ld_k=256, v=A[2], ld_v=256, qw=A[3], kw=A[4], eps=1e-6, cs=A[5],
         max_pos=100, rot=64, inter=0, pos=A[6], slots=A[7], T=5, Hq=4, Hk=2, D=128, out=A[8],
         ld_o=512, kc=A[9], vc=A[10], nb=10, bs=16, ks=A[11], vs=A[12]):
    return _attention.lib().fp8_validate_qk_norm_rope_cache(
        q, ld_q, k, ld_k, v, ld_v, qw, kw, eps, cs, max_pos, rot, inter, pos, slots, T, Hq, Hk, D,
        out, ld_o, kc, vc, nb, bs, ks, vs)


def test_norm_rope_arguments():
    assert rope() == OK
    assert rope(T=0, q=None) == OK
    assert rope(rot=0, cs=None) == OK
    assert rope(nb=0, kc=None, vc=None) == OK
    for bad in (dict(T=-1), dict(Hq=0), dict(Hk=0), dict(D=120, rot=16), dict(D=528), dict(rot=24),
                dict(rot=-16), dict(rot=144), dict(max_pos=-1), dict(eps=-1.0), dict(eps=math.nan),
                dict(eps=math.inf), dict(bs=0), dict(nb=-1), dict(T=1 << 31),
                dict(T=1 << 30, Hq=32, ld_q=4096, ld_o=4096)):
        assert rope(**bad) == SHAPE, bad
    for name in ("q", "k", "v", "qw", "kw", "cs", "pos", "slots", "out", "kc", "vc", "ks", "vs"):
        assert rope(**{name: None}) == NULL, name
    for name in ("q", "k", "v", "qw", "kw", "cs", "out", "kc", "vc"):
        assert rope(**{name: A[13] + 8}) == ALIGN, name
    assert rope(pos=A[13] + 4) == ALIGN
    for name in ("ld_q", "ld_o"):
        assert rope(**{name: 504}) == STRIDE and rope(**{name: 516}) == ALIGN
        assert rope(**{name: 1 << 60}) == STRIDE
    assert rope(ld_k=248) == STRIDE and rope(ld_v=260) == ALIGN
    assert rope(out=A[0]) == ALIAS
    assert rope(k=A[0] + 1024, v=A[0] + 1536, ld_q=1024, ld_k=1024, ld_v=1024) == OK   # one QKV row
    assert rope(vc=A[9] + 16 * 10 * 256 - 16) == ALIAS
    assert rope(cs=A[8] + 16) == ALIAS


def attn(q=A[0], ld_q=512, kc=A[1], vc=A[2], nb=10, bs=16, pt=None, pw=0, pl=None, table=A[3],
         ld=8, width=8, lens=A[4], offs=A[5], B=3, ks=A[6], vs=A[7], scale=0.1, window=0, sinks=0,
         out=A[8], ld_o=512, lse=A[9], T=5, Hq=4, Hk=2, D=128, ws=A[10], ws_bytes=4096, need=4096):
    return _attention.lib().fp8_validate_attention(
        q, ld_q, kc, vc, nb, bs, pt, pw, pl, table, ld, width, lens, offs, B, ks, vs, scale, window,
        sinks, out, ld_o, lse, T, Hq, Hk, D, ws, ws_bytes, need)


def test_attention_arguments():
    assert attn() == OK
    assert attn(lse=None) == OK
    assert attn(T=0, q=None) == OK and attn(B=0, lens=None) == OK
    assert attn(nb=0, kc=None, vc=None) == OK
    assert attn(width=0, ld=0, table=None) == OK
    assert attn(pt=A[11], pw=3, pl=A[12]) == OK
    for D in (64, 256):
        assert attn(D=D, ld_q=1024, ld_o=1024) == OK
    for bad in (dict(D=32), dict(D=96), dict(D=512, ld_q=2048, ld_o=2048), dict(Hq=5), dict(Hq=0),
                dict(Hk=0), dict(T=-1), dict(B=-1), dict(bs=0), dict(nb=-1), dict(width=-1),
                dict(window=-1), dict(sinks=-1), dict(window=1 << 31), dict(scale=math.nan),
                dict(scale=math.inf), dict(nb=1 << 27), dict(T=1 << 29)):
        assert attn(**bad) == SHAPE, bad
    for name in ("q", "kc", "vc", "table", "lens", "offs", "ks", "vs", "out"):
        assert attn(**{name: None}) == NULL, name
    assert attn(pt=A[11], pw=3) == NULL and attn(pw=3, pl=A[11]) == NULL and attn(pw=3) == NULL
    assert attn(pl=A[11]) == OK                          # a prefix of no blocks
    for name in ("q", "kc", "vc", "out"):
        assert attn(**{name: A[13] + 8}) == ALIGN, name
    for name in ("table", "lens", "offs", "ks", "vs", "lse"):
        assert attn(**{name: A[13] + 2}) == ALIGN, name
    assert attn(ld_q=504) == STRIDE and attn(ld_o=516) == ALIGN and attn(ld=7) == STRIDE
    assert attn(ws=None) == WORKSPACE and attn(ws_bytes=4095) == WORKSPACE
    assert attn(ws=A[10] + 8, ws_bytes=1 << 20) == WORKSPACE
    assert attn(ws=None, ws_bytes=0, need=0) == OK
    assert attn(out=A[0]) == ALIAS and attn(lse=A[8]) == ALIAS
    assert attn(ws=A[8] - 4080) == ALIAS and attn(ws=A[4]) == ALIAS
    assert attn(pt=A[8], pw=3, pl=A[12]) == ALIAS


def test_workspace_of_an_empty_call():
    lib = _attention.lib()
    assert lib.fp8_attention_workspace_bytes(0, 0, 4, 8, 2, 128) == 0
    assert lib.fp8_attention_workspace_bytes(0, 4, 4, 8, 3, 128) == 0
    assert lib.fp8_attention_workspace_bytes(1, 4, 4, 8, 2, 96) == 0
    assert lib.fp8_prefix_attention(A[0], 512, A[1], A[2], 10, 16, A[12], 4, None, A[3], 8, 8, A[4],
                                    A[5], 3, A[6], A[7], 0.1, A[8], 512, None, 5, 4, 2, 128, A[10],
                                    1 << 30, None) == NULL


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        _attention.kv_slot_map(i, i, torch.zeros((4, 2), dtype=torch.int32), i, 16, 4)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((2, 16, 2, 64), dtype=torch.uint8)
    with pytest.raises(ValueError):
        _attention.paged_attention(x, c, c, i.view(2, 2), i[:2], i[:3], torch.ones(1),
                                   torch.ones(1))
    with pytest.raises(ValueError):
        _attention.qk_norm_rope_cache(x, x, x, x[0, 0], x[0, 0], torch.zeros((4, 64)), i[:3], i[:3],
                                      c, c, torch.ones(1), torch.ones(1))
    with pytest.raises(TypeError):
        _attention.prefix_attention(x, c, c, None, None, i.view(2, 2), i[:2], i[:3], torch.ones(1),
                                    torch.ones(1))
