"""The C ABI of fp8w8a8_step.h on the host: the library exports what the header
declares, the binding's types are the header's, and every argument error is
reported before any device work (CPU only; only the host-only validation entry
points are called)."""

import ctypes
import math
import os
import re

import pytest
import torch

from fp8_w8a8_block_amd import _step

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8w8a8_step.h")

OK, NULL, SHAPE, STRIDE, ALIGN, BLOCK, SCHEME, WORKSPACE, ALIAS = 0, 1, 2, 3, 4, 5, 6, 7, 10
BLOCKS, TENSOR, ROWS = 0, 1, 2

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
    sigs, lib = signatures(), _step.lib()
    assert sorted(sigs) == sorted(_step._SIGS) and len(sigs) == 14
    for name, (ret, params) in sigs.items():
        assert hasattr(lib, name)
        b_ret, b_args = _step._SIGS[name]
        assert b_ret is c_of[ret], name
        want = [ctypes.c_void_p if t.endswith("*") else c_of[t] for t in params]
        assert b_args == want, name
    m = re.search(r"#define FP8_MAX_TOP (\d+)", open(HEADER).read())
    assert int(m.group(1)) == _step.MAX_TOP


def norm(x=A[0], ld_x=256, r=A[1], ld_r=256, ro=A[2], ld_ro=256, w=A[3], eps=1e-6, y=A[4], ld_y=256,
         q=A[5], ld_q=256, s=A[6], ld_s=2, mode=BLOCKS, scale=None, T=5, H=256):
    return _step.lib().fp8_validate_add_rms_norm_quant(x, ld_x, r, ld_r, ro, ld_ro, w, eps, y, ld_y, q,
                                                       ld_q, s, ld_s, mode, scale, T, H)


def test_norm_arguments():
    assert norm() == OK
    assert norm(T=0, x=None) == OK
    assert norm(ro=A[1]) == OK                                       # in place
    assert norm(r=None, ro=None, ld_r=0, ld_ro=0) == OK
    assert norm(y=None, ld_y=0) == OK and norm(q=None, ld_q=0, s=None, mode=7) == OK
    assert norm(mode=ROWS, ld_s=1) == OK and norm(mode=TENSOR, s=None, ld_s=0, scale=A[7]) == OK
    assert norm(H=65536, **{k: 65536 for k in ("ld_x", "ld_r", "ld_ro", "ld_y", "ld_q")}, ld_s=512) == OK
    assert norm(mode=3) == SCHEME
    for bad in (dict(T=-1), dict(T=1 << 31), dict(T=1 << 22), dict(H=0), dict(H=192), dict(H=65664),
                dict(eps=-1e-9), dict(eps=math.nan), dict(eps=math.inf)):
        assert norm(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(w=None), dict(r=None), dict(ro=None), dict(s=None),
                dict(y=None, q=None), dict(mode=TENSOR), dict(mode=ROWS, s=None)):
        assert norm(**bad) == NULL, bad
    for name in ("ld_x", "ld_r", "ld_ro", "ld_y", "ld_q"):
        assert norm(**{name: 248}) == STRIDE and norm(**{name: 1 << 60}) == STRIDE, name
        assert norm(**{name: 260}) == ALIGN, name
    assert norm(ld_s=1) == STRIDE and norm(mode=ROWS, ld_s=0) == STRIDE
    assert norm(ld_q=264) == ALIGN
    for name in ("x", "r", "ro", "w", "y", "q"):
        assert norm(**{name: A[8] + 8}) == ALIGN, name
    assert norm(s=A[8] + 2) == ALIGN and norm(mode=TENSOR, scale=A[8] + 2) == ALIGN
    assert norm(ro=A[1] + 16) == ALIAS                               # neither in place nor apart
    assert norm(ro=A[1], ld_ro=512) == ALIAS
    assert norm(ro=A[0]) == ALIAS and norm(y=A[0]) == ALIAS and norm(y=A[2]) == ALIAS
    assert norm(q=A[3] + 256) == ALIAS                               # the weight's second half
    assert norm(s=A[5] + 4 * 256 + 252) == ALIAS
    assert norm(mode=TENSOR, scale=A[5]) == ALIAS


def mrope(sections=(16, 8, 8), order=0, q=A[0], ld_q=512, k=A[1], ld_k=256, v=A[2], ld_v=256, qw=A[3],
          kw=A[4], eps=1e-6, cs=A[5], max_pos=100, rot=64, inter=0, pos=A[6], ld_pos=5, slots=A[7], T=5,
          Hq=4, Hk=2, D=128, out=A[8], ld_o=512, kc=A[9], vc=A[10], nb=10, bs=16, ks=A[11], vs=A[12],
          n=None):
    s = None if sections is None else (ctypes.c_int64 * max(1, len(sections)))(*sections)
    n = len(sections) if n is None else n
    return _step.lib().fp8_validate_qk_norm_mrope_cache(
        q, ld_q, k, ld_k, v, ld_v, qw, kw, eps, cs, max_pos, rot, inter, pos, ld_pos, n, s, order,
        slots, T, Hq, Hk, D, out, ld_o, kc, vc, nb, bs, ks, vs)


def test_mrope_arguments():
    assert mrope() == OK and mrope((32,)) == OK and mrope((8, 8, 8, 8), 1) == OK
    assert mrope((32, 0, 0)) == OK and mrope((0, 0, 32)) == OK and mrope(ld_pos=9) == OK
    assert mrope((0,), rot=0, cs=None) == OK and mrope(T=0, q=None) == OK
    assert mrope((12, 10, 10), 1) == OK                # 1 + 3 * 9 = 28, 2 + 3 * 9 = 29 below 32
    assert mrope(order=2) == SCHEME
    for bad in (dict(sections=(16, 8, 7)), dict(sections=(16, 24, -8)), dict(sections=(33,)),
                dict(sections=(8, 12, 12), order=1),   # 2 + 3 * 11 = 35
                dict(sections=(10, 11, 11), order=1),  # 2 + 3 * 10 = 32
                dict(sections=(32,), n=0), dict(sections=(8, 8, 8, 8, 0)), dict(rot=-16), dict(rot=80),
                dict(rot=24, sections=(12,)), dict(T=-1), dict(D=120), dict(eps=-1.0)):
        assert mrope(**bad) == SHAPE, bad
    assert mrope(sections=None, n=3) == NULL
    for name in ("q", "k", "v", "qw", "kw", "cs", "pos", "slots", "out", "kc", "vc", "ks", "vs"):
        assert mrope(**{name: None}) == NULL, name
    assert mrope(ld_pos=4) == STRIDE and mrope(ld_pos=1 << 60) == STRIDE and mrope((32,), ld_pos=0) == OK
    assert mrope(pos=A[13] + 4) == ALIGN
    assert mrope(pos=A[8] - 8 * 5 * 2) == ALIAS        # the third axis
    assert mrope(pos=A[8] - 8 * 5 * 3) == OK
    assert mrope(ld_q=504) == STRIDE and mrope(out=A[0]) == ALIAS


def test_int4_weight_arguments():
    def pack(v=A[0], ld=256, c=A[1], N=3, K=256):
        return _step.lib().fp8_validate_int4_pack(v, ld, c, N, K)

    assert pack() == OK and pack(N=0, v=None) == OK and pack(ld=264) == OK
    for bad in (dict(N=-1), dict(K=0), dict(K=192), dict(N=1 << 31)):
        assert pack(**bad) == SHAPE, bad
    assert pack(v=None) == NULL and pack(c=None) == NULL
    assert pack(ld=128) == STRIDE and pack(ld=260) == ALIGN and pack(v=A[2] + 4) == ALIGN
    assert pack(c=A[2] + 8) == ALIGN and pack(c=A[0] + 2 * 256 + 240) == ALIAS

    def quant(w=A[0], ld=256, c=A[1], s=A[2], z=A[3], N=3, K=256, g=64):
        return _step.lib().fp8_validate_int4_quant_weight(w, ld, c, s, z, N, K, g)

    assert quant() == OK and quant(z=None) == OK and quant(N=0, w=None) == OK
    for g in (0, 16, 96, 256, -32):
        assert quant(g=g) == BLOCK
    for bad in (dict(N=-1), dict(K=0), dict(K=320 + 32)):
        assert quant(**bad) == SHAPE, bad
    for name in ("w", "c", "s"):
        assert quant(**{name: None}) == NULL, name
    assert quant(ld=248) == STRIDE and quant(ld=260) == ALIGN and quant(s=A[4] + 2) == ALIGN
    assert quant(w=A[4] + 8) == ALIGN and quant(c=A[4] + 8) == ALIGN
    assert quant(z=A[2] + 47) == ALIAS and quant(z=A[2] + 48) == OK and quant(s=A[0]) == ALIAS


def int4(x=A[0], ld_x=256, c=A[1], s=A[2], z=A[3], g=64, out=A[4], ld_o=100, M=5, N=100, K=256,
         ws=None, n=0):
    return _step.lib().fp8_validate_int4_linear(x, ld_x, c, s, z, g, out, ld_o, M, N, K, ws, n)


def test_int4_linear_arguments():
    assert int4() == OK and int4(z=None) == OK and int4(M=0, x=None) == OK
    assert int4(N=1, ld_o=1) == OK and int4(out=A[4] + 2, ld_o=101) == OK
    for g in (0, 16, 256):
        assert int4(g=g) == BLOCK
    for bad in (dict(M=-1), dict(N=0), dict(N=-1), dict(K=0), dict(K=192), dict(M=1 << 31),
                dict(K=1 << 24, ld_x=1 << 24), dict(M=1 << 30, N=1 << 20, ld_o=1 << 20)):
        assert int4(**bad) == SHAPE, bad
    for name in ("x", "c", "s", "out"):
        assert int4(**{name: None}) == NULL, name
    assert int4(ld_x=248) == STRIDE and int4(ld_o=99) == STRIDE and int4(ld_x=1 << 60) == STRIDE
    assert int4(ld_x=260) == ALIGN and int4(out=A[4] + 1) == ALIGN
    for name in ("x", "c", "s"):
        assert int4(**{name: A[5] + 8}) == ALIGN, name
    assert int4(out=A[3] + 398) == ALIAS and int4(out=A[3] + 400) == OK
    assert int4(out=A[0]) == ALIAS and int4(out=A[2] + 1598) == ALIAS
    assert int4(ws=A[6], n=64) == OK and int4(ws=A[6] + 8, n=64) == WORKSPACE
    assert int4(ws=A[4] + 992, n=64) == ALIAS and int4(ws=A[0] - 16, n=32) == ALIAS
    assert int4(ws=A[0] - 32, n=32) == OK


def test_int4_workspace_sizes():
    def size(M, N, K):
        return _step.lib().fp8_int4_workspace_bytes(M, N, K)

    for bad in ((0, 256, 256), (-1, 256, 256), (5, 0, 256), (5, 256, 200), (5, 256, 1 << 24)):
        assert size(*bad) == 0
    assert size(1, 256, 4096) == 0 and size(4, 4096, 14336) == 0    # the waves of a workgroup share K
    assert size(16, 128000, 4096) == 0 and size(16, 256, 4096) == 0
    n = size(16, 4096, 14336)                                       # x would be read 256 times
    assert n > 0 and n % (16 * 4096 * 4) == 0 and n // (16 * 4096 * 4) <= 14
    assert size(64, 65536, 4096) == 0                               # tiles for every compute unit
    assert size(64, 256, 384) == 0                                  # less than 2 runs of 4 blocks
    n = size(64, 256, 4096)
    assert n > 0 and n // (64 * 256 * 4) <= 8


def probs(x=A[0], kind=0, ld=1000, tok=A[1], scale=1.0, T=5, V=1000, k=3, lp=A[2], r=A[3], e=A[4],
          lse=A[5], top=A[6], ids=A[7], ws=A[8], n=4096, need=4096):
    return _step.lib().fp8_validate_token_logprobs(x, kind, ld, tok, scale, T, V, k, lp, r, e, lse, top,
                                                   ids, ws, n, need)


def test_logprob_arguments():
    assert probs() == OK and probs(kind=1) == OK and probs(k=0, top=None, ids=None) == OK
    assert probs(T=0, x=None) == OK and probs(x=A[0] + 2, ld=1001) == OK and probs(ws=None, n=0, need=0) == OK
    assert probs(kind=2) == SCHEME
    for bad in (dict(T=-1), dict(V=0, ld=0, k=0), dict(k=-1), dict(k=65), dict(V=2, k=3), dict(V=1 << 31),
                dict(T=1 << 31), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
                dict(scale=math.nan), dict(T=1 << 24)):
        assert probs(**bad) == SHAPE, bad
    for name in ("x", "tok", "lp", "r", "e", "lse", "top", "ids"):
        assert probs(**{name: None}) == NULL, name
        assert probs(**{name: A[9] + 1}) == ALIGN, name
    assert probs(kind=1, x=A[9] + 2) == ALIGN and probs(tok=A[9] + 4) == ALIGN
    assert probs(ld=999) == STRIDE and probs(ld=1 << 60) == STRIDE
    assert probs(ws=None) == WORKSPACE and probs(n=4095) == WORKSPACE and probs(ws=A[8] + 8) == WORKSPACE
    assert probs(lp=A[0] + 2 * 4999) == ALIGN and probs(lp=A[0] + 2 * 4998) == ALIAS
    assert probs(r=A[2] + 16) == ALIAS and probs(ids=A[6] + 56) == ALIAS and probs(ws=A[7] - 4096 + 16) == ALIAS


def test_logprob_workspace_sizes():
    def size(T, V, k=1, kind=0):
        return _step.lib().fp8_logprobs_workspace_bytes(kind, T, V, k)

    assert size(0, 1000) == 0 and size(5, 0) == 0 and size(5, 1000, 65) == 0 and size(5, 1000, 1, 2) == 0
    assert size(4096, 128000) == 0                    # a workgroup per row
    assert size(1, 4000) == 0                         # little to share
    n = size(1, 128000)                               # parts of at least 2 sweeps of 64 segments
    assert 0 < n <= 16 * 16 + 4 * 2112
    assert size(4096, 1 << 20) > 0                    # more segments than LDS holds


def test_logprob_workspace_of_any_number_of_rows():
    """What a buffer for up to T rows needs is the size's largest value over them: 0 or growing
    from 256 rows on, so that of the first 255 and T."""
    def size(T, V, kind):
        return _step.lib().fp8_logprobs_workspace_bytes(kind, T, V, 1)

    for kind in (0, 1):
        for V in (1, 32000, 100003, 128000, 262145, 600000, 1 << 20, 5000000):
            few = max(size(T, V, kind) for T in range(1, 256))
            last = size(256, V, kind)
            for T in [*range(257, 700, 13), *range(700, 5000, 331), 65536]:
                n = size(T, V, kind)
                assert n == last == 0 or n > last
                last = n
            assert V < 262145 or few > 0


def test_binding_refuses_before_the_library():
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16)
    import fp8_w8a8_block_amd as fp8
    with pytest.raises(ValueError):
        fp8.add_rms_norm_quant(x, w)                  # host tensors
    with pytest.raises(ValueError):
        fp8.add_rms_norm_quant(x, w, scale_mode="channel")
    with pytest.raises(ValueError):
        fp8.int4_linear(x, x, x)
    with pytest.raises(ValueError):
        fp8.token_logprobs(x, w)
    with pytest.raises(TypeError):
        fp8.token_logprobs(None, w)


def test_whole_calls_refuse_what_is_no_gpu_tensor():
    from fp8_w8a8_block_amd import _attention
    import fp8_w8a8_block_amd as fp8
    fp8.lib()
    calls, gpu = _attention._tensor_args, torch.device("cuda", 0)      # a name; no GPU is needed here
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    for t in (x, None, 3):
        assert calls.int4_linear(0, t, t, t, None, t, None, gpu, 0) is None
        assert calls.add_rms_norm(0, t, None, None, t, 1e-6, t, None, None, 0, None, gpu, 0) is None
        assert calls.qk_norm_mrope_cache(0, *[t] * 5, 1e-6, t, 0, t, (1, 2), 0, *[t] * 6, gpu, 0) is None
        assert calls.token_logprobs(0, t, t, 1.0, 0, *[t] * 6, None, gpu, 0) is None
    for name, n in (("int4_linear", 9), ("add_rms_norm", 13), ("qk_norm_mrope_cache", 20),
                    ("token_logprobs", 14)):
        for wrong in (0, n - 1, n + 1):
            with pytest.raises(TypeError):
                getattr(calls, name)(*[None] * wrong)
    with pytest.raises(TypeError):
        calls.add_rms_norm(0, x, None, None, x, "eps", x, None, None, 0, None, gpu, 0)
    with pytest.raises(TypeError):
        calls.qk_norm_mrope_cache(0, *[x] * 5, 1e-6, x, 0, x, ("a",), 0, *[x] * 6, gpu, 0)
