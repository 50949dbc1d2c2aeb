"""ctypes binding of what a serving step runs around the linears and the paged
attention (include/fp8w8a8_step.h): argument marshalling only, with the
conventions of _lib and _attention.

No call synchronizes or needs a value on the host, so all of them can be
captured in a graph with the buffers that they are given.

Calls with arguments as they should be are made whole by _tensor_args
(csrc/tensor_args.cpp); the checks written out here say what is wrong with the
others.
"""

import ctypes
import functools

import torch

from . import _attention, _lib
from ._attention import (_caches, _call, _device_of, _f32, _heads, _matrix, _on, _raw_stream, _scale,
                         _vector)
from ._lib import SCALE_BLOCK, SCALE_ROW, SCALE_TENSOR, _check, _i64, _int, _mode, _sz, _vp, _workspace

LOGITS_BF16 = 0
LOGITS_F32 = 1
MAX_TOP = 64

_NORM = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _f32, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64,
         _i64]
_MROPE = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _f32, _vp, _i64, _i64, _int, _vp, _i64, _i64, _vp,
          _int, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp]
_PACK = [_vp, _i64, _vp, _i64, _i64]
_QUANT = [_vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64]
_INT4 = [_vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _sz]
_PROBS = [_vp, _int, _i64, _vp, _f32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz]

_SIGS = {
    "fp8_add_rms_norm_quant": (_int, _NORM + [_vp]),
    "fp8_validate_add_rms_norm_quant": (_int, _NORM),
    "fp8_qk_norm_mrope_cache": (_int, _MROPE + [_vp]),
    "fp8_validate_qk_norm_mrope_cache": (_int, _MROPE),
    "fp8_int4_pack": (_int, _PACK + [_vp]),
    "fp8_validate_int4_pack": (_int, _PACK),
    "fp8_int4_quant_weight": (_int, _QUANT + [_vp]),
    "fp8_validate_int4_quant_weight": (_int, _QUANT),
    "fp8_int4_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8_int4_linear": (_int, _INT4 + [_vp]),
    "fp8_validate_int4_linear": (_int, _INT4),
    "fp8_logprobs_workspace_bytes": (_sz, [_int, _i64, _i64, _i64]),
    "fp8_token_logprobs": (_int, _PROBS + [_vp]),
    "fp8_validate_token_logprobs": (_int, _PROBS + [_sz]),
}

_bound = None


def lib():
    """The loaded shared library with this header's argument types set, too."""
    global _bound
    if _bound is None:
        l = _lib.lib()
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _bound = l
    return _bound


@functools.lru_cache(maxsize=None)
def _address(name):
    """Address of a function of the library."""
    return ctypes.cast(getattr(lib(), name), _vp).value


def _stream_here(device):
    """The stream to call on if this GPU is the current device, else None."""
    if device.type == "cuda" and torch._C._cuda_getDevice() == device.index:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return None


def _rows(t, name, dtype, device, shape=None):
    """A 2-D device tensor with unit column stride -> (pointer, rows, columns, ld)."""
    got = _attention._tensor_args.rows(t, dtype, device)
    if got is None:
        _on(t, name, dtype, device)
        raise ValueError(f"{name} must be 2-D with unit column stride")
    if shape is not None and got[1:3] != shape:
        raise ValueError(f"{name} must have shape {shape}, got {got[1:3]}")
    return got


def _norm(x, weight, residual, eps, mode, scale, out, q, scales, residual_out):
    """Both norms; mode None: no codes."""
    dev = _device_of(x, "x")
    stream = _stream_here(dev)
    if stream is not None and x.dim() == 2 and (mode == SCALE_TENSOR) == (scale is not None) and \
            (residual is not None or residual_out is None) and \
            not (mode == SCALE_TENSOR and scales is not None):
        if mode is not None:
            T, H = x.shape
            if q is None:
                q = torch.empty((T, H), dtype=torch.uint8, device=dev)
            if scales is None and mode != SCALE_TENSOR:
                scales = torch.empty((T, H // 128) if mode == SCALE_BLOCK else (T,),
                                     dtype=torch.float32, device=dev)
        st = _attention._tensor_args.add_rms_norm(
            _address("fp8_add_rms_norm_quant"), x, residual,
            residual if residual_out is None else residual_out, weight, eps, out, q, scales,
            0 if mode is None else mode, scale, dev, stream)
        if st is not None:
            if st:
                _check(st)
            return q, scale if mode == SCALE_TENSOR else scales
    xp, T, H, ld_x = _rows(x, "x", torch.bfloat16, dev)
    rp, ld_r, rop, ld_ro = None, 0, None, 0
    if residual is not None:
        rp, _, _, ld_r = _rows(residual, "residual", torch.bfloat16, dev, (T, H))
        rop, ld_ro = rp, ld_r
        if residual_out is not None and residual_out is not residual:
            rop, _, _, ld_ro = _rows(residual_out, "residual_out", torch.bfloat16, dev, (T, H))
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    yp, ld_y, qp, ld_q, sp, ld_s, given = None, 0, None, 0, None, 0, None
    if out is not None:
        yp, _, _, ld_y = _rows(out, "out", torch.bfloat16, dev, (T, H))
    if mode is not None:
        if q is None:
            q = torch.empty((T, H), dtype=torch.uint8, device=dev)
        qp, _, _, ld_q = _rows(q, "q", torch.uint8, dev, (T, H))
        if mode == SCALE_TENSOR:
            if scale is None or scales is not None:
                raise ValueError("a per-tensor scale is calibrated: pass scale, not scales")
            given, scales = _scale(scale, "scale", dev), scale
        else:
            if scale is not None:
                raise ValueError("scale is for scale_mode 'tensor'")
            if scales is None:
                scales = torch.empty((T, H // 128) if mode == SCALE_BLOCK else (T,),
                                     dtype=torch.float32, device=dev)
            if mode == SCALE_BLOCK:
                sp, _, _, ld_s = _rows(scales, "scales", torch.float32, dev, (T, H // 128))
            else:
                _on(scales, "scales", torch.float32, dev)
                if tuple(scales.shape) != (T,):
                    raise ValueError(f"scales must have shape {(T,)}")
                sp, ld_s = scales.data_ptr(), scales.stride(0) if T > 1 else 1
    args = (xp, ld_x, rp, ld_r, rop, ld_ro, _vector(weight, "weight", torch.bfloat16, dev, H),
            float(eps), yp, ld_y, qp, ld_q, sp, ld_s, 0 if mode is None else mode, given, T, H)
    _check(_call(dev, lambda: lib().fp8_add_rms_norm_quant(*args, _raw_stream(dev))))
    return q, scales


def add_rms_norm_quant(x, weight, residual=None, eps=1e-6, scale_mode="block", scale=None, out=None,
                       q=None, scales=None, residual_out=None):
    """The residual's addition, RMS norm and FP8 quantization of bf16 x [T, H] in one
    pass -> (codes uint8 [T, H], scales), as block_gemm takes them.

    residual bf16 [T, H] becomes bf16(x + residual), in place or in
    residual_out, and is what is normalized; without one x is.  scale_mode
    "block" gives scales [T, H/128], "row" [T]; "tensor" takes a calibrated
    one in `scale` (1-element float32) and returns it.  `out` gets the norm in
    bf16, too."""
    mode = _mode(scale_mode)
    if mode not in (SCALE_BLOCK, SCALE_ROW, SCALE_TENSOR):
        raise ValueError(f"unknown scale mode {scale_mode!r}")
    return _norm(x, weight, residual, eps, mode, scale, out, q, scales, residual_out)


def add_rms_norm(x, weight, residual=None, eps=1e-6, out=None, residual_out=None):
    """add_rms_norm_quant without the quantization -> the norm, bf16 [T, H]."""
    dev = _device_of(x, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
    _norm(x, weight, residual, eps, None, None, out, None, None, residual_out)
    return out


def qk_norm_mrope_cache(query, key, value, q_weight, k_weight, cos_sin, positions, sections,
                        slot_mapping, key_cache, value_cache, k_scale, v_scale, eps=1e-6,
                        in_turn=False, interleaved=False, query_out=None):
    """qk_norm_rope_cache with a position on each of several axes (time, height,
    width): positions int64 [A, T], sections A numbers of rotated pairs,
    rot_dim / 2 in all.

    The first sections[0] pairs of a head turn by the first axis' position,
    and so on; with in_turn, pair i belongs to axis i % A while that axis has
    pairs left, else to the first.  Tokens with a position outside the table
    on any axis are padding."""
    dev, sections = _device_of(query, "query"), tuple(sections)
    stream = _stream_here(dev)
    if stream is not None:
        if query_out is None:
            query_out = torch.empty(query.shape, dtype=torch.bfloat16, device=dev)
        st = _attention._tensor_args.qk_norm_mrope_cache(
            _address("fp8_qk_norm_mrope_cache"), query, key, value, q_weight, k_weight, eps, cos_sin,
            bool(interleaved), positions, sections, bool(in_turn), slot_mapping, query_out,
            key_cache, value_cache, k_scale, v_scale, dev, stream)
        if st is not None:
            if st:
                _check(st)
            return query_out
    q, T, Hq, D, ld_q = _heads(query, "query", dev)
    k, Tk, Hk, Dk, ld_k = _heads(key, "key", dev)
    v, Tv, Hv, Dv, ld_v = _heads(value, "value", dev)
    if Tk != T or Dk != D or Tv != T or Hv != Hk or Dv != D:
        raise ValueError("query, key and value shapes do not match")
    kc, vc, nb, bs, Hc, Dc = _caches(key_cache, value_cache, dev)
    if Hc != Hk or Dc != D:
        raise ValueError("cache shapes do not match the tokens")
    cs, max_pos, rot = _matrix(cos_sin, "cos_sin", torch.float32, dev)
    pos, A, Tp, ld_pos = _rows(positions, "positions", torch.int64, dev)
    if Tp != T or A != len(sections):
        raise ValueError(f"positions must be [{len(sections)}, {T}]: a row for each section")
    if query_out is None:
        query_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    o, To, Ho, Do, ld_o = _heads(query_out, "query_out", dev)
    if To != T or Ho != Hq or Do != D:
        raise ValueError(f"query_out must be [{T}, {Hq}, {D}]")
    args = (q, ld_q, k, ld_k, v, ld_v,
            _vector(q_weight, "q_weight", torch.bfloat16, dev, D),
            _vector(k_weight, "k_weight", torch.bfloat16, dev, D), float(eps), cs,
            max_pos, rot, int(bool(interleaved)), pos, ld_pos, A,
            (_i64 * A)(*sections), int(bool(in_turn)),
            _vector(slot_mapping, "slot_mapping", torch.int64, dev, T), T, Hq, Hk, D,
            o, ld_o, kc, vc, nb, bs,
            _scale(k_scale, "k_scale", dev), _scale(v_scale, "v_scale", dev))
    _check(_call(dev, lambda: lib().fp8_qk_norm_mrope_cache(*args, _raw_stream(dev))))
    return query_out


def int4_pack(values):
    """4-bit values, one a byte (uint8 [N, K], rows' strides free) -> packed codes
    uint8 [N, K / 2], as int4_linear takes them."""
    dev = _device_of(values, "values")
    p, N, K, ld = _rows(values, "values", torch.uint8, dev)
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    _check(_call(dev, lambda: lib().fp8_int4_pack(p, ld, codes.data_ptr(), N, K, _raw_stream(dev))))
    return codes


def int4_quant_weight(w, group=128, symmetric=False):
    """bf16 w [N, K] rounded to 4 bits by groups of 32, 64 or 128 values ->
    (codes uint8 [N, K / 2], scales float32 [N, K / group], zeros uint8
    [N, K / group], None if symmetric)."""
    dev = _device_of(w, "w")
    p, N, K, ld = _rows(w, "w", torch.bfloat16, dev)
    groups = K // group if group > 0 else 0
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, groups), dtype=torch.float32, device=dev)
    zeros = None if symmetric else torch.empty((N, groups), dtype=torch.uint8, device=dev)
    _check(_call(dev, lambda: lib().fp8_int4_quant_weight(
        p, ld, codes.data_ptr(), scales.data_ptr(), None if symmetric else zeros.data_ptr(), N, K,
        int(group), _raw_stream(dev))))
    return codes, scales, zeros


def int4_workspace_bytes(M, N, K):
    """Workspace bytes with which int4_linear cuts K into runs (0: it does not)."""
    return _int4_workspace(int(M), int(N), int(K))


@functools.lru_cache(maxsize=4096)
def _int4_workspace(M, N, K):
    return int(lib().fp8_int4_workspace_bytes(M, N, K))


def int4_linear(x, codes, scales, zeros=None, out=None, workspace=None):
    """out = x . W^T of bf16 x [M, K] with 4-bit weights: packed codes uint8 [N, K / 2],
    scales float32 [N, K / group], zero points uint8 of the same shape (None: 8)
    -> bf16 [M, N].  Sizes that cut K into runs (int4_workspace_bytes > 0) get a
    workspace, allocated here unless given."""
    dev = _device_of(x, "x")
    stream = _stream_here(dev)
    if stream is not None and x.dim() == 2 and isinstance(codes, torch.Tensor) and codes.dim() == 2:
        M, N, ws = x.shape[0], codes.shape[0], workspace
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        if ws is None and M > 4:
            n = _int4_workspace(M, N, x.shape[1])
            if n:
                ws = torch.empty(n, dtype=torch.uint8, device=dev)
        st = _attention._tensor_args.int4_linear(_address("fp8_int4_linear"), x, codes, scales, zeros, out,
                                                 ws, dev, stream)
        if st is not None:
            if st:
                _check(st)
            return out
    xp, M, K, ld_x = _rows(x, "x", torch.bfloat16, dev)
    cp, N, half = _matrix(codes, "codes", torch.uint8, dev)
    sp, Ns, groups = _matrix(scales, "scales", torch.float32, dev)
    if half * 2 != K or Ns != N or groups == 0 or K % groups:
        raise ValueError(f"x {(M, K)}, codes {(N, half)} and scales {(Ns, groups)} do not match")
    zp = None
    if zeros is not None:
        zp, Nz, gz = _matrix(zeros, "zeros", torch.uint8, dev)
        if Nz != N or gz != groups:
            raise ValueError("zeros and scales shapes differ")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    op, _, _, ld_out = _rows(out, "out", torch.bfloat16, dev, (M, N))

    def call():
        l, ws = lib(), workspace
        if ws is None and M > 4:
            n = l.fp8_int4_workspace_bytes(M, N, K)
            if n:
                ws = torch.empty(n, dtype=torch.uint8, device=dev)
        ws_ptr, ws_len = _workspace(ws, dev)
        return l.fp8_int4_linear(xp, ld_x, cp, sp, zp, K // groups, op, ld_out, M, N, K, ws_ptr, ws_len,
                                 _raw_stream(dev))

    _check(_call(dev, call))
    return out


def logprobs_workspace_bytes(T, V, k=0, dtype=torch.bfloat16):
    """Workspace bytes of token_logprobs for logits [T, V] of this type.

    Fewer rows may need more: a buffer for any count up to T has the largest
    size over 1 .. min(T, 255) and T."""
    return _logprobs_workspace(_logits_type(dtype), int(T), int(V), int(k))


@functools.lru_cache(maxsize=4096)
def _logprobs_workspace(kind, T, V, k):
    return int(lib().fp8_logprobs_workspace_bytes(kind, T, V, k))


def _logits_type(dtype):
    if dtype is torch.bfloat16:
        return LOGITS_BF16
    if dtype is torch.float32:
        return LOGITS_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {dtype}")


def token_logprobs(logits, tokens, k=0, scale=1.0, logprobs=None, ranks=None, entropy=None, lse=None,
                   top_logprobs=None, top_ids=None, workspace=None):
    """Log probabilities of the tokens (int64 [T]) under softmax(scale * logits),
    logits bf16 or float32 [T, V] -> (logprobs [T], ranks int32 [T]: how many
    logits are larger, entropy [T], lse [T], top_logprobs [T, k], top_ids int32
    [T, k]: the k most likely, of equal ones the lower index first).

    A token outside [0, V) is padding (log probability 0, rank -1).  A row with
    a NaN or +inf gives NaN and -1.  k is at most 64."""
    dev = _device_of(logits, "logits")
    kind = _logits_type(logits.dtype)
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D with unit column stride")
    (T, V), k = logits.shape, int(k)
    if k < 0 or k > MAX_TOP or k > V:
        raise ValueError(f"k must be 0 .. {min(V, MAX_TOP)}, got {k}")
    f32, i32 = torch.float32, torch.int32
    if logprobs is None:
        logprobs = torch.empty(T, dtype=f32, device=dev)
    if ranks is None:
        ranks = torch.empty(T, dtype=i32, device=dev)
    if entropy is None:
        entropy = torch.empty(T, dtype=f32, device=dev)
    if lse is None:
        lse = torch.empty(T, dtype=f32, device=dev)
    if top_logprobs is None:
        top_logprobs = torch.empty((T, k), dtype=f32, device=dev)
    if top_ids is None:
        top_ids = torch.empty((T, k), dtype=i32, device=dev)
    if workspace is None:
        n = _logprobs_workspace(kind, T, V, k)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    stream = _stream_here(dev)
    if stream is not None:
        st = _attention._tensor_args.token_logprobs(
            _address("fp8_token_logprobs"), logits, tokens, scale, k, logprobs, ranks, entropy, lse,
            top_logprobs, top_ids, workspace, dev, stream)
        if st is not None:
            if st:
                _check(st)
            return logprobs, ranks, entropy, lse, top_logprobs, top_ids
    p, T, V, ld = _rows(logits, "logits", logits.dtype, dev)
    top = _matrix(top_logprobs, "top_logprobs", f32, dev)
    ids = _matrix(top_ids, "top_ids", i32, dev)
    if top[1:] != (T, k) or ids[1:] != (T, k):
        raise ValueError(f"top_logprobs and top_ids must be [{T}, {k}]")
    ws_ptr, ws_len = _workspace(workspace, dev)
    args = (p, kind, ld, _vector(tokens, "tokens", torch.int64, dev, T), float(scale), T, V, k,
            _vector(logprobs, "logprobs", f32, dev, T), _vector(ranks, "ranks", i32, dev, T),
            _vector(entropy, "entropy", f32, dev, T), _vector(lse, "lse", f32, dev, T),
            top[0], ids[0], ws_ptr, ws_len)
    _check(_call(dev, lambda: lib().fp8_token_logprobs(*args, _raw_stream(dev))))
    return logprobs, ranks, entropy, lse, top_logprobs, top_ids
