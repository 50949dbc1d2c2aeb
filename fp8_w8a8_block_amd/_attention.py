"""ctypes binding of the paged attention step (include/fp8w8a8_attention.h):
argument marshalling only, with the conventions of _lib.

Every length, offset and table stays on the device; no call synchronizes, so
a whole step can be captured in a graph.

Arguments as they should be are read by _tensor_args (csrc/tensor_args.cpp), one
call each; the checks written out here say what is wrong with the others.
"""

import ctypes
import importlib

import torch

from . import _lib
from ._lib import _check, _device_tensor, _i64, _int, _sz, _vp, _workspace

_f32 = ctypes.c_float

_SIGS = {
    "fp8_kv_slot_map": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i64,
                               _vp, _vp, _vp, _vp]),
    "fp8_validate_kv_slot_map": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp,
                                        _i64, _vp, _vp, _vp]),
    "fp8_qk_norm_rope_cache": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _f32, _vp, _i64,
                                      _i64, _int, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp,
                                      _vp, _i64, _i64, _vp, _vp, _vp]),
    "fp8_validate_qk_norm_rope_cache": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _f32,
                                               _vp, _i64, _i64, _int, _vp, _vp, _i64, _i64, _i64,
                                               _i64, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp]),
    "fp8_attention_workspace_bytes": (_sz, [_int, _i64, _i64, _i64, _i64, _i64]),
    "fp8_paged_attention": (_int, [_vp, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64,
                                   _vp, _vp, _f32, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _i64,
                                   _i64, _vp, _sz, _vp]),
    "fp8_prefix_attention": (_int, [_vp, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i64,
                                    _i64, _vp, _vp, _i64, _vp, _vp, _f32, _vp, _i64, _vp, _i64,
                                    _i64, _i64, _i64, _vp, _sz, _vp]),
    "fp8_validate_attention": (_int, [_vp, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i64,
                                      _i64, _vp, _vp, _i64, _vp, _vp, _f32, _i64, _i64, _vp, _i64,
                                      _vp, _i64, _i64, _i64, _i64, _vp, _sz, _sz]),
}

_bound = None


class _Unloaded:
    """Loads _tensor_args in the first call's place, as lib() does the library: the
    package is imported to build it."""

    def __getattr__(self, name):
        global _tensor_args
        _tensor_args = importlib.import_module("._tensor_args", __package__)
        return getattr(_tensor_args, name)


_tensor_args = _Unloaded()


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


def _on(t, name, dtype, device):
    """A device tensor of this type on this device (the checks of
    _device_tensor, which says what is wrong)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device:
        _device_tensor(t, name, dtype, device)


def _device_of(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


def _vector(t, name, dtype, device, n=None):
    """A contiguous 1-D device tensor (of n elements) -> its pointer."""
    p = _tensor_args.vector(t, dtype, device, -1 if n is None else n)
    if p is not None:
        return p
    _on(t, name, dtype, device)
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be 1-D" + (f" of {n} elements" if n is not None else ""))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(t, name, device):
    """[T, H, D] bf16 with each token's H * D values contiguous
    -> (pointer, T, H, D, token stride)."""
    got = _tensor_args.heads(t, device)
    if got is not None:
        return got
    _on(t, name, torch.bfloat16, device)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, H, D]")
    T, H, D = t.shape
    if T * H * D > 0:
        raise ValueError(f"{name} must be [T, H, D] with contiguous heads")
    return t.data_ptr(), T, H, D, H * D


def _scale(t, name, device):
    p = _tensor_args.vector(t, torch.float32, device, 1)
    if p is not None:
        return p
    _on(t, name, torch.float32, device)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one value")
    return t.data_ptr()


def _block_table(t, name, device, rows):
    """[rows, width] int32 with unit column stride -> (pointer, row stride, width)."""
    got = _tensor_args.table(t, device, rows)
    if got is not None:
        return got
    _on(t, name, torch.int32, device)
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must be [{rows}, width]")
    width, (ld, step) = t.shape[1], t.stride()
    if step != 1 and width > 1 and rows > 0:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), (ld if rows > 1 else width), width


def _matrix(t, name, dtype, device):
    """A contiguous 2-D device tensor -> (pointer, rows, columns)."""
    got = _tensor_args.matrix(t, dtype, device)
    if got is None:
        _on(t, name, dtype, device)
        raise ValueError(f"{name} must be 2-D and contiguous")
    return got


def _caches(key_cache, value_cache, device):
    """Both paged caches -> (key pointer, value pointer, blocks, block_size, H, D)."""
    got = _tensor_args.caches(key_cache, value_cache, device)
    if got is not None:
        return got
    for c, name in ((key_cache, "key_cache"), (value_cache, "value_cache")):
        _on(c, name, torch.uint8, device)
        if c.dim() != 4 or not c.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [blocks, block_size, H, D] tensor")
    raise ValueError("key_cache and value_cache shapes differ")


def _raw_stream(device):
    """Handle of the device's current stream (no Stream object around it)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _call(device, call):
    """Runs call() with `device` current."""
    if torch._C._cuda_getDevice() == device.index:
        return call()
    with torch.cuda.device(device):
        return call()


def kv_slot_map(computed_lens, new_lens, block_table, free_blocks, block_size, num_tokens,
                slot_mapping=None, positions=None, query_offsets=None, seq_lens=None,
                blocks_taken=None):
    """Block tables and slot maps of one step from the requests' lengths.

    computed_lens, new_lens int32 [B]: tokens in the cache, tokens added;
    block_table int32 [B, width] gets the new blocks (in place), taken in
    order from free_blocks int32.  Returns (slot_mapping int64 [num_tokens],
    positions int64 [num_tokens], query_offsets int32 [B + 1], seq_lens int32
    [B], blocks_taken int32 [1]); slots and positions behind the last token
    are -1, and so are slots of tokens that no free block was left for
    (blocks_taken then exceeds the number of free blocks)."""
    dev = _device_of(computed_lens, "computed_lens")
    computed = _vector(computed_lens, "computed_lens", torch.int32, dev)
    B, T = computed_lens.shape[0], int(num_tokens)
    if T < 0:
        raise ValueError("num_tokens must not be negative")
    if slot_mapping is None:
        slot_mapping = torch.empty(T, dtype=torch.int64, device=dev)
    if positions is None:
        positions = torch.empty(T, dtype=torch.int64, device=dev)
    if query_offsets is None:
        query_offsets = torch.empty(B + 1, dtype=torch.int32, device=dev)
    if seq_lens is None:
        seq_lens = torch.empty(B, dtype=torch.int32, device=dev)
    if blocks_taken is None:
        blocks_taken = torch.empty(1, dtype=torch.int32, device=dev)
    table, ld, width = _block_table(block_table, "block_table", dev, B)
    args = (computed, _vector(new_lens, "new_lens", torch.int32, dev, B), B, int(block_size),
            table, ld, width, _vector(free_blocks, "free_blocks", torch.int32, dev),
            free_blocks.shape[0], _vector(slot_mapping, "slot_mapping", torch.int64, dev, T),
            _vector(positions, "positions", torch.int64, dev, T), T,
            _vector(query_offsets, "query_offsets", torch.int32, dev, B + 1),
            _vector(seq_lens, "seq_lens", torch.int32, dev, B),
            _vector(blocks_taken, "blocks_taken", torch.int32, dev, 1))
    _check(_call(dev, lambda: lib().fp8_kv_slot_map(*args, _raw_stream(dev))))
    return slot_mapping, positions, query_offsets, seq_lens, blocks_taken


def qk_norm_rope_cache(query, key, value, q_weight, k_weight, cos_sin, positions, slot_mapping,
                       key_cache, value_cache, k_scale, v_scale, eps=1e-6, interleaved=False,
                       query_out=None):
    """Per-head RMS norm and rotation of query [T, Hq, D] and key [T, Hk, D]
    (bf16, token strides free), the keys and values stored as E4M3 codes in the
    paged caches at slot_mapping, in one pass -> the queries, bf16.

    cos_sin float32 [max_pos, rot_dim]: cosines then sines of each position;
    rot_dim < D rotates the first rot_dim values.  interleaved pairs
    neighbours instead of halves.  Tokens whose position is outside the table
    are padding: their rows of query_out stay as they were."""
    dev = _device_of(query, "query")
    q, T, Hq, D, ld_q = _heads(query, "query", dev)
    k, Tk, Hk, Dk, ld_k = _heads(key, "key", dev)
    v, Tv, Hv, Dv, ld_v = _heads(value, "value", dev)
    if Tk != T or Dk != D or Tv != T or Hv != Hk or Dv != D:
        raise ValueError("query, key and value shapes do not match")
    kc, vc, nb, bs, Hc, Dc = _caches(key_cache, value_cache, dev)
    if Hc != Hk or Dc != D:
        raise ValueError("cache shapes do not match the tokens")
    cs, max_pos, rot = _matrix(cos_sin, "cos_sin", torch.float32, dev)
    if query_out is None:
        query_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    o, To, Ho, Do, ld_o = _heads(query_out, "query_out", dev)
    if To != T or Ho != Hq or Do != D:
        raise ValueError(f"query_out must be [{T}, {Hq}, {D}]")
    args = (q, ld_q, k, ld_k, v, ld_v,
            _vector(q_weight, "q_weight", torch.bfloat16, dev, D),
            _vector(k_weight, "k_weight", torch.bfloat16, dev, D), float(eps), cs,
            max_pos, rot, int(bool(interleaved)),
            _vector(positions, "positions", torch.int64, dev, T),
            _vector(slot_mapping, "slot_mapping", torch.int64, dev, T), T, Hq, Hk, D,
            o, ld_o, kc, vc, nb, bs,
            _scale(k_scale, "k_scale", dev), _scale(v_scale, "v_scale", dev))
    _check(_call(dev, lambda: lib().fp8_qk_norm_rope_cache(*args, _raw_stream(dev))))
    return query_out


def attention_workspace_bytes(T, B, Hq, Hk, D, shared_prefix=False):
    """Workspace bytes of paged_attention (prefix_attention with
    shared_prefix) for T query tokens in B requests on the current device."""
    return int(lib().fp8_attention_workspace_bytes(int(bool(shared_prefix)), int(T), int(B),
                                                   int(Hq), int(Hk), int(D)))


def _attention(query, key_cache, value_cache, prefix, block_table, seq_lens, query_offsets, k_scale,
               v_scale, scale, window, sinks, out, lse, workspace):
    """Both attention calls; prefix: None or (prefix_table, prefix_len)."""
    dev = _device_of(query, "query")
    q, T, Hq, D, ld_q = _heads(query, "query", dev)
    kc, vc, nb, bs, Hk, Dc = _caches(key_cache, value_cache, dev)
    if Dc != D:
        raise ValueError("query and cache head sizes differ")
    lens = _vector(seq_lens, "seq_lens", torch.int32, dev)
    B = seq_lens.shape[0]
    table = _block_table(block_table, "block_table", dev, B)
    batch = (*table, lens, _vector(query_offsets, "query_offsets", torch.int32, dev, B + 1), B,
             _scale(k_scale, "k_scale", dev), _scale(v_scale, "v_scale", dev),
             float(D ** -0.5 if scale is None else scale))
    if prefix is not None:
        batch = (_vector(prefix[0], "prefix_table", torch.int32, dev), prefix[0].shape[0],
                 _vector(prefix[1], "prefix_len", torch.int32, dev, 1), *batch)
    else:
        batch = (*batch, int(window), int(sinks))
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    o, To, Ho, Do, ld_o = _heads(out, "out", dev)
    if To != T or Ho != Hq or Do != D:
        raise ValueError(f"out must be [{T}, {Hq}, {D}]")
    lse_ptr = None
    if lse is not None:
        lse_ptr, *shape = _matrix(lse, "lse", torch.float32, dev)
        if shape != [T, Hq]:
            raise ValueError(f"lse must be [{T}, {Hq}]")

    def call():
        l, ws = lib(), workspace
        if ws is None:
            n = l.fp8_attention_workspace_bytes(int(prefix is not None), T, B, Hq, Hk, D)
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
        ws_ptr, ws_len = _workspace(ws, dev)
        f = l.fp8_paged_attention if prefix is None else l.fp8_prefix_attention
        return f(q, ld_q, kc, vc, nb, bs, *batch, o, ld_o, lse_ptr, T, Hq, Hk, D, ws_ptr, ws_len,
                 _raw_stream(dev))

    _check(_call(dev, call))
    return out


def paged_attention(query, key_cache, value_cache, block_table, seq_lens, query_offsets, k_scale,
                    v_scale, scale=None, window=0, sinks=0, out=None, lse=None, workspace=None):
    """Causal attention of a ragged batch over the paged E4M3 caches
    [blocks, block_size, Hk, D]: query bf16 [T, Hq, D] -> bf16 [T, Hq, D].

    Request r's queries are tokens query_offsets[r] .. query_offsets[r + 1] - 1
    and the last of its seq_lens[r] cached tokens; key j's block is
    block_table[r, j // block_size].  window > 0 leaves a query its last
    `window` keys and the first `sinks`.  scale defaults to D ** -0.5; lse
    (float32 [T, Hq]) gets the log-sum-exp of the scores.  Rows that see no key
    are zeros (lse -inf), rows of no request stay as they were."""
    return _attention(query, key_cache, value_cache, None, block_table, seq_lens, query_offsets,
                      k_scale, v_scale, scale, window, sinks, out, lse, workspace)


def prefix_attention(query, key_cache, value_cache, prefix_table, prefix_len, block_table,
                     seq_lens, query_offsets, k_scale, v_scale, scale=None, out=None, lse=None,
                     workspace=None):
    """paged_attention for requests that all start with the same prefix_len
    (int32 [1], on the device) tokens in the blocks prefix_table (int32):
    block_table and seq_lens describe what follows it in each request.  The
    prefix's keys and values are read once for the whole batch.

    Every query sees the whole prefix.  A request of n queries needs
    seq_lens[r] >= n - 1 for that to be causal: with fewer own tokens its first
    queries are tokens of the prefix, which paged_attention over the joined
    tokens masks and this call does not."""
    if prefix_table is None or prefix_len is None:
        raise TypeError("prefix_table and prefix_len must be tensors")
    return _attention(query, key_cache, value_cache, (prefix_table, prefix_len), block_table,
                      seq_lens, query_offsets, k_scale, v_scale, scale, 0, 0, out, lse, workspace)
