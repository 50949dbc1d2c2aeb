"""ctypes binding of the paged attention step (include/fp8w8a8_attention.h):
argument marshalling only, with the conventions of _lib.

Every length, offset and table stays on the device; no call synchronizes, so
a whole step can be captured in a graph.
"""

import ctypes

import torch

from . import _lib
from ._lib import _cache, _check, _device_tensor, _i64, _int, _stream, _sz, _tokens, _vp, _workspace

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


def _vector(t, name, dtype, device, n=None):
    """A contiguous 1-D device tensor (of n elements) -> its pointer."""
    _device_tensor(t, name, dtype, device)
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be 1-D" + (f" of {n} elements" if n is not None else ""))
    if t.stride(0) != 1 and t.shape[0] > 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(t, name):
    """_tokens, where an empty step's strides do not matter."""
    if t.dim() == 3 and t.numel() == 0 and t.dtype == torch.bfloat16 and t.is_cuda:
        return (*t.shape, t.shape[1] * t.shape[2])
    return _tokens(t, name)


def _scale(t, name, device):
    _device_tensor(t, name, torch.float32, device)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one value")
    return t.data_ptr()


def _block_table(t, name, device, rows):
    """[rows, width] int32 with unit column stride -> (pointer, row stride, width)."""
    _device_tensor(t, name, torch.int32, device)
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must be [{rows}, width]")
    if t.numel() > 0 and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), (t.stride(0) if rows > 1 else t.shape[1]), t.shape[1]


def _caches(key_cache, value_cache, device):
    shape = _cache(key_cache, "key_cache")
    if _cache(value_cache, "value_cache") != shape:
        raise ValueError("key_cache and value_cache shapes differ")
    if key_cache.device != device or value_cache.device != device:
        raise ValueError(f"the caches must be tensors on {device}")
    return shape


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
    dev = computed_lens.device
    _vector(computed_lens, "computed_lens", torch.int32, dev)
    B, T = computed_lens.shape[0], int(num_tokens)
    if T < 0:
        raise ValueError("num_tokens must not be negative")
    with torch.cuda.device(dev):
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
        free = _vector(free_blocks, "free_blocks", torch.int32, dev)
        _check(lib().fp8_kv_slot_map(
            computed_lens.data_ptr(), _vector(new_lens, "new_lens", torch.int32, dev, B), B,
            int(block_size), table, ld, width, free, free_blocks.shape[0],
            _vector(slot_mapping, "slot_mapping", torch.int64, dev, T),
            _vector(positions, "positions", torch.int64, dev, T), T,
            _vector(query_offsets, "query_offsets", torch.int32, dev, B + 1),
            _vector(seq_lens, "seq_lens", torch.int32, dev, B),
            _vector(blocks_taken, "blocks_taken", torch.int32, dev, 1), _stream(computed_lens)))
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
    T, Hq, D, ld_q = _heads(query, "query")
    Tk, Hk, Dk, ld_k = _heads(key, "key")
    Tv, Hv, Dv, ld_v = _heads(value, "value")
    if (Tk, Dk) != (T, D) or (Tv, Hv, Dv) != (T, Hk, D):
        raise ValueError("query, key and value shapes do not match")
    dev = query.device
    if key.device != dev or value.device != dev:
        raise ValueError(f"key and value must be tensors on {dev}")
    nb, bs, Hc, Dc = _caches(key_cache, value_cache, dev)
    if (Hc, Dc) != (Hk, D):
        raise ValueError("cache shapes do not match the tokens")
    _device_tensor(cos_sin, "cos_sin", torch.float32, dev)
    if cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous [positions, rot_dim] tensor")
    with torch.cuda.device(dev):
        if query_out is None:
            query_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        To, Ho, Do, ld_o = _heads(query_out, "query_out")
        if (To, Ho, Do) != (T, Hq, D) or query_out.device != dev:
            raise ValueError(f"query_out must be [{T}, {Hq}, {D}] on {dev}")
        _check(lib().fp8_qk_norm_rope_cache(
            query.data_ptr(), ld_q, key.data_ptr(), ld_k, value.data_ptr(), ld_v,
            _vector(q_weight, "q_weight", torch.bfloat16, dev, D),
            _vector(k_weight, "k_weight", torch.bfloat16, dev, D), float(eps), cos_sin.data_ptr(),
            cos_sin.shape[0], cos_sin.shape[1], int(bool(interleaved)),
            _vector(positions, "positions", torch.int64, dev, T),
            _vector(slot_mapping, "slot_mapping", torch.int64, dev, T), T, Hq, Hk, D,
            query_out.data_ptr(), ld_o, key_cache.data_ptr(), value_cache.data_ptr(), nb, bs,
            _scale(k_scale, "k_scale", dev), _scale(v_scale, "v_scale", dev), _stream(query)))
    return query_out


def attention_workspace_bytes(T, B, Hq, Hk, D, shared_prefix=False):
    """Workspace bytes of paged_attention (prefix_attention with
    shared_prefix) for T query tokens in B requests on the current device."""
    return int(lib().fp8_attention_workspace_bytes(int(bool(shared_prefix)), int(T), int(B),
                                                   int(Hq), int(Hk), int(D)))


def _attention(query, key_cache, value_cache, prefix_table, prefix_len, block_table, seq_lens,
               query_offsets, k_scale, v_scale, scale, window, sinks, out, lse, workspace):
    T, Hq, D, ld_q = _heads(query, "query")
    dev = query.device
    nb, bs, Hk, Dc = _caches(key_cache, value_cache, dev)
    if Dc != D:
        raise ValueError("query and cache head sizes differ")
    lens = _vector(seq_lens, "seq_lens", torch.int32, dev)
    B = seq_lens.shape[0]
    offs = _vector(query_offsets, "query_offsets", torch.int32, dev, B + 1)
    table, ld_t, width = _block_table(block_table, "block_table", dev, B)
    ks, vs = _scale(k_scale, "k_scale", dev), _scale(v_scale, "v_scale", dev)
    shared = prefix_table is not None
    if shared:
        p_table = _vector(prefix_table, "prefix_table", torch.int32, dev)
        p_len = _vector(prefix_len, "prefix_len", torch.int32, dev, 1)
    if scale is None:
        scale = D ** -0.5
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        To, Ho, Do, ld_o = _heads(out, "out")
        if (To, Ho, Do) != (T, Hq, D) or out.device != dev:
            raise ValueError(f"out must be [{T}, {Hq}, {D}] on {dev}")
        lse_ptr = None
        if lse is not None:
            _device_tensor(lse, "lse", torch.float32, dev, (T, Hq))
            if not lse.is_contiguous():
                raise ValueError("lse must be contiguous")
            lse_ptr = lse.data_ptr()
        l = lib()
        if workspace is None:
            n = int(l.fp8_attention_workspace_bytes(int(shared), T, B, Hq, Hk, D))
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        ws_ptr, ws_len = _workspace(workspace, dev)
        if shared:
            _check(l.fp8_prefix_attention(
                query.data_ptr(), ld_q, key_cache.data_ptr(), value_cache.data_ptr(), nb, bs,
                p_table, prefix_table.shape[0], p_len, table, ld_t, width, lens, offs, B, ks, vs,
                float(scale), out.data_ptr(), ld_o, lse_ptr, T, Hq, Hk, D, ws_ptr, ws_len,
                _stream(query)))
        else:
            _check(l.fp8_paged_attention(
                query.data_ptr(), ld_q, key_cache.data_ptr(), value_cache.data_ptr(), nb, bs,
                table, ld_t, width, lens, offs, B, ks, vs, float(scale), int(window), int(sinks),
                out.data_ptr(), ld_o, lse_ptr, T, Hq, Hk, D, ws_ptr, ws_len, _stream(query)))
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
    return _attention(query, key_cache, value_cache, None, None, block_table, seq_lens,
                      query_offsets, k_scale, v_scale, scale, window, sinks, out, lse, workspace)


def prefix_attention(query, key_cache, value_cache, prefix_table, prefix_len, block_table,
                     seq_lens, query_offsets, k_scale, v_scale, scale=None, out=None, lse=None,
                     workspace=None):
    """paged_attention for requests that all start with the same prefix_len
    (int32 [1], on the device) tokens in the blocks prefix_table (int32):
    block_table and seq_lens describe what follows it in each request.  The
    prefix's keys and values are read once for the whole batch."""
    if prefix_table is None or prefix_len is None:
        raise TypeError("prefix_table and prefix_len must be tensors")
    return _attention(query, key_cache, value_cache, prefix_table, prefix_len, block_table,
                      seq_lens, query_offsets, k_scale, v_scale, scale, 0, 0, out, lse, workspace)
