"""Timed cases of the paged-attention operators: slot maps, the fused query /
key norm with rotation and cache store, windowed attention over the paged
FP8 cache, and attention of a batch that shares a prefix.

``own`` chooses between the operators' plain form (elementary torch
operations in 32 bits) and the framework's calls; both take what ``prepare``
makes.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # block bookkeeping of one decode step: every request grows by a token
        dict(name="slots_decode", op="slots", requests=256, tokens=256, most=32768, page=16,
             decode=True),
        # the same of a prefill batch: prompts of many lengths, some already cached in part
        dict(name="slots_prefill", op="slots", requests=96, tokens=65536, most=8192, page=16,
             decode=False),
        # one decode step of a few requests: latency alone
        dict(name="rope_decode", op="rope", tokens=16, q_heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, page=16, reach=131072),
        # a prefill chunk of a grouped-query 8B-class model, one token short of 8192
        dict(name="rope_prefill", op="rope", tokens=8191, q_heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, page=16, reach=131072),
        # rotation of a part of wide heads, neighbours paired, a ragged batch
        dict(name="rope_partial", op="rope", tokens=2049, q_heads=16, kv_heads=2, dim=256, rot=64,
             interleaved=True, page=32, reach=40000),
        # a few short windowed requests: the smallest decode step
        dict(name="decode_window", op="attention", requests=4, tokens=4, lo=700, hi=30000,
             q_heads=64, kv_heads=8, dim=64, page=16, window=1000, sinks=4, lse=False),
        # a decode batch of ragged contexts, the whole context visible
        dict(name="decode_batch", op="attention", requests=64, tokens=64, lo=1000, hi=8192,
             q_heads=32, kv_heads=8, dim=128, page=16, window=0, sinks=0, lse=False),
        # one long-document request: the context has to be split over the card
        dict(name="decode_long", op="attention", requests=1, tokens=1, lo=131071, hi=131071,
             q_heads=32, kv_heads=8, dim=128, page=16, window=0, sinks=0, lse=True),
        # a chunk of three prompts, with what earlier chunks cached before them
        dict(name="prefill_full", op="attention", requests=3, tokens=8192, lo=0, hi=4096,
             q_heads=32, kv_heads=8, dim=128, page=16, window=0, sinks=0, lse=True),
        # windowed layers of a long prompt, the first tokens kept
        dict(name="prefill_window", op="attention", requests=2, tokens=8001, lo=0, hi=2000,
             q_heads=64, kv_heads=8, dim=64, page=16, window=1000, sinks=4, lse=False),
        # a decode batch behind one system prompt
        dict(name="prefix_batch", op="prefix", requests=64, tokens=64, prefix=8192, hi=512,
             q_heads=32, kv_heads=8, dim=128, page=16, lse=False),
        # many samples of one long document
        dict(name="prefix_long", op="prefix", requests=250, tokens=250, prefix=32761, hi=200,
             q_heads=32, kv_heads=4, dim=128, page=16, lse=True),
    ]


def _between(rng, lo, hi):
    """A whole number of lo..hi, its logarithm spread evenly."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


HEADS = ((32, 8), (64, 8), (16, 2), (8, 8), (12, 1), (28, 4), (5, 5))


def draw(rng):
    op = rng.choice(["slots", "rope", "attention", "attention", "prefix"])
    page = rng.choice([1, 7, 16, 16, 32, 64])
    if op == "slots":
        decode = rng.random() < 0.5
        requests = _between(rng, 1, 512)
        return dict(op=op, requests=requests, decode=decode, page=page,
                    tokens=requests if decode else _between(rng, requests, 65536),
                    most=_between(rng, 64, 32768 if decode else 8192))
    hq, hk = rng.choice(HEADS)
    dim = rng.choice([64, 128, 128, 256])
    if op == "rope":
        cost = hq * dim / 4096.0
        return dict(op=op, tokens=_between(rng, 1, int(8191 / max(1.0, 1.3 * cost))), q_heads=hq,
                    kv_heads=hk, dim=dim, rot=rng.choice([dim, dim // 2, dim // 4]),
                    interleaved=rng.random() < 0.5, page=page, reach=_between(rng, 9000, 131072))
    lse = rng.random() < 0.5
    if op == "prefix":
        requests = _between(rng, 1, 128)
        tokens = requests * rng.choice([1, 1, 1, 2])
        return dict(op=op, requests=requests, tokens=tokens,
                    prefix=_between(rng, 17, min(32768, 2 ** 35 // (tokens * hq * dim))),
                    hi=_between(rng, 8, 400), q_heads=hq, kv_heads=hk, dim=dim, page=page, lse=lse)
    window = rng.choice([0, 0, _between(rng, 16, 4096)])
    sinks = rng.choice([0, 1, 4, 130]) if window else 0
    if rng.random() < 0.6:
        requests = _between(rng, 1, 64)
        hi = _between(rng, 64, min(131071, 2 ** 28 // (requests * hk * dim)))
        return dict(op=op, requests=requests, tokens=requests * rng.choice([1, 1, 1, 3]),
                    lo=_between(rng, 4, hi), hi=hi, q_heads=hq, kv_heads=hk, dim=dim, page=page,
                    window=window, sinks=sinks, lse=lse)
    requests = _between(rng, 1, 6)
    return dict(op=op, requests=requests, tokens=_between(rng, 100, min(8000, 2 ** 24 // (hq * dim))),
                lo=0, hi=_between(rng, 8, 2000), q_heads=hq, kv_heads=hk, dim=dim, page=page,
                window=window, sinks=sinks, lse=lse)


def _lengths(case):
    """(new tokens, context before them) of each request, from the case alone."""
    b, t = case["requests"], case["tokens"]
    if t % b == 0 and t // b <= 4:
        new = [t // b] * b
        before = [max(0, case["lo"] + (case["hi"] - case["lo"]) * i // max(1, b - 1) - new[i])
                  for i in range(b)]
        if b == 1:
            before = [max(0, case["hi"] - new[0])]
        return new, before
    share = [i + 1 for i in range(b)]
    new = [max(1, t * s // sum(share)) for s in share]
    new[-1] += t - sum(new)
    return new, [case["lo"] + (case["hi"] - case["lo"]) * (b - i) // b for i in range(b)]


def _suffixes(case):
    """Length of each request's own part (its new tokens counted)."""
    b, n = case["requests"], case["tokens"] // case["requests"]
    return [max(n, 1 + (case["hi"] - 1) * (i + 1) // b) for i in range(b)]


# ---- inputs --------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _codes(g, *shape):
    """E4M3 codes of normal values at a scale of 1/32, as raw bytes."""
    n, out = shape[0], torch.empty(shape, dtype=torch.uint8, device=DEV)
    step = max(1, 2 ** 27 // max(1, math.prod(shape[1:])))
    for i in range(0, n, step):
        x = torch.randn((min(step, n - i),) + shape[1:], generator=g, device=DEV)
        out[i:i + step] = x.mul_(32).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _one(value, dtype=torch.float32):
    return torch.tensor([value], dtype=dtype, device=DEV)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(pool, lengths, page, width=1):
    """Block table of requests of these lengths, their blocks taken from ``pool``; -1 behind them."""
    blocks = [-(-n // page) for n in lengths]
    first = np.cumsum([0] + blocks)
    i = torch.arange(max(width, max(blocks)), device=DEV)
    b, f = (torch.tensor(v, device=DEV)[:, None] for v in (blocks, first[:-1].tolist()))
    at = torch.where(i < b, f + i, 0)
    return torch.where(i < b, pool[at], -1).to(torch.int32).contiguous(), int(first[-1])


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def _prepare_slots(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng([11, seed])
    b, t, page = case["requests"], case["tokens"], case["page"]
    computed = r.integers(0, case["most"] + 1, b)
    if case["decode"]:
        new = np.ones(b, dtype=np.int64)
    else:  # a composition of the tokens, the first requests started earlier
        cuts = np.sort(r.integers(0, t + 1, b - 1))
        new = np.diff(np.concatenate([[0], cuts, [t]]))
        computed[b // 4:] = 0
    have = -(-computed // page)
    need = -(-(computed + new) // page)
    total = int(need.sum())
    pool = torch.randperm(total + 64, generator=g, device=DEV).to(torch.int32)
    # rows for the longest context that the program serves
    table, used = _table(pool, (have * page).tolist(), page,
                         width=-(-(case["most"] + (1 if case["decode"] else t)) // page))
    # outputs and the step's buffers stay in place from step to step, as in a captured graph
    return dict(case=case, computed=_ints(computed.tolist()), new=_ints(new.tolist()),
                table=table, free=pool[used:].contiguous(), tokens=t, page=page,
                slots=torch.empty(t, dtype=torch.int64, device=DEV),
                positions=torch.empty(t, dtype=torch.int64, device=DEV),
                offsets=torch.empty(b + 1, dtype=torch.int32, device=DEV),
                lens=torch.empty(b, dtype=torch.int32, device=DEV),
                taken=torch.empty(1, dtype=torch.int32, device=DEV))


def _prepare_rope(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, hq, hk, d, page = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim", "page"))
    rot, reach = case["rot"], case["reach"]
    # queries, keys and values are slices of the projection's one output row
    qkv = _normal(g, t, hq + 2 * hk, d)
    qkv[:, hq:hq + hk, :4] *= 20
    qkv = qkv.to(torch.bfloat16)
    freq = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(reach, dtype=torch.float64, device=DEV)[:, None] * freq
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    start = int(torch.randint(0, reach - t, (1,), generator=g, device=DEV)) if reach > t else 0
    positions = (start + torch.arange(t, device=DEV)) % reach
    blocks = 2 * -(-t // page) + 3
    pool = torch.randperm(blocks, generator=g, device=DEV)
    i = torch.arange(t, device=DEV)
    return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:],
                qw=(1 + 0.1 * _normal(g, d)).to(torch.bfloat16),
                kw=(1 + 0.1 * _normal(g, d)).to(torch.bfloat16),
                cos_sin=table, positions=positions, slots=pool[i // page] * page + i % page,
                key_cache=_codes(g, blocks, page, hk, d), value_cache=_codes(g, blocks, page, hk, d),
                ks=_one(16 / 448), vs=_one(1.0), eps=1e-6,
                out=torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV))


def _prepare_attention(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng([12, seed])
    t, hq, hk, d, page = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim", "page"))
    new, before = _lengths(case)
    order = r.permutation(len(new))
    new, lens = [new[i] for i in order], [new[i] + before[i] for i in order]
    blocks = sum(-(-n // page) for n in lens) + 5
    pool = torch.randperm(blocks, generator=g, device=DEV)
    table, _ = _table(pool, lens, page)
    return dict(case=case, q=(_normal(g, t, hq, d) * 1.5).to(torch.bfloat16),
                key_cache=_codes(g, blocks, page, hk, d), value_cache=_codes(g, blocks, page, hk, d),
                table=table, lens=_ints(lens), most=max(new), longest=max(lens),
                offsets=_ints(np.cumsum([0] + new).tolist()), ks=_one(1 / 32), vs=_one(1 / 32),
                **_outputs(case))


def _prepare_prefix(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng([13, seed])
    t, hq, hk, d, page = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim", "page"))
    lens = r.permutation(_suffixes(case)).tolist()
    shared = -(-case["prefix"] // page)
    blocks = shared + sum(-(-n // page) for n in lens) + 5
    pool = torch.randperm(blocks, generator=g, device=DEV)
    table, _ = _table(pool[shared:], lens, page)
    n = t // len(lens)
    return dict(case=case, q=(_normal(g, t, hq, d) * 1.5).to(torch.bfloat16),
                key_cache=_codes(g, blocks, page, hk, d), value_cache=_codes(g, blocks, page, hk, d),
                prefix_table=pool[:shared].to(torch.int32), prefix_len=_one(case["prefix"], torch.int32),
                prefix=case["prefix"], table=table, lens=_ints(lens), most=n, longest=max(lens),
                offsets=_ints(list(range(0, t + 1, n))), ks=_one(1 / 32), vs=_one(1 / 32),
                **_outputs(case))


def _outputs(case):
    """Buffers that a serving program keeps: the output and the log-sum-exp."""
    t, hq, d = (case[k] for k in ("tokens", "q_heads", "dim"))
    return dict(out=torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV),
                lse=torch.empty((t, hq), dtype=torch.float32, device=DEV) if case["lse"] else None)


_PREPARE = dict(slots=_prepare_slots, rope=_prepare_rope, attention=_prepare_attention,
                prefix=_prepare_prefix)


# ---- one pass --------------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _own_slots(s):
    import fp8_w8a8_block_amd as fp8
    slots, positions, offsets, lens, taken = fp8.kv_slot_map(
        s["computed"], s["new"], s["table"], s["free"], s["page"], s["tokens"],
        slot_mapping=s["slots"], positions=s["positions"], query_offsets=s["offsets"],
        seq_lens=s["lens"], blocks_taken=s["taken"])
    return dict(slots=slots, positions=positions, offsets=offsets, lens=lens, taken=taken,
                table=s["table"])


def _own_rope(s):
    import fp8_w8a8_block_amd as fp8
    q = fp8.qk_norm_rope_cache(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["cos_sin"],
                               s["positions"], s["slots"], s["key_cache"], s["value_cache"],
                               s["ks"], s["vs"], eps=s["eps"],
                               interleaved=s["case"]["interleaved"], query_out=s["out"])
    return _rope_outputs(s, q)


def _own_attention(s):
    import fp8_w8a8_block_amd as fp8
    out = fp8.paged_attention(s["q"], s["key_cache"], s["value_cache"], s["table"], s["lens"],
                              s["offsets"], s["ks"], s["vs"], window=s["case"]["window"],
                              sinks=s["case"]["sinks"], out=s["out"], lse=s["lse"])
    return dict(out=out, lse=s["lse"])


def _own_prefix(s):
    import fp8_w8a8_block_amd as fp8
    out = fp8.prefix_attention(s["q"], s["key_cache"], s["value_cache"], s["prefix_table"],
                               s["prefix_len"], s["table"], s["lens"], s["offsets"], s["ks"],
                               s["vs"], out=s["out"], lse=s["lse"])
    return dict(out=out, lse=s["lse"])


def _plain_slots(s):
    page, c, n = s["page"], s["computed"].long(), s["new"].long()
    lens, ends = c + n, n.cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    have, need = (c + page - 1) // page, (lens + page - 1) // page
    take = need - have
    first = take.cumsum(0) - take
    col = torch.arange(s["table"].shape[1], device=DEV)
    at = first[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    given = s["free"][at.clamp(0, s["free"].numel() - 1)]
    s["table"].copy_(torch.where(fresh, given, s["table"]))
    t = torch.arange(s["tokens"], device=DEV)
    r = torch.searchsorted(ends, t, right=True)
    live = r < n.numel()
    r = r.clamp(max=n.numel() - 1)
    pos = c[r] + t - offsets[r]
    slot = s["table"][r, (pos // page).clamp(0, col.numel() - 1)].long() * page + pos % page
    return dict(slots=torch.where(live, slot, -1), positions=torch.where(live, pos, -1),
                offsets=offsets.int(), lens=lens.int(), taken=take.sum(0, keepdim=True).int(),
                table=s["table"])


def _plain_rope(s):
    case = s["case"]
    d, rot = case["dim"], case["rot"]
    half = rot // 2
    cos, sin = s["cos_sin"][s["positions"]].unsqueeze(1).split(half, -1)

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1) if rot < d else y

    def stored(cache, x, scale):
        codes = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache.view(-1, *cache.shape[2:])[s["slots"]] = codes

    s["out"].copy_(turned(s["q"], s["qw"]))
    stored(s["key_cache"], turned(s["k"], s["kw"]), s["ks"])
    stored(s["value_cache"], s["v"].float(), s["vs"])
    return _rope_outputs(s, s["out"])


def _rope_outputs(s, q):
    return dict(q=q, key_cache=s["key_cache"].view(torch.float8_e4m3fn),
                value_cache=s["value_cache"].view(torch.float8_e4m3fn))


def _gathered(s, table, longest):
    """Keys and values of each row of a block table in 32 bits, [B, Hk, L, D]."""
    page = s["case"]["page"]
    j = torch.arange(longest, device=DEV)
    slot = table[:, j // page].long().clamp(min=0) * page + j % page

    def of(cache, scale):
        x = cache.view(-1, *cache.shape[2:])[slot].view(torch.float8_e4m3fn).float()
        return (x * scale).transpose(1, 2)

    return of(s["key_cache"], s["ks"]), of(s["value_cache"], s["vs"])


def _padded(s):
    """Queries as [B, Hk, N * G, D] in 32 bits, the row of q that each [B, N] is, and whether it is one."""
    case = s["case"]
    hk, d = case["kv_heads"], case["dim"]
    g = case["q_heads"] // hk
    i = torch.arange(s["most"], device=DEV)
    n = (s["offsets"][1:] - s["offsets"][:-1]).long()
    row = (s["offsets"][:-1, None] + i).clamp(max=case["tokens"] - 1).long()
    q = s["q"].float()[row].view(row.shape[0], s["most"], hk, g, d).transpose(1, 2)
    return q.reshape(row.shape[0], hk, -1, d), row, i < n[:, None], n


def _unpadded(s, row, live, o, lse):
    """[B, Hk, N, G, D] and [B, Hk, N, G] back to the tokens, in the outputs' types."""
    case = s["case"]
    t, hq, d = case["tokens"], case["q_heads"], case["dim"]
    at = torch.where(live, row, t).flatten()     # what is no query goes to a row behind the last
    out = torch.empty((t + 1, hq, d), dtype=torch.float32, device=DEV)
    out[at] = o.transpose(1, 2).reshape(-1, hq, d)
    s["out"].copy_(out[:t])
    if s["lse"] is not None:
        e = torch.empty((t + 1, hq), dtype=torch.float32, device=DEV)
        e[at] = lse.transpose(1, 2).reshape(-1, hq)
        s["lse"].copy_(e[:t])
    return dict(out=s["out"], lse=s["lse"])


def _softmax(x):
    """exp(x - max) in place, its row sums and the log-sum-exp; a row of -inf gives zeros and -inf."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    total = x.sub_(top).exp_().sum(-1, keepdim=True)
    return x, torch.where(total > 0, total, 1.0), (total.log() + top).squeeze(-1)


def _plain_attention(s):
    case = s["case"]
    hk, g = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    q, row, live, n = _padded(s)
    k, v = _gathered(s, s["table"], s["longest"])
    x = torch.matmul(q * case["dim"] ** -0.5, k.transpose(-1, -2))
    del k
    j = torch.arange(s["longest"], device=DEV)
    pos = (s["lens"].long() - n)[:, None] + torch.arange(s["most"], device=DEV)
    seen = j <= pos[..., None]
    if case["window"]:
        seen &= (j > pos[..., None] - case["window"]) | (j < case["sinks"])
    b, _, _, l = x.shape
    x = x.view(b, hk, s["most"], g, l).masked_fill_(~seen[:, None, :, None], -math.inf)
    p, total, lse = _softmax(x)
    o = torch.matmul(p.view(b, hk, -1, l), v).view(b, hk, s["most"], g, -1) / total
    return _unpadded(s, row, live, o, lse)


def _plain_prefix(s):
    case = s["case"]
    hk, g, d = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["dim"]
    q, row, live, n = _padded(s)
    b, m, far = q.shape[0], s["most"], s["prefix"]
    q = q * d ** -0.5
    pk, pv = _gathered(s, s["prefix_table"][None], far)
    k, v = _gathered(s, s["table"], s["longest"])
    flat = q.transpose(0, 1).reshape(hk, -1, d)
    x = torch.matmul(flat, pk[0].transpose(-1, -2)).view(hk, b, m, g, far).transpose(0, 1)
    y = torch.matmul(q, k.transpose(-1, -2)).view(b, hk, m, g, -1)
    pos = (s["lens"].long() - n)[:, None] + torch.arange(m, device=DEV)
    seen = torch.arange(s["longest"], device=DEV) <= pos[..., None]
    y.masked_fill_(~seen[:, None, :, None], -math.inf)
    p, total, lse = _softmax(torch.cat([x, y], -1))
    o = torch.matmul(p[..., :far].transpose(0, 1).reshape(hk, -1, far), pv[0])
    o = o.view(hk, b, m, g, d).transpose(0, 1)
    o = o + torch.matmul(p[..., far:].reshape(b, hk, m * g, -1), v).view(b, hk, m, g, d)
    return _unpadded(s, row, live, o / total, lse)


_PLAIN = dict(slots=_plain_slots, rope=_plain_rope, attention=_plain_attention,
              prefix=_plain_prefix)
_OWN = dict(slots=_own_slots, rope=_own_rope, attention=_own_attention, prefix=_own_prefix)


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    t, b = case["tokens"], case.get("requests", 1)
    if case["op"] == "slots":
        fresh = -(-t // case["page"])
        return dict(bytes=8.0 * b + 16.0 * t + 8.0 * b + 8.0 * fresh, flops=0.0)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        row = 2.0 * (2 * hq + 2 * hk) * d + 2.0 * hk * d + 4.0 * case["rot"] + 16.0
        return dict(bytes=t * row, flops=t * (hq + hk) * d * 9.0)
    rows = 4.0 * t * hq * d + (4.0 * t * hq if case["lse"] else 0.0)
    if case["op"] == "prefix":
        lens, n = _suffixes(case), t // b
        keys = case["prefix"] + sum(lens)
        pairs = t * case["prefix"] + sum(n * l - n * (n - 1) // 2 for l in lens)
        return dict(bytes=rows + 2.0 * hk * d * keys, flops=4.0 * d * hq * pairs)
    window, sinks, keys, pairs = case["window"], case["sinks"], 0, 0
    for n, before in zip(*_lengths(case)):
        pos = np.arange(before, before + n, dtype=np.int64)
        if window:
            low = np.maximum(0, pos - window + 1)
            pairs += int((pos + 1 - low + np.minimum(sinks, low)).sum())
            keys += int(before + n - low[0] + min(sinks, low[0]))
        else:
            pairs += int((pos + 1).sum())
            keys += before + n
    return dict(bytes=rows + 2.0 * hk * d * keys, flops=4.0 * d * hq * pairs)


# ---- the definitions in 64 bits ------------------------------------------------------

def exact(case, seed):
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    hq, hk, d, page = (case[k] for k in ("q_heads", "kv_heads", "dim", "page"))
    out = torch.zeros((case["tokens"], hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((case["tokens"], hq), -math.inf, dtype=torch.float64, device=DEV)
    first = s["offsets"].tolist()
    for r, length in enumerate(s["lens"].tolist()):
        a, e = first[r], first[r + 1]
        own_slots = _slots_of(s["table"][r], length, page)
        far = 0
        if case["op"] == "prefix":
            far = case["prefix"]
            own_slots = torch.cat([_slots_of(s["prefix_table"], far, page), own_slots])
        j = torch.arange(own_slots.numel(), device=DEV)
        i = far + length - (e - a) + torch.arange(e - a, device=DEV)
        hidden = j[None] > i[:, None]
        if case.get("window"):
            hidden |= (i[:, None] - j[None] >= case["window"]) & (j[None] >= case["sinks"])
        for h in range(hk):
            k = _values(s["key_cache"], own_slots, h) * s["ks"].double()
            v = _values(s["value_cache"], own_slots, h) * s["vs"].double()
            for c in range(h * (hq // hk), (h + 1) * (hq // hk)):
                z = (s["q"][a:e, c].double() @ k.t()) / math.sqrt(d)
                z[hidden] = -math.inf
                lse[a:e, c] = torch.logsumexp(z, 1)
                out[a:e, c] = torch.softmax(z, 1) @ v
    return dict(out=out, lse=lse if case["lse"] else None)


def _slots_of(row, length, page):
    blocks = row[:-(-length // page)].long()
    return (blocks[:, None] * page + torch.arange(page, device=DEV)).flatten()[:length]


def _values(cache, slots, head):
    return cache.flatten(0, 1)[:, head][slots].view(torch.float8_e4m3fn).double()


def _exact_rope(s):
    case = s["case"]
    rot, pos = case["rot"], s["positions"]
    turn = torch.complex(*s["cos_sin"][pos].double().chunk(2, 1))[:, None]

    def of(x, w):
        x = x.double()
        x = x / (x.square().mean(2, keepdim=True) + s["eps"]).sqrt() * w.double()
        part = x[..., :rot]
        pairs = part.unflatten(2, (-1, 2)) if case["interleaved"] else \
            part.unflatten(2, (2, -1)).transpose(2, 3)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        pairs = pairs if case["interleaved"] else pairs.transpose(2, 3)
        return torch.cat([pairs.flatten(2), x[..., rot:]], 2)

    def cached(cache, x, scale):
        got = cache.view(torch.float8_e4m3fn).double()
        got.view(-1, *got.shape[2:])[s["slots"]] = (x / scale.double()).clamp(-448, 448)
        return got

    return dict(q=of(s["q"], s["qw"]), key_cache=cached(s["key_cache"], of(s["k"], s["kw"]), s["ks"]),
                value_cache=cached(s["value_cache"], s["v"].double(), s["vs"]))
