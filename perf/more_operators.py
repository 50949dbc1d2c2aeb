"""Timed cases of the operators around a serving step's linears and attention:
the residual's addition with RMS norm and FP8 output, the query / key norm with
rotary positions of several axes and cache store, products with 4-bit weights
and group scales, and log probabilities of given tokens with entropy and top
alternatives.

``own`` chooses between the operators' plain form (elementary torch
operations in 32 bits) and the framework's calls; both take what ``prepare``
makes.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one decode step of a few requests before the QKV linear: latency alone
        dict(name="norm_decode", op="norm", tokens=4, width=4096, mode="block", residual=True,
             both=False),
        # a prompt chunk before a block-scaled linear, one token short of 8192
        dict(name="norm_prompt", op="norm", tokens=8191, width=4096, mode="block", residual=True,
             both=False),
        # a wide model's chunk with a scale per token, the unquantized norm kept too
        dict(name="norm_tokens", op="norm", tokens=2049, width=7168, mode="row", residual=True,
             both=True),
        # a decode step behind images: time, height and width in sections
        dict(name="axes_decode", op="axes", tokens=16, q_heads=32, kv_heads=8, dim=128, rot=128,
             sections="16 24 24", in_turn=False, interleaved=False, page=16, reach=32768),
        # a prompt of text and images, the axes taken in turn over the frequencies
        dict(name="axes_prompt", op="axes", tokens=8191, q_heads=32, kv_heads=8, dim=128, rot=128,
             sections="24 20 20", in_turn=True, interleaved=False, page=16, reach=32768),
        # one token through an attention-sized projection: the smallest product
        dict(name="int4_token", op="int4", rows=1, n=4096, k=4096, group=128, zeros=False),
        # one token through an MLP's down projection, groups of 64 with zero points
        dict(name="int4_down", op="int4", rows=1, n=4096, k=14336, group=64, zeros=True),
        # a decode batch of ragged size through an output head
        dict(name="int4_head", op="int4", rows=13, n=128000, k=4096, group=128, zeros=True),
        # a prompt chunk through the up projection of the same weights
        dict(name="int4_prompt", op="int4", rows=1000, n=11008, k=4096, group=128, zeros=False),
        # one decoded token, alternatives for the user
        dict(name="probs_token", op="probs", rows=1, vocab=128000, k=20, dtype="bf16"),
        # a decode batch with an odd vocabulary, fp32 logits, part of them masked
        dict(name="probs_batch", op="probs", rows=61, vocab=100003, k=5, dtype="f32"),
        # scoring a prompt: every position of a chunk
        dict(name="probs_prompt", op="probs", rows=2047, vocab=128000, k=1, dtype="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number of lo..hi, its logarithm spread evenly."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


HEADS = ((32, 8), (64, 8), (16, 2), (8, 8), (12, 1), (28, 4), (5, 5))


def draw(rng):
    op = rng.choice(["norm", "axes", "int4", "int4", "probs", "probs"])
    if op == "norm":
        width = 128 * _between(rng, 1, 128)
        return dict(op=op, width=width, tokens=_between(rng, 1, min(8191, 2 ** 24 // width)),
                    mode=rng.choice(["block", "block", "row", "tensor", "none"]),
                    residual=rng.random() < 0.8, both=rng.random() < 0.3)
    if op == "axes":
        hq, hk = rng.choice(HEADS)
        dim = rng.choice([64, 80, 128, 128, 256])
        rot = rng.choice([dim, dim, dim // 2 // 16 * 16])
        axes, half = rng.choice([1, 2, 3, 3, 3, 4]), rot // 2
        in_turn = rng.random() < 0.5
        # in turn, an axis but the first has at most its share of the frequencies
        most = half // axes if in_turn else half
        sections, left = [], half
        for _ in range(axes - 1):
            sections.append(rng.randint(0, min(most, left)))
            left -= sections[-1]
        cost = hq * dim / 4096.0
        return dict(op=op, tokens=_between(rng, 1, int(8191 / max(1.0, 1.3 * cost))), q_heads=hq,
                    kv_heads=hk, dim=dim, rot=rot, sections=" ".join(map(str, [left] + sections)),
                    in_turn=in_turn, interleaved=rng.random() < 0.3,
                    page=rng.choice([1, 7, 16, 16, 64]), reach=_between(rng, 9000, 65536))
    if op == "int4":
        rows = rng.choice([1, 1, _between(rng, 1, 16), _between(rng, 1, 64), _between(rng, 1, 1000)])
        k = 128 * _between(rng, 1, 128)
        n = _between(rng, 16, min(128000, 2 ** 28 // k, 2 ** 35 // (k * rows)))
        return dict(op=op, rows=rows, n=n if rng.random() < 0.3 else max(16, n // 16 * 16), k=k,
                    group=rng.choice([32, 64, 128, 128]), zeros=rng.random() < 0.5)
    vocab = _between(rng, 1000, 200000)
    dtype = rng.choice(["bf16", "f32"])
    return dict(op=op, vocab=vocab, dtype=dtype, k=rng.choice([0, 1, 5, 20, 64]),
                rows=_between(rng, 1, min(2047, 2 ** (27 if dtype == "bf16" else 26) // vocab)))


# ---- inputs --------------------------------------------------------------------

def _sections(case):
    """Rotated pairs of each axis."""
    return [int(n) for n in case["sections"].split()]


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV)


def _one(value):
    return torch.tensor([value], dtype=torch.float32, device=DEV)


def _codes(g, *shape):
    """E4M3 codes of normal values at a scale of 1/32, as raw bytes."""
    return (_normal(g, *shape) * 32).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    return _PREPARE[case["op"]](case, torch.Generator(device=DEV).manual_seed(seed))


def _prepare_norm(case, g):
    t, h, mode = case["tokens"], case["width"], case["mode"]
    x, r = _normal(g, t, h), _normal(g, t, h) * 2
    loud = _ints(g, 0, h, max(1, h // 500))           # channels far above the others
    r[:, loud] *= 30
    scales = dict(block=(t, h // 128), row=(t,), tensor=(1,), none=(0,))[mode]
    s = dict(case=case, x=x.to(torch.bfloat16),
             residual=r.to(torch.bfloat16) if case["residual"] else None,
             weight=(1 + 0.2 * _normal(g, h)).to(torch.bfloat16), eps=1e-6, scale=None,
             residual_out=torch.empty((t, h), dtype=torch.bfloat16, device=DEV)
             if case["residual"] else None,
             y=torch.empty((t, h), dtype=torch.bfloat16, device=DEV)
             if case["both"] or mode == "none" else None)
    if mode != "none":
        s["q"] = torch.empty((t, h), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(scales, dtype=torch.float32, device=DEV)
    if mode == "tensor":
        s["scale"] = _one(12 / 448)                   # calibrated; the loudest values clip
    return s


def _positions(g, axes, t, reach):
    """Positions [axes, t] of text with pictures in it: a picture holds the first
    axis and counts its rows and columns on the others; text counts on all."""
    i = torch.arange(t, device=DEV)
    start = int(_ints(g, 0, max(1, reach - t), 1))
    side, words = 24, 100
    block = side * side + words
    inside, before = i % block, i // block * (side + words)
    picture = inside < side * side
    text = inside - side * side + side
    rows = []
    for a in range(axes):
        step = (torch.zeros_like(i), inside // side, inside % side, inside % 3)[a]
        rows.append(start + before + torch.where(picture, step, text))
    return torch.stack(rows) % reach


def _prepare_axes(case, g):
    t, hq, hk, d, page = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim", "page"))
    rot, reach, axes = case["rot"], case["reach"], len(_sections(case))
    # queries, keys and values are slices of the projection's one output row
    qkv = _normal(g, t, hq + 2 * hk, d)
    qkv[:, hq:hq + hk, :4] *= 20
    qkv = qkv.to(torch.bfloat16)
    freq = 1000000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(reach, dtype=torch.float64, device=DEV)[:, None] * freq
    blocks = 2 * -(-t // page) + 3
    pool = torch.randperm(blocks, generator=g, device=DEV)
    i = torch.arange(t, device=DEV)
    return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:],
                qw=(1 + 0.1 * _normal(g, d)).to(torch.bfloat16),
                kw=(1 + 0.1 * _normal(g, d)).to(torch.bfloat16),
                cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
                positions=_positions(g, axes, t, reach), slots=pool[i // page] * page + i % page,
                key_cache=_codes(g, blocks, page, hk, d), value_cache=_codes(g, blocks, page, hk, d),
                ks=_one(16 / 448), vs=_one(1.0), eps=1e-6,
                out=torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV))


def _prepare_int4(case, g):
    m, n, k, group = (case[key] for key in ("rows", "n", "k", "group"))
    # 8 values to 4 bytes: the even ones' bits in the lower two, the odd ones' in the upper two
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=DEV)
    step = max(1, 2 ** 26 // k)
    for i in range(0, n, step):
        j = min(n, i + step)
        v = (_normal(g, j - i, k // 8, 2, 2, 2) * 2.7 + 7.7).round_().clamp_(0, 15).to(torch.uint8)
        v = v.permute(0, 1, 4, 2, 3)                  # [.., value parity, byte, half]
        codes[i:j] = (v[..., 0] | v[..., 1] << 4).reshape(j - i, k // 2)
    x = _normal(g, m, k)
    x[:, _ints(g, 0, k, max(1, k // 500))] *= 20      # channels far above the others
    return dict(case=case, x=x.to(torch.bfloat16), codes=codes,
                scales=0.008 * (0.5 + _uniform(g, n, k // group)),
                zeros=(_normal(g, n, k // group) + 7.5).round().clamp(0, 15).to(torch.uint8)
                if case["zeros"] else None,
                out=torch.empty((m, n), dtype=torch.bfloat16, device=DEV))


def _prepare_probs(case, g):
    t, v, k = case["rows"], case["vocab"], case["k"]
    x = _normal(g, t, v) * 2.5
    at = _ints(g, 0, v, t, 4)
    x.scatter_add_(1, at, 8 + 4 * _normal(g, t, 4))   # a few likely ones
    if case["dtype"] == "f32":                        # a grammar's mask on every fourth row
        x[::4].masked_fill_(_uniform(g, len(x[::4]), v) < 0.7, -math.inf)
    # mostly what was sampled, here and there an unlikely one or padding
    tokens = torch.where(_uniform(g, t) < 0.7, at[:, 0], _ints(g, 0, v, t))
    tokens[_uniform(g, t) < 0.02] = -1
    return dict(case=case, logits=x.to(torch.bfloat16) if case["dtype"] == "bf16" else x,
                tokens=tokens, scale=1 / 0.8,
                logprobs=torch.empty(t, dtype=torch.float32, device=DEV),
                ranks=torch.empty(t, dtype=torch.int32, device=DEV),
                entropy=torch.empty(t, dtype=torch.float32, device=DEV),
                lse=torch.empty(t, dtype=torch.float32, device=DEV),
                top=torch.empty((t, k), dtype=torch.float32, device=DEV),
                ids=torch.empty((t, k), dtype=torch.int32, device=DEV))


_PREPARE = dict(norm=_prepare_norm, axes=_prepare_axes, int4=_prepare_int4, probs=_prepare_probs)


# ---- one pass --------------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _own_norm(s):
    import fp8_w8a8_block_amd as fp8
    mode = s["case"]["mode"]
    if mode == "none":
        fp8.add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=s["eps"], out=s["y"],
                         residual_out=s["residual_out"])
    else:
        fp8.add_rms_norm_quant(s["x"], s["weight"], residual=s["residual"], eps=s["eps"],
                               scale_mode=mode, scale=s["scale"], q=s["q"],
                               scales=None if mode == "tensor" else s["scales"], out=s["y"],
                               residual_out=s["residual_out"])
    return _norm_outputs(s)


def _norm_outputs(s):
    mode = s["case"]["mode"]
    return dict(residual=s["residual_out"], y=s["y"],
                q=None if mode == "none" else s["q"].view(torch.float8_e4m3fn),
                scales=s["scales"] if mode in ("block", "row") else None)


def _own_axes(s):
    import fp8_w8a8_block_amd as fp8
    case = s["case"]
    q = fp8.qk_norm_mrope_cache(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["cos_sin"],
                                s["positions"], _sections(case), s["slots"], s["key_cache"],
                                s["value_cache"], s["ks"], s["vs"], eps=s["eps"],
                                in_turn=case["in_turn"], interleaved=case["interleaved"],
                                query_out=s["out"])
    return _axes_outputs(s, q)


def _axes_outputs(s, q):
    return dict(q=q, key_cache=s["key_cache"].view(torch.float8_e4m3fn),
                value_cache=s["value_cache"].view(torch.float8_e4m3fn))


def _own_int4(s):
    import fp8_w8a8_block_amd as fp8
    return dict(out=fp8.int4_linear(s["x"], s["codes"], s["scales"], zeros=s["zeros"],
                                    out=s["out"]))


def _own_probs(s):
    import fp8_w8a8_block_amd as fp8
    fp8.token_logprobs(s["logits"], s["tokens"], k=s["case"]["k"], scale=s["scale"],
                       logprobs=s["logprobs"], ranks=s["ranks"], entropy=s["entropy"],
                       lse=s["lse"], top_logprobs=s["top"], top_ids=s["ids"])
    return _probs_outputs(s)


def _probs_outputs(s):
    return {key: s[key] for key in ("logprobs", "ranks", "entropy", "lse", "top", "ids")}


def _plain_norm(s):
    case, t = s["case"], s["x"].float()
    if s["residual"] is not None:
        # what later layers read is what is normalized: the sum in bf16
        s["residual_out"].copy_(t + s["residual"].float())
        t = s["residual_out"].float()
    y = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    if s["y"] is not None:
        s["y"].copy_(y)
    if case["mode"] == "none":
        return _norm_outputs(s)
    if case["mode"] == "tensor":
        z = y / s["scale"]
    else:
        groups = y.view(y.shape[0], -1, 128) if case["mode"] == "block" else y[:, None]
        scales = groups.abs().amax(-1) / 448
        s["scales"].copy_(scales.view(s["scales"].shape))
        z = (groups / torch.where(scales > 0, scales, 1.0)[..., None]).view(y.shape)
    s["q"].copy_(z.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    return _norm_outputs(s)


def _axis_of(case):
    """Axis of each rotated pair: the sections one after the other, or the axes in
    turn (pair i belongs to axis i modulo their number while that axis has pairs
    left, else to the first)."""
    sections = _sections(case)
    n = len(sections)
    if not case["in_turn"]:
        return [a for a in range(n) for _ in range(sections[a])]
    return [i % n if i < n * sections[i % n] else 0 for i in range(case["rot"] // 2)]


def _plain_axes(s):
    case = s["case"]
    d, rot = case["dim"], case["rot"]
    half = rot // 2
    pair = torch.arange(half, device=DEV)
    row = s["positions"][torch.tensor(_axis_of(case), device=DEV)].t()      # [T, half]
    cos, sin = s["cos_sin"][row, pair].unsqueeze(1), s["cos_sin"][row, half + pair].unsqueeze(1)

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
    return _axes_outputs(s, s["out"])


def _weights(codes):
    """The 4-bit values [N, K] of packed codes, as bytes."""
    b = codes.view(codes.shape[0], -1, 2, 2)          # [.., value parity, byte]
    v = torch.stack([b & 15, b >> 4], -1)             # [.., value parity, byte, half]
    return v.permute(0, 1, 3, 4, 2).reshape(codes.shape[0], -1)


def _plain_int4(s):
    n, k, group = (s["case"][key] for key in ("n", "k", "group"))
    w = _weights(s["codes"]).float().view(n, -1, group)
    w = (w - (8.0 if s["zeros"] is None else s["zeros"].float()[..., None])) * s["scales"][..., None]
    s["out"].copy_(s["x"].float() @ w.view(n, k).t())
    return dict(out=s["out"])


def _plain_probs(s):
    case = s["case"]
    v, k = case["vocab"], case["k"]
    x = s["logits"].float() * s["scale"]
    most = x.amax(-1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(-1)
    lse = total.log() + most[:, 0]
    s["lse"].copy_(lse)
    s["entropy"].copy_(total.log() - torch.where(e > 0, e * (x - most), 0.0).sum(-1) / total)
    given, token = s["tokens"] >= 0, s["tokens"].clamp(min=0)[:, None]
    s["logprobs"].copy_(torch.where(given, x.gather(1, token)[:, 0] - lse, 0.0))
    # the order is that of the logits themselves: the scaled ones may round together
    s["ranks"].copy_(torch.where(given, (s["logits"] > s["logits"].gather(1, token)).sum(-1), -1))
    if k:
        # whole numbers in the values' order, the lowest index first among equal ones
        bits = (s["logits"].float() + 0.0).view(torch.int32).long()
        key = torch.where(bits >= 0, bits, -2 ** 31 - bits) * 2 ** 32
        key = key + (v - 1 - torch.arange(v, device=DEV))
        ids = v - 1 - (torch.topk(key, k, dim=-1).values & (2 ** 32 - 1))
        s["ids"].copy_(ids)
        s["top"].copy_(x.gather(1, ids) - lse[:, None])
    return _probs_outputs(s)


_PLAIN = dict(norm=_plain_norm, axes=_plain_axes, int4=_plain_int4, probs=_plain_probs)
_OWN = dict(norm=_own_norm, axes=_own_axes, int4=_own_int4, probs=_own_probs)


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    if case["op"] == "norm":
        t, h = case["tokens"], case["width"]
        row = 2.0 * h + (4.0 * h if case["residual"] else 0.0)
        row += 2.0 * h if case["both"] or case["mode"] == "none" else 0.0
        row += dict(block=h + h / 32.0, row=h + 4.0, tensor=h, none=0.0)[case["mode"]]
        return dict(bytes=t * row + 2.0 * h, flops=t * h * 8.0)
    if case["op"] == "axes":
        t, hq, hk, d = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim"))
        row = 2.0 * (2 * hq + 2 * hk) * d + 2.0 * hk * d + 4.0 * case["rot"]
        return dict(bytes=t * (row + 8.0 * len(_sections(case)) + 8.0), flops=t * (hq + hk) * d * 9.0)
    if case["op"] == "int4":
        m, n, k, group = (case[key] for key in ("rows", "n", "k", "group"))
        scales = (5.0 if case["zeros"] else 4.0) * n * k / group
        return dict(bytes=n * k / 2.0 + scales + 2.0 * m * (n + k), flops=2.0 * m * n * k)
    t, v, k = case["rows"], case["vocab"], case["k"]
    return dict(bytes=t * ((2.0 if case["dtype"] == "bf16" else 4.0) * v + 24.0 + 8.0 * k),
                flops=6.0 * t * v)


# ---- the definitions in 64 bits ------------------------------------------------------

def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _exact_norm(s):
    mode, r = s["case"]["mode"], s["x"].double()
    residual = None
    if s["residual"] is not None:
        residual = r + s["residual"].double()
        r = residual.to(torch.bfloat16).double()      # two bf16 values: the sum in 64 bits is exact
    y = r / (r.square().sum(1, keepdim=True) / r.shape[1] + s["eps"]).sqrt() * s["weight"].double()
    q = scales = None
    if mode == "tensor":
        q = (y / s["scale"].double()).clamp(-448, 448)
    elif mode != "none":
        parts = y.unflatten(1, (-1, 128 if mode == "block" else y.shape[1]))
        top = parts.abs().max(2, keepdim=True).values / 448
        q = torch.where(top > 0, parts / top, parts).flatten(1)
        scales = top.view(s["scales"].shape)
    return dict(residual=residual, y=y if s["y"] is not None else None, q=q, scales=scales)


def _exact_axes(s):
    case = s["case"]
    rot = case["rot"]
    table = torch.complex(*s["cos_sin"].double().chunk(2, 1))
    turn = torch.stack([table[s["positions"][a], i] for i, a in enumerate(_axis_of(case))], 1)[:, None]

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


def _exact_int4(s):
    m, n, k, group = (s["case"][key] for key in ("rows", "n", "k", "group"))
    out, x = torch.empty((m, n), dtype=torch.float64, device=DEV), s["x"].double()
    at = torch.arange(k, device=DEV)
    byte = at // 8 * 4 + at % 2 * 2 + at % 8 // 4     # where each value's bits are
    shift = (at % 4 // 2 * 4).to(torch.uint8)
    step = max(1, 2 ** 27 // k)
    for i in range(0, n, step):
        w = (s["codes"][i:i + step][:, byte] >> shift & 15).double()
        zero = 8 if s["zeros"] is None else s["zeros"][i:i + step].repeat_interleave(group, 1).double()
        w = (w - zero) * s["scales"][i:i + step].double().repeat_interleave(group, 1)
        out[:, i:i + step] = x @ w.t()
    return dict(out=out)


def _exact_probs(s):
    k, parts = s["case"]["k"], []
    for x, token in zip(s["logits"].split(64), s["tokens"].split(64)):
        x = x.double() * s["scale"]
        lse = torch.logsumexp(x, 1)
        logp = x - lse[:, None]
        at = token.clamp(min=0)[:, None]
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k] if k else \
            token.new_zeros((len(x), 0))
        parts.append((torch.where(token < 0, 0.0, logp.gather(1, at)[:, 0]),
                      torch.where(token < 0, -1, (x > x.gather(1, at)).sum(1)).int(),
                      torch.special.entr(logp.exp()).sum(1), lse, logp.gather(1, order), order.int()))
    return dict(zip(("logprobs", "ranks", "entropy", "lse", "top", "ids"),
                    (torch.cat(p) for p in zip(*parts))))


_EXACT = dict(norm=_exact_norm, axes=_exact_axes, int4=_exact_int4, probs=_exact_probs)
