"""The operators around the quantized linear layers of a decoder, as cases to measure.

norm       residual addition, root-mean-square norm and int8 codes with a scale for each token: what
           w4a8_gemm takes.
append     rotary positions on queries and keys, keys and values quantized to 4 bits for each token
           and head and written into a paged cache.
attention  softmax attention of new tokens over that cache, ragged over the sequences.

Cache layout, shared by the last two: uint8 [pages, kv_heads, page_size / 16, 16 * D + 128], where the last
axis is one unit of 16 tokens of one head:
  bytes [0, 8 D)        keys: for each token D / 2 bytes, the 32-bit words of eight channels in the AWQ
                        order (nibble i of a word holds channel [0, 2, 4, 6, 1, 3, 5, 7][i] of its eight);
  bytes [8 D, 16 D)     values: 16-bit halves of four channels (lowest nibble first), indexed
                        [token / 8][channel / (D / 8)][token % 8 / 2][channel % (D / 8) / 4][token % 2];
  bytes [16 D, +128)    for each token four fp16: key scale, key zero, value scale, value zero.
A code u in 0..15 stands for zero + u * scale.
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
ROPE_BASE = 10000.0


# --------------------------------------------------------------------------------------------- cases

def _norm(name, tokens, width, dtype, residual=True):
    return {"name": name, "op": "norm", "tokens": tokens, "width": width, "dtype": dtype, "residual": residual}


def _append(name, seqs, q_len, heads, kv_heads, dim, dtype, page, rot, interleaved):
    return {"name": name, "op": "append", "seqs": seqs, "q_len": q_len, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "page": page, "rot": rot, "interleaved": interleaved}


def _attention(name, seqs, q_len, kv_len, ragged, heads, kv_heads, dim, dtype, page, window=0):
    return {"name": name, "op": "attention", "seqs": seqs, "q_len": q_len, "kv_len": kv_len, "ragged": ragged,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "page": page, "window": window}


def listed():
    return [
        # one decode step of a few sequences: latency is all there is
        _norm("norm_decode", 8, 4096, "fp16"),
        # one prefill chunk of a 4096-wide model
        _norm("norm_prefill", 4096, 4096, "fp16"),
        # a long prefill at an odd width, bf16, the first layer's norm (no residual yet)
        _norm("norm_ragged", 7001, 11016, "bf16", residual=False),
        # one decode step of a full batch, grouped heads
        _append("append_decode", 64, 1, 32, 8, 128, "fp16", 64, 128, False),
        # prompts of a model with as many key heads as query heads, part of the head rotated, pairs interleaved
        _append("append_prefill", 5, 1633, 32, 32, 128, "bf16", 16, 64, True),
        # the smallest call: one short chat, one new token
        _attention("decode_short", 1, 1, 177, False, 32, 8, 128, "fp16", 16),
        # one sequence at the 4096 tokens of a 7B model's context, a key head for each query head
        _attention("decode_single", 1, 1, 4096, False, 32, 32, 128, "fp16", 64),
        # a serving batch: every sequence at another length
        _attention("decode_ragged", 64, 1, 8191, True, 32, 8, 128, "fp16", 64),
        # long contexts, the largest cache
        _attention("decode_long", 16, 1, 32768, False, 32, 8, 128, "bf16", 128),
        # a few drafted tokens verified at once, small heads, small pages
        _attention("verify", 24, 5, 2050, True, 16, 8, 64, "bf16", 16),
        # long sequences that look back over a sliding window only
        _attention("decode_window", 32, 1, 16000, True, 32, 8, 128, "bf16", 32, window=4096),
        # one chunk of a long prompt, against itself and what is in the cache before it
        _attention("prefill_chunk", 2, 1024, 4500, True, 32, 8, 128, "fp16", 64),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], uniform in its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("norm", "append", "attention", "attention"))
    dtype = rng.choice(("fp16", "bf16"))
    if op == "norm":
        width = 8 * (2 * _spread(rng, 8, 1024) + 1)  # the widths are odd multiples of 8
        tokens = _spread(rng, 1, min(16384, 7001 * 11016 // width))
        return {k: v for k, v in _norm("", tokens, width, dtype, rng.random() < 0.7).items() if k != "name"}
    kv_heads = rng.choice((1, 2, 4, 8, 16, 32))
    per = rng.choice((1, 2, 4, 5, 7, 8)) if kv_heads <= 8 else rng.choice((1, 2))
    dim = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        most = 5 * 1633 * 32 * 3 // (kv_heads * (per + 2))
        q_len = 1 if rng.random() < 0.5 else _spread(rng, 2, min(2048, most))
        rot = rng.choice((dim, dim // 2, dim // 4))
        return {k: v for k, v in _append("", _spread(rng, 1, max(1, min(256, most // q_len))), q_len, kv_heads * per,
                                         kv_heads, dim, dtype, page, rot, rng.random() < 0.5).items() if k != "name"}
    kv_len = _spread(rng, 1, 32768)
    kind = rng.random()
    q_len = 1 if kind < 0.6 else min(kv_len, _spread(rng, 2, 8) if kind < 0.8 else _spread(rng, 16, 1024))
    most = min(16 * 32768 * 8 * 128 // (kv_len * kv_heads * dim), 2 * 1024 * 4500 * 32 * 128 // (q_len * kv_len * kv_heads * per * dim))
    if most < 1:  # too much for one sequence: fewer new tokens
        q_len, most = 1, 1
    seqs = _spread(rng, 1, max(1, min(128, most)))
    window = _spread(rng, 1, kv_len) if rng.random() < 0.2 else 0
    return {k: v for k, v in _attention("", seqs, q_len, kv_len, rng.random() < 0.6, kv_heads * per, kv_heads, dim,
                                        dtype, page, window).items() if k != "name"}


def _lengths(case):
    """(context length, new tokens) of each sequence: the lengths of a ragged batch spread over 1..kv_len."""
    n = case["seqs"]
    lens = [case["kv_len"]] * n
    if case["ragged"]:
        lens = [1 + int((case["kv_len"] - 1) * ((0.91 + 0.6180339887 * b) % 1.0)) for b in range(n)]
    return [(length, min(case["q_len"], length)) for length in lens]


def work(case):
    if case["op"] == "norm":
        m, k = case["tokens"], case["width"]
        # x, the residual in and out, the codes; the scales and the weight
        return {"bytes": m * k * (7 if case["residual"] else 3) + 4 * m + 2 * k, "flops": 6 * m * k}
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        t = case["seqs"] * case["q_len"]
        # q, k, v in; q, the cache entries and their values out; the rows of the table, positions and slots
        moved = t * (2 * heads * dim * 2 + kv_heads * (2 * dim * 2 + dim + 8 + 2 * dim * 2)) + t * (4 * case["rot"] + 12)
        return {"bytes": moved, "flops": t * (3 * (heads + kv_heads) * case["rot"] + 12 * kv_heads * dim)}
    cells = pairs = rows = 0
    for length, new in _lengths(case):
        rows += new
        window = case["window"] or length
        cells += min(length, window + new - 1)
        first = length - new  # the position of the first new token
        if window >= length:
            pairs += new * first + new * (new + 1) // 2
        else:
            pairs += sum(min(window, first + i + 1) for i in range(new))
    pages = sum(-(-length // case["page"]) for length, _ in _lengths(case))
    return {"bytes": cells * kv_heads * (dim + 8) + rows * heads * dim * 4 + 4 * pages + 8 * case["seqs"],
            "flops": 4 * pairs * heads * dim}


# ------------------------------------------------------------------------------------------ preparing

def _table(positions, rot, device):
    """cos and sin of every position, fp32 [positions, rot]: rot / 2 cosines, then rot / 2 sines."""
    freq = ROPE_BASE ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), dim=1).float()


def _pages(lengths, page, gen, device):
    """A block table for sequences of these lengths whose pages lie anywhere in a pool somewhat larger."""
    need = [-(-length // page) for length in lengths]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device=device).int()
    first = torch.tensor([0] + need, device=device).cumsum(0)[:-1]
    column = torch.arange(max(need), device=device)
    return order[(first[:, None] + column).clamp(max=pool - 1)].contiguous(), pool


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    s = dict(case)
    if case["op"] == "norm":
        m, k = case["tokens"], case["width"]
        x = normal(m, k)
        x[:, :: max(8, k // 5)] *= 20.0  # a few channels far above the others, as hidden states have them
        s["x"] = x.to(dtype)
        s["weight"] = (1.0 + 0.2 * normal(k)).to(dtype)
        s["res"] = (2.0 * normal(m, k)).to(dtype) if case["residual"] else None
        s["values"] = torch.empty((m, k), dtype=dtype, device=device)
        return s
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    unit = 16 * dim + 128
    if case["op"] == "append":
        n, q_len = case["seqs"], case["q_len"]
        t = n * q_len
        # q, k and v are the columns of one projection's output
        qkv = normal(t, (heads + 2 * kv_heads) * dim)
        qkv[:, heads * dim + 5 :: dim] *= 6.0  # one channel of every head is larger
        s["qkv"] = qkv.to(dtype)
        start = [(37 * b) % 501 for b in range(n)]
        table, pool = _pages([a + q_len for a in start], page, gen, device)
        pos = torch.tensor(start, device=device)[:, None] + torch.arange(q_len, device=device)
        s["slots"] = (table.gather(1, pos // page).long() * page + pos % page).reshape(-1)
        s["positions"] = pos.reshape(-1).int()
        s["table"] = _table(1 << 13, case["rot"], device)
        s["cache"] = torch.zeros((pool, kv_heads, page // 16, unit), dtype=torch.uint8, device=device)
        return s
    lengths = _lengths(case)
    s["block_table"], pool = _pages([length for length, _ in lengths], page, gen, device)
    s["kv_len"] = torch.tensor([length for length, _ in lengths], dtype=torch.int32, device=device)
    new = torch.tensor([n for _, n in lengths], device=device)
    s["q_start"] = torch.cat((new.new_zeros(1), new.cumsum(0))).int()
    rows = sum(n for _, n in lengths)
    s["max_q"] = max(n for _, n in lengths)
    s["q"] = (2.5 * normal(rows, heads, dim)).to(dtype)
    # codes as keys and values of normal distribution give them, and their scales and zeros
    cache = torch.empty((pool, kv_heads, page // 16, unit), dtype=torch.uint8, device=device)
    code = torch.randn(cache[..., : 16 * dim].shape, generator=gen, device=device, dtype=torch.float16)
    code = code.mul_(2.7).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
    more = torch.randn(code.shape, generator=gen, device=device, dtype=torch.float16)
    cache[..., : 16 * dim] = code.bitwise_or_(more.mul_(2.7).add_(7.5).round_().clamp_(0, 15).to(torch.uint8).mul_(16))
    meta = cache[..., 16 * dim :].view(torch.float16).unflatten(-1, (16, 2, 2))
    sigma = torch.exp(0.25 * normal(*meta.shape[:-1]))
    meta[..., 0] = (sigma / 2.7).half()
    meta[..., 1] = (-7.5 * sigma / 2.7 + 0.05 * normal(*sigma.shape)).half()
    s["cache"] = cache
    return s


# ------------------------------------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    if s["op"] == "append":
        return _own_append(s) if own else _plain_append(s)
    return _own_attention(s) if own else _plain_attention(s)


def _own_norm(s):
    from bit_weight_only_awq_gb300 import awq
    xq, s_tok, res = awq.w4a8_rmsnorm_quant(s["x"], s["weight"], residual=s["res"], eps=EPS)
    torch.mul(xq, s_tok[:, None], out=s["values"])  # what the codes stand for
    return {"values": s["values"], "s_tok": s_tok, "res": res}


def _own_append(s):
    from bit_weight_only_awq_gb300 import awq
    heads, kv_heads, dim = s["heads"], s["kv_heads"], s["dim"]
    q, k, v = s["qkv"].unflatten(1, (heads + 2 * kv_heads, dim)).split((heads, kv_heads, kv_heads), dim=1)
    q = awq.kv4_append(s["cache"], k, v, s["positions"], s["slots"], s["table"], q=q, interleaved=s["interleaved"])
    k, v = awq.kv4_gather(s["cache"], s["slots"], dtype=q.dtype)
    return {"q": q, "k": k, "v": v}


def _own_attention(s):
    from bit_weight_only_awq_gb300 import awq
    return awq.kv4_attention(s["q"], s["cache"], s["block_table"], s["kv_len"], q_start=s["q_start"],
                             max_q=s["max_q"], window=s["window"])


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    # the codes of h * rstd * weight do not depend on rstd: it divides out of value and scale
    t = h * s["weight"].float()
    step = t.abs().amax(dim=1, keepdim=True) / torch.full((1, 1), 127.0, device=t.device)
    code = torch.where(step > 0, torch.round(t / step), torch.zeros_like(t)).clamp(-128, 127)
    s_tok = step * rstd
    res = h.to(s["x"].dtype) if s["res"] is not None else None
    return {"values": (code * s_tok).to(s["x"].dtype), "s_tok": s_tok[:, 0], "res": res}


def _rotate(x, cos, sin, interleaved):
    """x fp32 [tokens, heads, dim]; cos, sin [tokens, 1, rot / 2]."""
    half = cos.shape[-1]
    head, rest = x[..., : 2 * half], x[..., 2 * half :]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((head, rest), dim=-1)


def _quantize(x):
    """Codes (fp32 0..15), scale and zero (fp16) of each head of each token."""
    low, high = x.amin(dim=-1, keepdim=True), x.amax(dim=-1, keepdim=True)
    scale = ((high - low) / torch.full_like(low, 15.0)).half()
    zero = low.half()
    code = torch.round((x - zero.float()) / scale.float()).clamp(0, 15)
    return torch.where(scale > 0, code, torch.zeros_like(code)), scale, zero


def _plain_append(s):
    heads, kv_heads, dim, page = s["heads"], s["kv_heads"], s["dim"], s["page"]
    q, k, v = s["qkv"].float().unflatten(1, (heads + 2 * kv_heads, dim)).split((heads, kv_heads, kv_heads), dim=1)
    cos, sin = s["table"][s["positions"].long()][:, None].chunk(2, dim=-1)
    q = _rotate(q, cos, sin, s["interleaved"])
    (ku, ks, kz), (vu, vs, vz) = _quantize(_rotate(k, cos, sin, s["interleaved"])), _quantize(v)
    cache, slots = s["cache"], s["slots"]
    at, unit, token = slots // page, slots % page // 16, slots % 16
    # keys: nibble i of a word is channel [0, 2, 4, 6, 1, 3, 5, 7][i], so byte j of it is channels (0, 4, 1, 5)[j] and + 2
    word = ku.to(torch.uint8).unflatten(-1, (-1, 8))
    packed = (word[..., [0, 4, 1, 5]] | word[..., [2, 6, 3, 7]] << 4).flatten(-2)
    cache[..., : 8 * dim].unflatten(-1, (16, dim // 2))[at, :, unit, token] = packed
    word = vu.to(torch.uint8).unflatten(-1, (8, dim // 32, 2, 2))
    packed = word[..., 0] | word[..., 1] << 4
    view = cache[..., 8 * dim : 16 * dim].unflatten(-1, (2, 8, 4, dim // 32, 2, 2))
    view[at, :, unit, token // 8, :, token % 8 // 2, :, token % 2] = packed
    meta = cache[..., 16 * dim :].view(torch.float16).unflatten(-1, (16, 4))
    meta[at, :, unit, token] = torch.cat((ks, kz, vs, vz), dim=-1)
    dtype = s["qkv"].dtype
    return {"q": q.to(dtype), "k": (kz.float() + ku * ks.float()).to(dtype), "v": (vz.float() + vu * vs.float()).to(dtype)}


def _read(cache, dim):
    """fp32 keys and values [..., 16, dim] of units [..., 16 * dim + 128]."""
    keys = cache[..., : 8 * dim].unflatten(-1, (16, dim // 8, 4))
    nibbles = torch.stack((keys & 15, keys >> 4), dim=-1).flatten(-2)
    keys = nibbles[..., [0, 4, 1, 5, 2, 6, 3, 7]].flatten(-2)
    values = cache[..., 8 * dim : 16 * dim].unflatten(-1, (2, 8, 4, dim // 32, 2, 2))
    values = torch.stack((values & 15, values >> 4), dim=-1).flatten(-2)  # [s, g, t, J, parity, 4]
    values = values.movedim((-4, -2), (-5, -4)).flatten(-6, -4).flatten(-3, -1)  # [(s, t, parity), (g, J, 4)]
    meta = cache[..., 16 * dim :].view(torch.float16).unflatten(-1, (16, 4)).float()
    ks, kz, vs, vz = meta.split(1, dim=-1)
    return kz + ks * keys.float(), vz + vs * values.float()


def _plain_attention(s):
    heads, kv_heads, dim = s["heads"], s["kv_heads"], s["dim"]
    per, n, most = heads // kv_heads, s["seqs"], s["max_q"]
    units = s["cache"][s["block_table"].long()]  # [seqs, pages, kv_heads, units, bytes]
    units = units.movedim(2, 1).flatten(2, 3)
    keys, values = (x.flatten(2, 3) for x in _read(units, dim))  # [seqs, kv_heads, tokens, dim]
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    row = torch.arange(most, device=new.device)
    fits = row < new[:, None]
    index = (s["q_start"][:-1, None] + row).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"].float()[index].unflatten(2, (kv_heads, per)).movedim(2, 1).flatten(2, 3)  # [seqs, kv_heads, most * per, dim]
    score = torch.matmul(q, keys.transpose(2, 3)) * (1.0 / math.sqrt(dim))
    position = s["kv_len"].long()[:, None] - new[:, None] + row  # [seqs, most]
    key = torch.arange(keys.shape[2], device=new.device)
    seen = key <= position[..., None]
    if s["window"]:
        seen = seen & (key > position[..., None] - s["window"])
    seen = seen[:, None, :, None].expand(n, 1, most, per, key.shape[0]).flatten(2, 3)
    score = score.masked_fill(~seen, float("-inf"))
    top = score.amax(dim=-1, keepdim=True).clamp(min=-3.0e38)
    weight = torch.exp(score - top)
    out = torch.matmul(weight, values) / weight.sum(dim=-1, keepdim=True)
    out = out.unflatten(2, (most, per)).movedim(2, 1).flatten(2, 3)  # [seqs, most, heads, dim]
    return out[fits].to(s["q"].dtype)


# ---------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() + (s["res"].double() if s["res"] is not None else 0.0)
        y = h * s["weight"].double() / torch.sqrt(h.square().sum(1, keepdim=True) / h.shape[1] + EPS)
        scale = torch.linalg.vector_norm(y, ord=math.inf, dim=1, keepdim=True) / 127
        values = torch.round(y / scale) * scale
        return {"values": values, "s_tok": scale[:, 0], "res": h if s["res"] is not None else None}
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        x = s["qkv"].double().reshape(-1, heads + 2 * kv_heads, dim)
        rot = case["rot"]
        # a rotation in the plane is a product with exp(i angle)
        angle = s["positions"].double()[:, None] * ROPE_BASE ** (-torch.arange(rot // 2, device=x.device).double() * 2 / rot)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        first = torch.arange(rot // 2, device=x.device)
        a, b = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + rot // 2)
        qk = x[:, : heads + kv_heads].clone()
        z = torch.complex(qk[..., a], qk[..., b]) * turn
        qk[..., a], qk[..., b] = z.real, z.imag
        found = {"q": qk[:, :heads]}
        for name, y in (("k", qk[:, heads:]), ("v", x[:, heads + kv_heads :])):
            zero = y.min(dim=2, keepdim=True).values
            step = ((y.max(dim=2, keepdim=True).values - zero) / 15).half().double()
            zero = zero.half().double()
            found[name] = zero + step * torch.round((y - zero) / step).clamp(0, 15)
        return found
    per, page = heads // kv_heads, case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    channel = torch.arange(dim, device=out.device)
    token16 = torch.arange(16, device=out.device)[:, None]
    # where each code is: its byte of the unit, and whether it is the byte's high nibble
    slot = channel % 8 // 2 + 4 * (channel % 2)
    key_byte = token16 * (dim // 2) + channel // 8 * 4 + slot // 2
    wide = dim // 8
    half = ((token16 // 8 * 8 + channel // wide) * 4 + token16 % 8 // 2) * (dim // 32) + channel % wide // 4
    value_byte = 8 * dim + (half * 2 + token16 % 2) * 2 + channel % 4 // 2
    begin = 0
    for b, (length, new) in enumerate(_lengths(case)):
        end = begin + new
        pages = s["block_table"][b, : -(-length // page)].long()
        units = s["cache"][pages].transpose(0, 1).reshape(kv_heads, -1, 16 * dim + 128)
        first = max(0, length - new - case["window"] + 1) // 16 if case["window"] else 0
        units = units[:, first : -(-length // 16)]
        meta = units[..., 16 * dim :].contiguous().view(torch.float16).double().reshape(kv_heads, -1, 4)
        k = (units[..., key_byte] >> (4 * (slot % 2)).to(torch.uint8) & 15).double().reshape(kv_heads, -1, dim)
        v = (units[..., value_byte] >> (4 * (channel % 2)).to(torch.uint8) & 15).double().reshape(kv_heads, -1, dim)
        k, v = k * meta[..., 0:1] + meta[..., 1:2], v * meta[..., 2:3] + meta[..., 3:4]
        q = s["q"][begin:end].double().reshape(new, kv_heads, per, dim)
        score = torch.einsum("ihgd,hjd->hgij", q, k) / dim ** 0.5
        at = torch.arange(length - new, length, device=out.device)[:, None]
        j = first * 16 + torch.arange(k.shape[1], device=out.device)
        hidden = (j > at) | ((at - j >= case["window"]) if case["window"] else (j < 0))
        weight = torch.softmax(score.masked_fill(hidden, -math.inf), dim=-1)
        out[begin:end] = torch.einsum("hgij,hjd->ihgd", weight, v).reshape(new, heads, dim)
        begin = end
    return out
