"""The feed-forward half of a decoder with experts, and fp8 linear layers, as cases to measure.

route    the router of a layer with experts: softmax over the experts' logits, the top_k of each token, and the plan
         that puts the chosen (token, expert) rows in the experts' order.
experts  a whole sparse feed-forward layer on 4-bit weights in the AWQ layout, from the router's logits on: route, the
         product with gate and up grouped by expert, silu(gate) * up, the product with down, the weighted sum of
         each token's rows.
fp8      a linear layer on e4m3 weights with an fp32 scale for each block of 128 x 128 and activations that are
         quantized to e4m3 with a scale for each token and 128 channels.

Ties of the router go to the lowest expert.  Rows of one expert keep the order of their tokens.
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
GROUP = 128
E4M3_MAX = 448.0


# --------------------------------------------------------------------------------------------- cases

def _route(name, tokens, experts, top_k, dtype, normalize=True):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "dtype": dtype,
            "normalize": normalize}


def _experts(name, tokens, experts, top_k, width, inner, dtype, symmetric=False, normalize=True):
    return {"name": name, "op": "experts", "tokens": tokens, "experts": experts, "top_k": top_k, "width": width,
            "inner": inner, "dtype": dtype, "symmetric": symmetric, "normalize": normalize}


def _fp8(name, tokens, inputs, outputs, dtype):
    return {"name": name, "op": "fp8", "tokens": tokens, "inputs": inputs, "outputs": outputs, "dtype": dtype}


def listed():
    return [
        # the router of one decode step of a few sequences: latency is all there is
        _route("route_decode", 3, 8, 2, "fp16"),
        # the router of a long prefill over many experts, logits kept in fp32, weights not normalized again
        _route("route_prefill", 8191, 128, 8, "fp32", normalize=False),
        # one token through a layer of 8 wide experts: two experts' weights are streamed
        _experts("experts_token", 1, 8, 2, 4096, 14336, "fp16"),
        # a few drafted tokens over many small experts, symmetric weights: hardly two rows share an expert
        _experts("experts_verify", 13, 64, 6, 2048, 1408, "bf16", symmetric=True),
        # one decode step of a serving batch: every expert has some rows, all weights are streamed
        _experts("experts_batch", 96, 8, 2, 4096, 14336, "fp16"),
        # a prefill chunk over many small experts: every expert's share another, none a whole tile
        _experts("experts_many", 4001, 128, 8, 2048, 768, "bf16", normalize=False),
        # a prefill chunk through 8 wide experts, the largest product
        _experts("experts_prefill", 4096, 8, 2, 4096, 14336, "fp16"),
        # one token through the attention projection of a 4096-wide model
        _fp8("fp8_token", 1, 4096, 6144, "bf16"),
        # one decode step of a batch through a down projection
        _fp8("fp8_batch", 48, 14336, 4096, "bf16"),
        # a prompt of odd length through a layer whose outputs end inside a block
        _fp8("fp8_ragged", 1111, 11008, 4072, "fp16"),
        # a prefill chunk through gate and up
        _fp8("fp8_prefill", 4096, 4096, 28672, "bf16"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], uniform in its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("route", "experts", "experts", "experts", "fp8", "fp8"))
    if op == "route":
        experts = rng.choice((4, 8, 16, 60, 64, 128, 160, 256))
        case = _route("", _spread(rng, 1, 8191 * 128 // max(128, experts)), experts, _spread(rng, 1, min(8, experts)),
                      rng.choice(("fp16", "bf16", "fp32")), rng.random() < 0.5)
    elif op == "experts":
        width, inner = 128 * _spread(rng, 2, 32), 128 * _spread(rng, 1, 112)
        experts = _spread(rng, 2, max(2, min(160, 8 * 4096 * 14336 // (width * inner))))
        top_k = _spread(rng, 1, min(8, experts))
        rows = min(32768, 8192 * 4096 * 14336 // (width * inner))
        case = _experts("", _spread(rng, 1, max(1, rows // top_k)), experts, top_k, width, inner,
                        rng.choice(("fp16", "bf16")), rng.random() < 0.3, rng.random() < 0.5)
    else:
        inputs, outputs = 16 * _spread(rng, 16, 896), 8 * _spread(rng, 16, 3584)
        most = 4096 * 4096 * 28672 // (inputs * outputs)
        case = _fp8("", _spread(rng, 1, max(1, min(8192, most))), inputs, outputs, rng.choice(("fp16", "bf16")))
    del case["name"]
    return case


def work(case):
    t = case["tokens"]
    if case["op"] == "fp8":
        k, n = case["inputs"], case["outputs"]
        blocks = -(-k // GROUP) * -(-n // GROUP)
        return {"bytes": 2 * t * k + n * k + 4 * blocks + 2 * t * n, "flops": 2 * t * n * k}
    e, top = case["experts"], case["top_k"]
    rows = t * top
    if case["op"] == "route":
        size = 4 if case["dtype"] == "fp32" else 2
        # logits in; experts and weights, offsets, order and places out
        return {"bytes": t * e * size + rows * 16 + 4 * (e + 1), "flops": t * e * 4}
    width, inner = case["width"], case["inner"]
    # experts that have a row, were the tokens' choices spread evenly
    active = min(e, rows, e * (1.0 - (1.0 - top / e) ** t))
    weight = 3 * width * inner * (0.5 + (2.0 if case["symmetric"] else 2.5) / GROUP)
    return {"bytes": round(active * weight) + 2 * t * e + 4 * t * width, "flops": rows * 6 * width * inner}


# ------------------------------------------------------------------------------------------ preparing

def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _logits(case, gen):
    """Logits of a router that prefers some experts; where there are many, two get nothing at all."""
    t, e = case["tokens"], case["experts"]
    bias = 0.6 * torch.randn(e, generator=gen, device="cuda")
    if e >= 16:
        bias[[e // 3, e - 1]] = -40.0
    return (bias + 1.2 * torch.randn(t, e, generator=gen, device="cuda")).to(DTYPES[case["dtype"]])


def _awq_weights(e, k, n, dtype, symmetric, gen):
    """Random codes of e layers [k, n] in the AWQ layout, zero points 6..9 (None for 8 everywhere), scales."""
    words = torch.randint(-2 ** 31, 2 ** 31, (e, k, n // 8), generator=gen, device="cuda", dtype=torch.int32)
    zeros = None
    if not symmetric:
        zeros = torch.randint(-2 ** 31, 2 ** 31, (e, k // GROUP, n // 8), generator=gen, device="cuda", dtype=torch.int32)
        zeros = (zeros & 0x33333333) + 0x66666666
    scales = 0.2 / math.sqrt(k) * (0.5 + torch.rand(e, k // GROUP, n, generator=gen, device="cuda"))
    return words, zeros, scales.to(dtype)


def _inputs(case, seed):
    gen = _generator(seed)
    s = dict(case)
    if case["op"] == "fp8":
        t, k, n = case["tokens"], case["inputs"], case["outputs"]
        x = torch.randn(t, k, generator=gen, device="cuda")
        x[:, :: max(8, k // 5)] *= 20.0  # a few channels far above the others, as hidden states have them
        s["x"] = x.to(DTYPES[case["dtype"]])
        w = torch.randn(n, k, generator=gen, device="cuda").mul_(110.0).clamp_(-E4M3_MAX, E4M3_MAX)
        s["wq"] = w.to(torch.float8_e4m3fn)
        s["s_w"] = (0.5 + torch.rand(-(-n // GROUP), -(-k // GROUP), generator=gen, device="cuda")) * (0.01 / math.sqrt(k))
        return s
    s["logits"] = _logits(case, gen)
    if case["op"] == "experts":
        dtype, e, width, inner = DTYPES[case["dtype"]], case["experts"], case["width"], case["inner"]
        s["x"] = torch.randn(case["tokens"], width, generator=gen, device="cuda").to(dtype)
        s["up"] = _awq_weights(e, width, 2 * inner, dtype, case["symmetric"], gen)  # gate, then up
        s["down"] = _awq_weights(e, inner, width, dtype, case["symmetric"], gen)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] == "experts":
        from bit_weight_only_awq_gb300 import awq
        s["up"] = awq.awq_moe_prepack(*s["up"], gated=True)  # laid out once, when the layer is loaded
        s["down"] = awq.awq_moe_prepack(*s["down"])
    return s


# ------------------------------------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "fp8":
        return _own_fp8(s) if own else _plain_fp8(s)
    if s["op"] == "route":
        return _own_route(s) if own else _plain_route(s)
    return _own_experts(s) if own else _plain_experts(s)


def _own_route(s):
    from bit_weight_only_awq_gb300 import awq
    weights, ids, plan = awq.awq_moe_route(s["logits"], s["top_k"], normalize=s["normalize"])
    return {"weights": weights, "ids": ids, "offsets": plan.offsets, "order": plan.order, "place": plan.place}


def _own_experts(s):
    from bit_weight_only_awq_gb300 import awq
    weights, _, plan = awq.awq_moe_route(s["logits"], s["top_k"], normalize=s["normalize"])
    return awq.awq_moe(s["x"], s["up"], s["down"], weights, plan)


def _own_fp8(s):
    from bit_weight_only_awq_gb300 import awq
    return awq.awq_fp8_linear(s["x"], s["wq"], s["s_w"])


def _plain_route(s):
    logits, top_k, e = s["logits"].float(), s["top_k"], s["experts"]
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top_k]
    weight = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    chosen = weight.gather(1, ids)
    weights = chosen / (chosen if s["normalize"] else weight).sum(dim=1, keepdim=True)
    flat = ids.flatten()
    order = torch.sort(flat, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.shape[0], device=order.device)
    expert = torch.arange(e + 1, device=flat.device)
    offsets = (flat[None, :] < expert[:, None]).sum(dim=1)
    return {"weights": weights, "ids": ids.int(), "offsets": offsets.int(), "order": order.int(), "place": place.int()}


def _dequantize(words, zeros, scales):
    """fp32 [k, n] of one layer in the AWQ layout: column j of eight is the nibble (0, 4, 1, 5, 2, 6, 3, 7)[j]."""
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=words.device)
    code = ((words[..., None] >> shift) & 15).flatten(-2).float().unflatten(0, (-1, GROUP))
    zero = 8.0 if zeros is None else ((zeros[..., None] >> shift) & 15).flatten(-2).float()[:, None]
    return ((code - zero) * scales.float()[:, None]).flatten(0, 1)


def _layer(weights, e):
    words, zeros, scales = weights
    return _dequantize(words[e], None if zeros is None else zeros[e], scales[e])


def _plain_experts(s):
    routed = _plain_route(s)
    x, inner = s["x"].float(), s["inner"]
    y = torch.zeros((s["tokens"] * s["top_k"], s["width"]), device=x.device)
    bounds = routed["offsets"].tolist()
    for e in range(s["experts"]):
        rows = routed["order"][bounds[e] : bounds[e + 1]].long()
        if rows.shape[0] == 0:
            continue
        h = torch.matmul(x[rows // s["top_k"]], _layer(s["up"], e))
        gate, up = h[:, :inner], h[:, inner:]
        y[rows] = torch.matmul(gate / (1.0 + torch.exp(-gate)) * up, _layer(s["down"], e))
    y = y.unflatten(0, (s["tokens"], s["top_k"])) * routed["weights"][..., None]
    return y.sum(dim=1).to(s["x"].dtype)


def _plain_fp8(s):
    x, k, n = s["x"].float(), s["inputs"], s["outputs"]
    pad = -k % GROUP
    x = torch.nn.functional.pad(x, (0, pad)).unflatten(1, (-1, GROUP))
    scale = x.abs().amax(dim=2, keepdim=True) / torch.full((1, 1, 1), E4M3_MAX, device=x.device)
    code = torch.where(scale > 0, x / scale, torch.zeros_like(x)).to(torch.float8_e4m3fn).float()
    x = (code * scale).flatten(1)[:, :k]
    s_w = s["s_w"].repeat_interleave(GROUP, 0)[:n].repeat_interleave(GROUP, 1)[:, :k]
    return torch.matmul(x, (s["wq"].float() * s_w).t()).to(s["x"].dtype)


# ---------------------------------------------------------------------- the definitions, in 64 bits

def _exact_route(s):
    logits = s["logits"].double()
    t, e, top_k = s["tokens"], s["experts"], s["top_k"]
    ids = torch.empty((t, top_k), dtype=torch.int64, device=logits.device)
    left = logits.clone()
    row = torch.arange(t, device=logits.device)
    number = torch.arange(e, device=logits.device).expand(t, e)
    for j in range(top_k):  # the largest that is left, the first of equals
        first = torch.where(left == left.max(dim=1, keepdim=True).values, number, e).min(dim=1).values
        ids[:, j] = first
        left[row, first] = -math.inf
    total = torch.logsumexp(logits.gather(1, ids) if s["normalize"] else logits, dim=1, keepdim=True)
    weights = torch.exp(logits.gather(1, ids) - total)
    count = torch.bincount(ids.flatten(), minlength=e)
    offsets = torch.cat((count.new_zeros(1), count.cumsum(0)))
    # by expert, then by position
    order = torch.argsort(ids.flatten() * (t * top_k) + torch.arange(t * top_k, device=ids.device))
    return {"weights": weights, "ids": ids.int(), "offsets": offsets.int(), "order": order.int(),
            "place": torch.argsort(order).int()}


def _exact_layer(weights, e):
    words, zeros, scales = weights
    columns = scales.shape[2]
    nibble = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=words.device).repeat(columns // 8)
    word = torch.arange(columns, device=words.device) // 8
    out = torch.empty((words.shape[1], columns), dtype=torch.float64, device=words.device)
    for g in range(scales.shape[1]):
        code = words[e, g * GROUP : (g + 1) * GROUP].long()[:, word] // 16 ** nibble % 16
        zero = 8 if zeros is None else zeros[e, g].long()[word] // 16 ** nibble % 16
        out[g * GROUP : (g + 1) * GROUP] = (code - zero).double() * scales[e, g].double()
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "experts":
        routed = _exact_route(s)
        x = s["x"].double()
        out = torch.zeros((case["tokens"], case["width"]), dtype=torch.float64, device=x.device)
        for e in range(case["experts"]):
            token, choice = (routed["ids"] == e).nonzero(as_tuple=True)
            if token.shape[0]:
                gate, up = torch.mm(x[token], _exact_layer(s["up"], e)).chunk(2, dim=1)
                y = torch.mm(gate * torch.sigmoid(gate) * up, _exact_layer(s["down"], e))
                out.index_add_(0, token, y * routed["weights"][token, choice][:, None])
        return out
    t, k, n = case["tokens"], case["inputs"], case["outputs"]
    out = torch.zeros((t, n), dtype=torch.float64, device="cuda")
    for g in range(0, k, GROUP):
        x = s["x"][:, g : g + GROUP].double()
        # scale and quotient are fp32 numbers by definition; the code is the nearest number of 3 + 1 bits
        scale = (torch.linalg.vector_norm(x, ord=math.inf, dim=1, keepdim=True) / E4M3_MAX).float().double()
        quotient = torch.nan_to_num(x / scale, nan=0.0).float().double()
        step = torch.exp2(torch.floor(torch.log2(quotient.abs().clamp(min=2.0 ** -6))) - 3)
        x = torch.round(quotient / step).mul(step).clamp(-E4M3_MAX, E4M3_MAX) * scale
        w = s["wq"][:, g : g + GROUP].double()
        out += torch.mm(x, w.t()) * s["s_w"][:, g // GROUP].double().repeat_interleave(GROUP)[:n]
    return out
