"""Cases of the operators of a mixture-of-experts layer in 8-bit blocks: quantizing activations to E4M3 with a scale for
each 128 elements, the product with weights that have a scale for each 128 x 128 block, routing tokens to experts,
and the experts' two products (gate and up with the activation between them, and down with the weighted sum).

Each case names one operator and the sizes of one call. `run` computes it either in plain torch operations in 32
bits (`own` false) or through the framework's entry points (`own` true); `exact` computes the definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-12


# ----------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------
def _quant(name, tokens, width):
    return {"name": name, "op": "quant", "tokens": tokens, "width": width}


def _linear(name, tokens, width, out):
    return {"name": name, "op": "linear", "tokens": tokens, "width": width, "out": out}


def _route(name, tokens, experts, top, **kw):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top": top, "scoring": "softmax",
            "bias": False, "groups": 1, "top_groups": 1, "group_best": 1, "renormalize": True, "scale": 1.0,
            "logits": "fp32", **kw}


def _experts(name, op, tokens, experts, top, hidden, inner, **kw):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "top": top, "hidden": hidden,
            "inner": inner, "padding": 0, **kw}


def listed():
    """Widths of the 8B layers (hidden 4096, qkv 6144, inner 14336) and of the 70B layers (hidden 8192, inner 28672);
    64 experts of the 8B layers' hidden width and an eighth of their inner one, 8 chosen for a token."""
    return [
        # one user's next token: nothing but latency
        _quant("quant-1x4096", 1, 4096),
        # the activations of a long prompt before a down projection
        _quant("quant-8192x14336", 8192, 14336),
        # one user's next token through qkv
        _linear("linear-1x4096-6144", 1, 4096, 6144),
        # 32 tenants, one token each, through a down projection
        _linear("linear-32x14336-4096", 32, 14336, 4096),
        # a prompt of odd length through a head of odd width, blocks of every kind cut short
        _linear("linear-509x2064-1000", 509, 2064, 1000),
        # a prefill chunk of 2048 tokens through the 70B layers' gate projection
        _linear("linear-2048x8192-28672", 2048, 8192, 28672),
        # one user's next token, softmax scores
        _route("route-1x128", 1, 128, 8),
        # a prefill batch with sigmoid scores, a bias that balances the experts, and a choice of groups first
        _route("route-4096x256-groups", 4096, 256, 8, scoring="sigmoid", bias=True, groups=8, top_groups=4,
               group_best=2, scale=2.5),
        # one user's next token: eight experts' weights read for it
        _experts("up-1", "up", 1, 64, 8, 4096, 1792),
        # a prefill batch: some hundreds of tokens an expert
        _experts("up-4096", "up", 4096, 64, 8, 4096, 1792),
        # a decoding batch captured for 64 tokens, 61 of them there: every expert read for a few tokens each
        _experts("down-64", "down", 64, 64, 8, 4096, 1792, padding=3),
        # the prefill batch
        _experts("down-4096", "down", 4096, 64, 8, 4096, 1792),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "route", "up", "down"])
    while True:
        if op == "quant":
            case = _quant("", _log_int(rng, 1, 8192), 16 * _log_int(rng, 1, 1024))
        elif op == "linear":
            case = _linear("", _log_int(rng, 1, 4096), 16 * _log_int(rng, 4, 1024), _log_int(rng, 16, 28672))
        elif op == "route":
            groups = rng.choice([1, 1, 2, 4, 8])
            experts = groups * rng.choice([2, 5, 8, 15, 16, 32, 40, 64])
            top_groups = rng.randint(1, groups)
            sums = groups > 1 and rng.random() < 0.5
            case = _route("", _log_int(rng, 1, 16384), experts, rng.randint(1, min(16, experts // groups * top_groups)),
                          scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                          top_groups=top_groups, group_best=2 if sums else 1, renormalize=rng.random() < 0.7,
                          scale=rng.choice([1.0, 2.5]), logits=rng.choice(["fp32", "bf16"]))
        else:
            experts, tokens = rng.choice([4, 7, 16, 32, 60, 64, 128]), _log_int(rng, 1, 4096)
            case = _experts("", op, tokens, experts, rng.randint(1, min(8, experts)), 16 * _log_int(rng, 8, 512),
                            16 * _log_int(rng, 4, 112), padding=rng.choice([0, 0, tokens // 7]))
        w, most = work(case), _most(case["op"])
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            del case["name"]
            return case


def _most(op):
    """The largest listed case's work, of each kind."""
    found = [work(c) for c in listed() if c["op"] == op]
    return {k: max(w[k] for w in found) for k in ("bytes", "flops")}


# ----------------------------------------------------------------------------------------------------------------
# work
# ----------------------------------------------------------------------------------------------------------------
def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    t = case["tokens"]
    if case["op"] == "quant":
        k = case["width"]
        return {"bytes": t * k * 3 + t * _blocks(k) * 4, "flops": 3 * t * k}
    if case["op"] == "linear":
        k, n = case["width"], case["out"]
        return {"bytes": 2 * t * (k + n) + n * k + 4 * _blocks(n) * _blocks(k), "flops": 2 * t * n * k}
    if case["op"] == "route":
        e, size = case["experts"], 4 if case["logits"] == "fp32" else 2
        return {"bytes": t * e * size + (4 * e if case["bias"] else 0) + t * case["top"] * 8, "flops": 8 * t * e}
    e, k, h, i = case["experts"], case["top"], case["hidden"], case["inner"]
    there = t - case["padding"]
    read = e * (1 - (1 - k / e) ** there)                   # experts that somebody chose, were the choices even
    if case["op"] == "up":
        moved = t * (2 * h + k * (4 + i + 4 * _blocks(i))) + read * 2 * (i * h + 4 * _blocks(i) * _blocks(h))
        return {"bytes": round(moved), "flops": 4 * there * k * h * i}
    moved = t * (2 * h + k * 8) + there * k * (i + 4 * _blocks(i)) + read * (i * h + 4 * _blocks(i) * _blocks(h))
    return {"bytes": round(moved), "flops": 2 * there * k * h * i}


# ----------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------
def _activations(t, k, g):
    """Rows of unlike size with a few channels that stand out, as a layer's activations have them."""
    x = torch.randn(t, k, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(t, 1, generator=g, device="cuda"))
    x *= torch.exp(0.7 * torch.randn(k, generator=g, device="cuda"))
    return x.to(torch.bfloat16)


def _weight(n, k, g):
    """E4M3 codes [n, k] and the scales of their 128 x 128 blocks, as a checkpoint holds them."""
    w = torch.zeros(_blocks(n) * BLOCK, _blocks(k) * BLOCK, device="cuda")
    w[:n, :k] = 0.02 * torch.randn(n, k, generator=g, device="cuda")
    w = w.view(_blocks(n), BLOCK, _blocks(k), BLOCK)
    scale = w.abs().amax((1, 3)).clamp_min(AMAX_FLOOR) / E4M3_MAX
    codes = (w / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(_blocks(n) * BLOCK, -1)[:n, :k].contiguous().view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, s = case["tokens"], {"case": case}
    if case["op"] == "quant":
        s["x"] = _activations(t, case["width"], g)
    elif case["op"] == "linear":
        s["x"] = _activations(t, case["width"], g)
        s["w"], s["w_scale"] = _weight(case["out"], case["width"], g)
    elif case["op"] == "route":
        e = case["experts"]
        logits = 1.5 * torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
        s["logits"] = logits.to(torch.float32 if case["logits"] == "fp32" else torch.bfloat16)
        s["bias"] = 0.05 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
    else:
        e, k, h, i = case["experts"], case["top"], case["hidden"], case["inner"]
        # some experts are chosen more often than others; the tokens that are not there have none
        liking = torch.randn(t, e, generator=g, device="cuda") + 0.7 * torch.randn(e, generator=g, device="cuda")
        score, ids = liking.topk(k, -1)
        s["ids"], s["weights"] = ids.to(torch.int32), torch.softmax(score, -1)
        there = t - case["padding"]
        s["ids"][there:], s["weights"][there:] = -1, 0
        s["gate_up"] = torch.empty(e, 2, i, h, dtype=torch.uint8, device="cuda")
        s["gate_up_scale"] = torch.empty(e, 2, _blocks(i), _blocks(h), device="cuda")
        s["down"] = torch.empty(e, h, i, dtype=torch.uint8, device="cuda")
        s["down_scale"] = torch.empty(e, _blocks(h), _blocks(i), device="cuda")
        for n in range(e):
            for part in range(2):
                s["gate_up"][n, part], s["gate_up_scale"][n, part] = _weight(i, h, g)
            s["down"][n], s["down_scale"][n] = _weight(h, i, g)
        if case["op"] == "up":
            s["x"] = _activations(t, h, g)
        else:
            # what an activation leaves: most elements small, a few large; nothing where there is no expert
            a, b = (torch.randn(t * k, i, generator=g, device="cuda") for _ in range(2))
            values, scale = _plain_quant((a * b).abs_().sub_(0.2))
            values = values.view(torch.uint8)
            values[there * k:], scale[:, there * k:] = 0, 0
            s["inner"], s["inner_scale"] = values.view(t, k, i), scale
    return s


# ----------------------------------------------------------------------------------------------------------------
# the operators through the framework, and in plain operations
# ----------------------------------------------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from precision_gemm_token_gb300 import blocks, moe
    case = s["case"]
    if case["op"] == "quant":
        codes, scale = blocks.block_quant(s["x"])
        return {"values": codes.view(torch.float8_e4m3fn), "scale": scale}
    if case["op"] == "route":
        ids, weights = moe.route(s["logits"], case["top"], bias=s["bias"], scoring=case["scoring"],
                                 groups=case["groups"], top_groups=case["top_groups"], group_best=case["group_best"],
                                 renormalize=case["renormalize"], scale=case["scale"])
        return {"ids": ids, "weights": weights}
    if "workspace" not in s:
        s["workspace"] = blocks.BlockWorkspace("cuda")
        s["handle"] = blocks.BlockWeight(s["w"], s["w_scale"]) if case["op"] == "linear" else \
            moe.ExpertWeights(s["gate_up"], s["gate_up_scale"], s["down"], s["down_scale"])
    if case["op"] == "linear":
        return blocks.block_linear(s["x"], s["handle"], workspace=s["workspace"])
    if case["op"] == "up":
        codes, scale = moe.experts_up(s["x"], s["ids"], s["handle"], workspace=s["workspace"])
        return {"values": codes.view(torch.float8_e4m3fn), "scale": scale}
    return moe.experts_down(s["inner"], s["inner_scale"], s["ids"], s["weights"], s["handle"], workspace=s["workspace"])


def _run_plain(s):
    if s["case"]["op"] == "quant":
        values, scale = _plain_quant(s["x"])
        return {"values": values, "scale": scale}
    if s["case"]["op"] == "linear":
        return (_plain_dequant(*_plain_quant(s["x"])) @ _plain_weight(s["w"], s["w_scale"]).T).to(torch.bfloat16)
    return {"route": _plain_route, "up": _plain_up, "down": _plain_down}[s["case"]["op"]](s)


def _in_blocks(x):
    """[rows, k] as [rows, blocks, 128], zeros behind the last element."""
    rows, k = x.shape
    return torch.nn.functional.pad(x, (0, _blocks(k) * BLOCK - k)).view(rows, _blocks(k), BLOCK)


def _plain_quant(x):
    """E4M3 values [rows, k] and scales [blocks, rows]."""
    rows, k = x.shape
    x = _in_blocks(x.float())
    scale = x.abs().amax(-1).clamp_min(AMAX_FLOOR)
    scale = scale / torch.full_like(scale, E4M3_MAX)        # (by a number it would be multiplied by the reciprocal)
    x = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return x.view(rows, -1)[:, :k].contiguous(), scale.T.contiguous()


def _plain_dequant(values, scale):
    rows, k = values.shape
    return (_in_blocks(values.float()) * scale.T[..., None]).view(rows, -1)[:, :k]


def _plain_weight(codes, scale):
    n, k = codes.shape
    spread = scale.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return codes.view(torch.float8_e4m3fn).float() * spread


def _plain_route(s):
    case = s["case"]
    t, e, groups = case["tokens"], case["experts"], case["groups"]
    logits = s["logits"].double()                   # two experts' scores may lie closer than 32 bits can tell
    scores = torch.softmax(logits, -1) if case["scoring"] == "softmax" else torch.sigmoid(logits)
    if s["bias"] is not None:
        choice = scores + s["bias"].double()
    else:
        choice = scores if case["group_best"] == 2 else logits
    if groups > 1:
        best = choice.view(t, groups, -1).sort(dim=-1, descending=True).values[..., :case["group_best"]].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        there = torch.zeros(t, groups, dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        choice = choice.masked_fill(~there.repeat_interleave(e // groups, 1), -math.inf)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :case["top"]]
    weights = scores.gather(1, ids)
    if case["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (weights * case["scale"]).float()}


def _slots(s):
    """(expert, its slots) for each expert that has any; slot j of token t is t * top + j."""
    flat = s["ids"].long().flatten()
    order = flat.argsort(stable=True)
    count = torch.bincount(flat + 1, minlength=s["case"]["experts"] + 1).tolist()       # (the first: no expert)
    at = count[0]
    for n, c in enumerate(count[1:]):
        if c:
            yield n, order[at:at + c]
        at += c


def _plain_up(s):
    case = s["case"]
    slots, i = case["tokens"] * case["top"], case["inner"]
    x = _plain_dequant(*_plain_quant(s["x"]))
    values = torch.zeros(slots, i, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(_blocks(i), slots, device="cuda")
    for n, mine in _slots(s):
        rows = x[mine // case["top"]]
        gate, up = (rows @ _plain_weight(s["gate_up"][n, part], s["gate_up_scale"][n, part]).T for part in range(2))
        codes, scale[:, mine] = _plain_quant(gate / (1 + torch.exp(-gate)) * up)
        values[mine] = codes.view(torch.uint8)
    return {"values": values.view(torch.float8_e4m3fn).view(case["tokens"], case["top"], i), "scale": scale}


def _plain_down(s):
    case = s["case"]
    inner = _plain_dequant(s["inner"].view(torch.float8_e4m3fn).flatten(0, 1), s["inner_scale"])
    out = torch.zeros(case["tokens"] * case["top"], case["hidden"], device="cuda")
    for n, mine in _slots(s):
        out[mine] = inner[mine] @ _plain_weight(s["down"][n], s["down_scale"][n]).T
    return (out.view(*s["ids"].shape, -1) * s["weights"][..., None]).sum(1).to(torch.bfloat16)


# ----------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------------
def _exact_e4m3(x):
    """The E4M3 number closest to each x (ties to the even one; the largest beyond it)."""
    step = torch.exp2(torch.frexp(x).exponent.double().sub_(1).clamp_(min=-6).sub_(3))
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quant(x):
    """Values [rows, k] and scales [rows, blocks]. Scale and quotient are 32-bit numbers by definition; rounding a
    64-bit quotient of 32-bit numbers to 32 bits rounds the quotient itself."""
    values, scales = torch.empty_like(x, dtype=torch.float64), []
    for first in range(0, x.shape[1], BLOCK):
        part = x[:, first:first + BLOCK].double()
        scale = (part.abs().max(1).values.clamp(min=AMAX_FLOOR).float().double() / E4M3_MAX).float().double()
        values[:, first:first + BLOCK] = _exact_e4m3((part / scale[:, None]).float().double())
        scales.append(scale)
    return values, torch.stack(scales, 1)


def _exact_product(values, scales, codes, w_scale):
    """Sums over the blocks of 128 along the rows' length."""
    n = codes.shape[0]
    out = torch.zeros(values.shape[0], n, dtype=torch.float64, device="cuda")
    w = codes.view(torch.float8_e4m3fn)
    for b in range(scales.shape[1]):
        part = slice(b * BLOCK, (b + 1) * BLOCK)
        rows = w_scale[:, b].double().repeat_interleave(BLOCK)[:n]
        out.addmm_(values[:, part] * scales[:, b, None], (w[:, part].float().double() * rows[:, None]).T)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        values, scales = _exact_quant(s["x"])
        return {"values": values, "scale": scales.T}
    if case["op"] == "linear":
        return _exact_product(*_exact_quant(s["x"]), s["w"], s["w_scale"])
    return {"route": _exact_route, "up": _exact_up, "down": _exact_down}[case["op"]](s)


def _exact_route(s):
    case = s["case"]
    t, e, k = case["tokens"], case["experts"], case["top"]
    z = s["logits"].double()
    if case["scoring"] == "softmax":
        score = torch.exp(z - z.max(1, keepdim=True).values)
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-z))
    by_score = s["bias"] is not None or case["group_best"] == 2
    left = (score if by_score else z) + (0 if s["bias"] is None else s["bias"].double())
    row, size = torch.arange(t, device="cuda"), e // case["groups"]
    if case["groups"] > 1:
        inside, value = left.reshape(t, -1, size).clone(), 0
        for _ in range(case["group_best"]):
            best = inside.max(2)
            value = value + best.values
            inside.scatter_(2, _first(inside, best.values)[..., None], -math.inf)
        shut = torch.ones(t, case["groups"], dtype=torch.bool, device="cuda")
        for _ in range(case["top_groups"]):
            pick = _first(value, value.max(1).values)
            value[row, pick], shut[row, pick] = -math.inf, False
        left = left.masked_fill(shut[:, torch.arange(e, device="cuda") // size], -math.inf)
    ids = torch.empty(t, k, dtype=torch.int32, device="cuda")
    for j in range(k):
        pick = _first(left, left.max(1).values)
        ids[:, j] = pick
        left[row, pick] = -math.inf
    weights = torch.stack([score[row, ids[:, j].long()] for j in range(k)], 1)
    if case["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    return {"ids": ids, "weights": weights * case["scale"]}


def _first(x, best):
    """The lowest index at which the last axis of x holds `best`."""
    at = torch.arange(x.shape[-1], device="cuda").expand(x.shape)
    return torch.where(x == best[..., None], at, x.shape[-1]).min(-1).values


def _exact_up(s):
    """The values before they are rounded: on which side of a border a sum comes to lie is not defined."""
    case = s["case"]
    x, x_scale = _exact_quant(s["x"])
    t, k, i = case["tokens"], case["top"], case["inner"]
    values = torch.zeros(t, k, i, dtype=torch.float64, device="cuda")
    scale = torch.zeros(_blocks(i), t, k, dtype=torch.float64, device="cuda")
    for n in range(case["experts"]):
        token, slot = torch.nonzero(s["ids"] == n, as_tuple=True)
        if len(token) == 0:
            continue
        gate, up = (_exact_product(x[token], x_scale[token], s["gate_up"][n, p], s["gate_up_scale"][n, p])
                    for p in range(2))
        inner = gate * torch.sigmoid(gate) * up
        for b in range(_blocks(i)):
            part = inner[:, b * BLOCK:(b + 1) * BLOCK]
            size = part.abs().max(1).values.clamp(min=AMAX_FLOOR) / E4M3_MAX
            values[token, slot, b * BLOCK:(b + 1) * BLOCK] = part / size[:, None]
            scale[b, token, slot] = size
    return {"values": values, "scale": scale.flatten(1)}


def _exact_down(s):
    case = s["case"]
    inner = s["inner"].view(torch.float8_e4m3fn).float().double()
    scale = s["inner_scale"].T.double().view(*s["ids"].shape, -1)
    out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
    for n in range(case["experts"]):
        token, slot = torch.nonzero(s["ids"] == n, as_tuple=True)
        if len(token):
            part = _exact_product(inner[token, slot], scale[token, slot], s["down"][n], s["down_scale"][n])
            out.index_add_(0, token, part * s["weights"][token, slot].double()[:, None])
    return out
