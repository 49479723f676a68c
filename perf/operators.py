"""Cases of the attention operators: appending to a paged key/value cache with the position rotation, attention of
new tokens over that cache, and attention over whole packed prompts.

Each case names one operator and the sizes of one call. `run` computes it either in plain torch operations in 32
bits (`own` false) or through the framework's entry points (`own` true); `exact` computes the definition in 64 bits.
"""
import math
import random

import torch

own = False

ROPE_THETA = 500000.0


# ----------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------
def _append(name, **kw):
    return {"name": name, "op": "append", "dim": 128, "fmt": "bf16", "page": 16, "order": "head", "decode": 0, "chunks": 0,
            "new": 1, "context": 1024, "interleaved": False, "lengths": 1, **kw}


def _paged(name, **kw):
    return {"name": name, "op": "paged", "dim": 128, "fmt": "bf16", "page": 16, "order": "head", "decode": 0, "chunks": 0,
            "new": 1, "context": 1024, "lengths": 1, **kw}


def _prompt(name, **kw):
    return {"name": name, "op": "prompt", "dim": 128, "prompts": 1, "longest": 512, "lengths": 1, **kw}


def listed():
    """Head shapes: 32 query over 8 key/value heads of 128 (the 8B layers' qkv 4096 -> 6144), 64 over 8 (the 70B
    layers' qkv 8192 -> 10240), and an odd group of small heads."""
    return [
        # one user's next token on the 8B layers: nothing but latency
        _append("append-1-token", heads=32, kv_heads=8, decode=1, context=1000),
        # the mixed serving batch on the 70B layers: 64 decoding sequences and one 2048-token prefill chunk, 8-bit cache
        _append("append-64+2048-e4m3", heads=64, kv_heads=8, decode=64, chunks=1, new=2048, context=4096, fmt="e4m3", page=64),
        # four long chunks of odd length, cache rows in token order, interleaved rotation
        _append("append-4x2011-interleaved", heads=32, kv_heads=8, chunks=4, new=2011, context=6001, order="token",
                interleaved=True, page=32),
        # one user's next token on the 8B layers, about a thousand tokens in
        _paged("decode-1x1023", heads=32, kv_heads=8, decode=1, context=1023),
        # 32 tenants, one token each, contexts of every length up to 4096
        _paged("decode-32x4096", heads=32, kv_heads=8, decode=32, context=4096),
        # 64 long conversations on the 70B layers with an 8-bit cache
        _paged("decode-64x16384-e4m3", heads=64, kv_heads=8, decode=64, context=16384, fmt="e4m3", page=64),
        # the mixed serving batch: 64 decoding sequences and one 2048-token prefill chunk
        _paged("mixed-64+2048", heads=64, kv_heads=8, decode=64, chunks=1, new=2048, context=4096),
        # a few tokens at a time (a follow-up question) over long histories; odd group of small heads, token-order cache
        _paged("chunk-4x37-d64", heads=14, kv_heads=2, dim=64, chunks=4, new=37, context=7999, order="token", page=32),
        # a 512-token chunk deep into a long document with an 8-bit cache
        _paged("chunk-1x512-e4m3", heads=32, kv_heads=8, chunks=1, new=512, context=16300, fmt="e4m3", page=128),
        # a short prompt
        _prompt("prompt-77", heads=32, kv_heads=8, prompts=1, longest=77),
        # a batch of prompts of every length up to a thousand
        _prompt("prompt-16x1024", heads=32, kv_heads=8, prompts=16, longest=1024),
        # one long document on the 70B layers
        _prompt("prompt-8192", heads=64, kv_heads=8, prompts=1, longest=8192),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    heads, kv_heads = rng.choice([(32, 8), (64, 8), (14, 2), (8, 8), (24, 8), (5, 1), (16, 1)])
    dim = rng.choice([64, 128, 128])
    op = rng.choice(["append", "paged", "paged", "prompt"])
    lengths = rng.randrange(1 << 20)
    while True:
        if op == "prompt":
            case = _prompt("", heads=heads, kv_heads=kv_heads, dim=dim, prompts=_log_int(rng, 1, 24),
                           longest=_log_int(rng, 1, 8192), lengths=lengths)
        else:
            context = _log_int(rng, 1, 16384)
            kind = rng.choice(["decode", "chunk", "mixed"])
            case = (_append if op == "append" else _paged)(
                "", heads=heads, kv_heads=kv_heads, dim=dim, fmt=rng.choice(["bf16", "e4m3"]),
                page=rng.choice([16, 32, 64, 128, 256]), order=rng.choice(["head", "token"]),
                decode=_log_int(rng, 1, 96) if kind != "chunk" else 0, chunks=_log_int(rng, 1, 6) if kind != "decode" else 0,
                new=_log_int(rng, 1, min(2048, context)), context=context, lengths=lengths)
            if op == "append":
                case["interleaved"] = rng.random() < 0.5
        w = work(case)
        if w["bytes"] <= 1.1e9 and w["flops"] <= 1.1e12 and _score_bytes(case) <= 20e9:
            del case["name"]
            return case


# ----------------------------------------------------------------------------------------------------------------
# lengths, work
# ----------------------------------------------------------------------------------------------------------------
def _spread(rng, longest, count):
    """`count` lengths: the longest first, the others spread evenly below it."""
    return [longest] + [rng.randint(1, longest) for _ in range(count - 1)]


def _sequences(case):
    """(new tokens, tokens after them) of each sequence: the decoding ones first, then the chunks."""
    rng = random.Random(case["lengths"])
    if case["op"] == "prompt":
        return [(n, n) for n in _spread(rng, case["longest"], case["prompts"])]
    seqs = [(1, n) for n in _spread(rng, case["context"], case["decode"])] if case["decode"] else []
    for _ in range(case["chunks"]):
        seqs.append((case["new"], rng.randint(max(case["new"], case["context"] * 7 // 8), case["context"])))
    return seqs


def _score_bytes(case):
    """Bytes of the plain form's padded scores."""
    seqs = _sequences(case)
    d = case.get("decode", 0)
    return sum(4 * case["heads"] * len(s) * max(n for n, _ in s) * max(m for _, m in s) for s in (seqs[:d], seqs[d:]) if s)


def work(case):
    seqs = _sequences(case)
    tokens, dim, heads, kv_heads = sum(n for n, _ in seqs), case["dim"], case["heads"], case["kv_heads"]
    size = 1 if case.get("fmt") == "e4m3" else 2
    rows = tokens * heads * dim * 2
    if case["op"] == "append":
        moved = 2 * rows + tokens * 2 * kv_heads * dim * (2 + size) + tokens * dim * 4
        return {"bytes": moved, "flops": 3 * tokens * (heads + kv_heads) * dim}
    pairs = sum(n * m - n * (n - 1) // 2 for n, m in seqs)
    moved = 2 * rows + sum(m for _, m in seqs) * 2 * kv_heads * dim * size
    return {"bytes": moved, "flops": 4 * dim * heads * pairs}


# ----------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------
def _qkv(case, tokens, g):
    """q, k, v as slices of one projection output; key channels of unlike size, as rotated heads have them."""
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    x = torch.randn(tokens, heads + 2 * kv_heads, dim, generator=g, device="cuda")
    x[:, heads:heads + kv_heads] *= _key_channels(case, g)
    x = x.to(torch.bfloat16)
    return x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]


def _key_channels(case, g):
    return torch.exp(0.5 * torch.randn(case["kv_heads"], case["dim"], generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    seqs = _sequences(case)
    new, total = torch.tensor([n for n, _ in seqs]), torch.tensor([m for _, m in seqs])
    tokens = int(new.sum())
    q_start = torch.zeros(len(seqs) + 1, dtype=torch.int32)
    q_start[1:] = new.cumsum(0)
    chunks = [m for _, m in seqs[case.get("decode", 0):]]
    s = {"case": case, "q_start": q_start.cuda(), "max_new": int(new.max()), "longest": int(total.max()),
         "longest_chunk": max(chunks, default=0), "scale": case["dim"] ** -0.5}
    if case["op"] == "prompt":
        s["q"], s["k"], s["v"] = _qkv(case, tokens, g)
        return s
    # a pool with half as many pages again as the sequences hold, handed out in random order
    page, kv_heads, dim = case["page"], case["kv_heads"], case["dim"]
    held = -(-total // page)
    count, widest = int(held.sum()), int(held.max())
    pages = count + count // 2 + 1
    order = torch.randperm(pages, generator=g, device="cuda")[:count].to(torch.int32).cpu()
    table = torch.zeros(len(seqs), widest, dtype=torch.int32)
    inside = torch.arange(widest)[None, :] < held[:, None]
    table[inside] = order
    shape = (pages, kv_heads, page, dim) if case["order"] == "head" else (pages, page, kv_heads, dim)
    s["k_scale"] = s["v_scale"] = None
    if case["fmt"] == "e4m3":
        s["k_scale"] = 0.02 + 0.02 * torch.rand(kv_heads, generator=g, device="cuda")
        s["v_scale"] = 0.01 + 0.01 * torch.rand(kv_heads, generator=g, device="cuda")
    for which in ("k", "v"):
        pool = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        pool = pool if case["order"] == "head" else pool.transpose(1, 2)        # [pages, kv_heads, page, dim], strided
        if which == "k":
            pool *= _key_channels(case, g).to(torch.bfloat16)[None, :, None, :]
        if case["fmt"] == "e4m3":
            pool = (pool / s[which + "_scale"][None, :, None, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
            pool = pool.view(torch.uint8)
        s[which + "_pool"] = pool
    s["kv_len"], s["table"] = total.to(torch.int32).cuda(), table.cuda()
    q, k, v = _qkv(case, tokens, g)
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = q, k, v
        turn = torch.arange(s["longest"], device="cuda", dtype=torch.float64)[:, None] * \
            ROPE_THETA ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
        s["cos_sin"] = torch.cat([turn.cos(), turn.sin()], 1).float()
    else:
        s["q"] = q.contiguous()
    return s


# ----------------------------------------------------------------------------------------------------------------
# the operators through the framework, and in plain operations
# ----------------------------------------------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _as_values(s):
    """The cache as the numbers it holds (before the scale of an 8-bit head)."""
    if s["case"]["fmt"] == "e4m3":
        return s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn)
    return s["k_pool"], s["v_pool"]


def _run_own(s):
    from precision_gemm_token_gb300 import attention as A
    op = s["case"]["op"]
    if op != "append" and "workspace" not in s:
        s["workspace"] = A.AttentionWorkspace(s["q"].device)
    if op == "prompt":
        return A.prompt_attention(s["q"], s["k"], s["v"], s["q_start"], scale=s["scale"], workspace=s["workspace"])
    if "cache" not in s:
        s["cache"] = A.PagedKVCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
    if op == "paged":
        return A.paged_attention(s["q"], s["cache"], s["q_start"], s["kv_len"], s["table"], max_new=s["max_new"],
                                 scale=s["scale"], workspace=s["workspace"])
    q = A.kv_append(s["q"], s["k"], s["v"], s["cache"], s["q_start"], s["kv_len"], s["table"], s["cos_sin"],
                    interleaved=s["case"]["interleaved"])
    return {"q": q, "cache": _as_values(s)}


def _run_plain(s):
    return {"append": _plain_append, "paged": _plain_paged, "prompt": _plain_prompt}[s["case"]["op"]](s)


def _rotate(x, cos, sin, interleaved):
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, dim=-1)
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _plain_append(s):
    case, page = s["case"], s["case"]["page"]
    start = s["q_start"].long()
    token = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(start[1:], token, right=True)
    position = s["kv_len"].long()[seq] - start[1:][seq] + token
    cos, sin = s["cos_sin"][position][:, None].chunk(2, dim=-1)
    q = _rotate(s["q"], cos, sin, case["interleaved"]).to(torch.bfloat16)
    k, v = _rotate(s["k"], cos, sin, case["interleaved"]), s["v"].float()
    where, row = s["table"][seq, position // page].long(), position % page
    if case["fmt"] == "e4m3":
        k, v = ((x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for x, scale in ((k, s["k_scale"]), (v, s["v_scale"])))
    s["k_pool"][where, :, row] = k.to(s["k_pool"].dtype)
    s["v_pool"][where, :, row] = v.to(s["v_pool"].dtype)
    return {"q": q, "cache": _as_values(s)}


def _attend(q, k, v, q_pos, scale):
    """q [B, n, heads, dim]; k, v [B, m, kv_heads, dim], all in 32 bits; q_pos [B, n] (-1: no token there). Row (b, i)
    attends to the positions up to q_pos[b, i]."""
    b, n, heads, dim = q.shape
    m, kv_heads = k.shape[1:3]
    group = heads // kv_heads
    q = q.view(b, n, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(b, kv_heads, group * n, dim)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(scale).view(b, kv_heads, group, n, m)
    hidden = torch.arange(m, device="cuda")[None, None, :] > q_pos[:, :, None]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    score -= score.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    score.exp_()
    score /= score.sum(-1, keepdim=True).clamp_min(1e-30)
    out = torch.matmul(score.view(b, kv_heads, group * n, m), v.permute(0, 2, 1, 3))
    return out.view(b, kv_heads, group, n, dim).permute(0, 3, 1, 2, 4).reshape(b, n, heads, dim)


def _padded(start, first, last, width):
    """Rows of the packed tokens of sequences first..last-1, [last - first, width], and which of them exist."""
    rows = start[first:last, None] + torch.arange(width, device="cuda")
    there = rows < start[first + 1:last + 1, None]
    return torch.where(there, rows, torch.zeros_like(rows)), there


def _plain_prompt(s):
    start = s["q_start"].long()
    rows, there = _padded(start, 0, len(start) - 1, s["longest"])
    position = torch.arange(s["longest"], device="cuda").expand_as(rows)
    out = _attend(s["q"][rows].float(), s["k"][rows].float(), s["v"][rows].float(), torch.where(there, position, -1), s["scale"])
    return out[there].to(torch.bfloat16)


def _plain_paged_part(s, first, last, most_new, longest):
    """Sequences first..last-1, padded to their longest."""
    page = s["case"]["page"]
    start, total = s["q_start"].long(), s["kv_len"].long()[first:last]
    rows, there = _padded(start, first, last, most_new)
    position = total[:, None] - (start[first + 1:last + 1] - start[first:last])[:, None] + torch.arange(most_new, device="cuda")
    at = torch.arange(longest, device="cuda")
    where = s["table"].long()[first:last, at // page]
    held = []
    for pool, scale in zip(_as_values(s), (s["k_scale"], s["v_scale"])):
        x = pool.permute(0, 2, 1, 3)[where, at % page].float()
        held.append(x if scale is None else x * scale[:, None])
    out = _attend(s["q"][rows].float(), *held, torch.where(there, position, -1), s["scale"])
    return out[there].to(torch.bfloat16)


def _plain_paged(s):
    case = s["case"]
    decode, seqs = case["decode"], len(s["q_start"]) - 1
    parts = []
    if decode:
        parts.append(_plain_paged_part(s, 0, decode, 1, case["context"]))
    if seqs > decode:
        parts.append(_plain_paged_part(s, decode, seqs, case["new"], s["longest_chunk"]))
    return torch.cat(parts)


# ----------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    seqs, dim, group = _sequences(case), case["dim"], case["heads"] // case["kv_heads"]
    starts = s["q_start"].tolist()
    if case["op"] == "append":
        return _exact_append(s, seqs, starts)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for (n, m), t in zip(seqs, starts):
        if case["op"] == "prompt":
            k, v = s["k"][t:t + n].double(), s["v"][t:t + n].double()
        else:
            k, v = _exact_cache(s, t, n, m, starts)
        for h in range(case["heads"]):
            kh, vh = k[:, h // group], v[:, h // group]
            for i in range(0, n, 2048):
                rows = min(2048, n - i)
                seen = m - n + i + rows                        # positions that the last of these rows sees
                x = s["q"][t + i:t + i + rows, h].double() @ kh[:seen].T / math.sqrt(dim)
                x += torch.full((rows, seen), -math.inf, dtype=torch.float64, device="cuda").triu(m - n + i + 1)
                out[t + i:t + i + rows, h] = torch.softmax(x, -1) @ vh[:seen]
    return out


def _exact_cache(s, t, n, m, starts):
    case, page = s["case"], s["case"]["page"]
    b = starts.index(t)
    found = []
    for pool, scale in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])):
        if case["fmt"] == "e4m3":
            pool = pool.view(torch.float8_e4m3fn)
        rows = pool[s["table"][b, :-(-m // page)].long()]      # [pages, kv_heads, page, dim]
        x = rows.to(torch.float32).double().transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])[:m]
        found.append(x if scale is None else x * scale.double()[:, None])
    return found


def _exact_append(s, seqs, starts):
    case, page, half = s["case"], s["case"]["page"], s["case"]["dim"] // 2
    position = torch.cat([torch.arange(m - n, m) for n, m in seqs])
    owner = torch.cat([torch.full((n,), b) for b, (n, _) in enumerate(seqs)])
    table = s["cos_sin"].double()[position.cuda()]
    turn = torch.complex(table[:, None, :half], table[:, None, half:])

    def rotated(x):
        x = x.double()
        if case["interleaved"]:
            return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous()) * turn).flatten(-2)
        y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
        return torch.cat([y.real, y.imag], -1)

    cache = []
    pages = s["table"].cpu()[owner, position // page].long().cuda()
    for pool, x, scale in ((s["k_pool"], rotated(s["k"]), s["k_scale"]), (s["v_pool"], s["v"].double(), s["v_scale"])):
        if case["fmt"] == "e4m3":
            pool, x = pool.view(torch.float8_e4m3fn).to(torch.float32), (x / scale.double()[:, None]).clamp(-448, 448)
        pool = pool.double()
        pool[pages, :, (position % page).cuda()] = x
        cache.append(pool)
    return {"q": rotated(s["q"]), "cache": tuple(cache)}
