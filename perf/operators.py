"""Measured cases of the decode-step operators: queries and keys normed and
rotated, the 4-bit paged key/value cache (append, attention, page copies).

`run` computes a case either with elementary torch operations in fp32 (the
plain form, `own` false) or with this package's calls (`own` true), on the
same inputs.  The plain form reads and writes the same packed cache:

  cache  uint8 [pages, kv_heads, page, D + 8 D/g], of which the bytes of one
         (page, head) are
           K codes  [page][D/2]         word w of a token at place (w % 4) D/32 + w / 4
           V codes  [page/4][D/8][4]    words: the word of four tokens side by side
           K params [D/g][page], V params [D/g][page]   32-bit words: binary16 scale, zero-point from bit 16
  word   8 channels: channel 2i at bits 4i, channel 2i+1 at bits 16+4i
  value  (code - zero) scale, one scale and zero-point per token, head and g channels
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def _attention(name, dtype, seqs, context, q_len, q_heads, kv_heads, head_dim, group, page, spread=0.0, window=0,
               sinks=0, empty=0):
    return {"name": name, "op": "attention", "dtype": dtype, "seqs": seqs, "context": context, "q_len": q_len,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "group": group, "page": page,
            "spread": spread, "window": window, "sinks": sinks, "empty": empty}


def _append(name, dtype, tokens, kv_heads, head_dim, group, page, padded=0):
    return {"name": name, "op": "append", "dtype": dtype, "tokens": tokens, "kv_heads": kv_heads,
            "head_dim": head_dim, "group": group, "page": page, "padded": padded}


def _rope(name, dtype, tokens, q_heads, kv_heads, head_dim, rot, interleaved, norm, positions):
    return {"name": name, "op": "rope", "dtype": dtype, "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot": rot, "interleaved": interleaved, "norm": norm, "positions": positions}


def _copy(name, layers, pages, moved, kv_heads, head_dim, group, page):
    return {"name": name, "op": "copy", "layers": layers, "pages": pages, "moved": moved, "kv_heads": kv_heads,
            "head_dim": head_dim, "group": group, "page": page}


def listed():
    return [
        # one user's next token early in a conversation: latency alone counts
        _attention("decode_one", "bf16", 1, 700, 1, 32, 8, 128, 64, 64),
        # a small odd batch of an older model with a key head for every query head, one slot of the batch unused
        _attention("decode_odd", "fp16", 7, 2301, 1, 32, 32, 128, 32, 16, spread=0.6, empty=1),
        # a full serving batch at 4k context, where the cache outweighs 4-bit weights
        _attention("decode_batch", "bf16", 64, 4096, 1, 32, 8, 128, 128, 64, spread=0.3),
        # two very long documents: few rows, a long axis
        _attention("decode_long", "bf16", 2, 131072, 1, 64, 8, 128, 64, 128, spread=0.1),
        # five drafted tokens to verify in each sequence, sliding window with first tokens kept, small heads
        _attention("verify_window", "fp16", 24, 30011, 5, 16, 2, 64, 64, 32, spread=0.5, window=1024, sinks=4),
        # chunks of long prompts behind a cached prefix
        _attention("prefill_chunk", "bf16", 3, 8192, 2048, 32, 8, 128, 128, 64, spread=0.3),
        # a decode step's new tokens into the cache, and read back
        _append("append_step", "bf16", 64, 8, 128, 64, 64, padded=3),
        # a prompt's tokens into the cache, small groups
        _append("append_prompt", "fp16", 8191, 8, 128, 32, 16),
        # a decode step's queries and keys
        _rope("rope_step", "bf16", 64, 32, 8, 128, 128, False, True, 131072),
        # a prompt's, in the interleaved layout, half the head rotated
        _rope("rope_prompt", "fp16", 8191, 64, 8, 128, 64, True, True, 16384),
        # five sequences forked: the last page of each, in each layer
        _copy("copy_fork", 32, 24, 5, 8, 128, 64, 64),
        # a fragmented cache compacted
        _copy("copy_compact", 16, 700, 256, 8, 128, 64, 64),
    ]


def _spread_over(rng, low, high):
    """A whole number of [low, high], evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "rope", "copy"])
    dtype = rng.choice(["bf16", "fp16"])
    head_dim = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if head_dim % g == 0])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "attention":
        ratio = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        context = _spread_over(rng, 1, 131072)
        q_len = rng.choice([1, 1, 1, rng.randint(2, 8), _spread_over(rng, 9, 2048)])
        q_len = min(q_len, context)
        seqs = _spread_over(rng, 1, 64)
        token = kv_heads * (head_dim + 8 * head_dim // group)
        seqs = max(1, min(seqs, int(2.9e8 / (context * token)), int(2.5e9 / (q_len * ratio * kv_heads * context))))
        if context * token > 2.9e8:
            context = max(q_len, int(2.9e8 / token))
        pairs = q_len * ratio * kv_heads * context * seqs
        if pairs > 2.5e9 or 4.0 * pairs * head_dim > 6e11:   # a long chunk on a long context: a shorter chunk
            q_len = max(1, min(int(2.5e9 / (ratio * kv_heads * context * seqs)),
                               int(1.5e11 / (head_dim * ratio * kv_heads * context * seqs))))
        window = rng.choice([0, 0, _spread_over(rng, 16, 8192)])
        c = _attention("", dtype, seqs, context, q_len, ratio * kv_heads, kv_heads, head_dim, group, page,
                       spread=round(rng.uniform(0.0, 0.9), 2), window=window,
                       sinks=rng.choice([0, 4, rng.randint(1, 64)]) if window else 0,
                       empty=1 if seqs > 3 and rng.random() < 0.3 else 0)
    elif op == "append":
        c = _append("", dtype, _spread_over(rng, 1, 8191), kv_heads, head_dim, group, page, padded=rng.choice([0, 0, 1]))
    elif op == "rope":
        rot = rng.choice([r for r in (32, 64, 128, head_dim) if r <= head_dim])
        c = _rope("", dtype, _spread_over(rng, 1, 8191), kv_heads * rng.choice([1, 2, 4, 8]), kv_heads, head_dim, rot,
                  rng.random() < 0.5, rng.random() < 0.7, _spread_over(rng, 64, 131072))
    else:
        moved = _spread_over(rng, 1, 256)
        layers = rng.randint(1, 32)
        page_bytes = kv_heads * page * (head_dim + 8 * head_dim // group)
        moved = max(1, min(moved, int(3e8 / (layers * page_bytes))))
        c = _copy("", layers, 2 * moved + rng.randint(0, 40), moved, kv_heads, head_dim, group, page)
    del c["name"]
    return c


def _contexts(case):
    """Cached tokens of each sequence: the longest, and others down by up to `spread`; unused slots of the batch last."""
    n, longest = case["seqs"], case["context"]
    r = random.Random(1000003 * n + longest)
    got = [longest] + [max(1, int(longest * (1.0 - case["spread"] * r.random()))) for _ in range(n - 1)]
    for i in range(case["empty"]):
        got[n - 1 - i] = 0
    return got


def _queries(case):
    """New tokens of each sequence (part of its cached ones); an unused slot has the one row that the batch keeps for it."""
    ctx, q = _contexts(case), case["q_len"]
    if q == 1:
        return [1] * len(ctx)
    return [max(1, min(c, q - (i * 517) % (q // 2 + 1))) if c else 0 for i, c in enumerate(ctx)]


def _visible(case, position):
    """Keys that a query at `position` sees."""
    seen = position + 1
    w, s = case["window"], case["sinks"]
    if w and seen > w:
        seen = w + min(s, seen - w)
    return max(0, seen)


def _needed(case, first, last):
    """Cached tokens that the queries at positions first..last need between them."""
    if last < 0:
        return 0
    if not case["window"]:
        return last + 1
    low = max(0, first - case["window"] + 1)
    return last + 1 - low + min(case["sinks"], low)


def work(case):
    d, h = case["head_dim"], case["kv_heads"]
    if case["op"] == "rope":
        n = case["tokens"] * (case["q_heads"] + h)
        return {"bytes": 4.0 * n * d + case["tokens"] * (8 + 4 * case["rot"]), "flops": float(n * (3 * case["rot"] + 3 * d))}
    token = h * (d + 8 * d // case["group"])
    if case["op"] == "append":
        n = case["tokens"]
        return {"bytes": float(n * (8 * h * d + token + 8)), "flops": 8.0 * n * h * d}
    if case["op"] == "copy":
        return {"bytes": 2.0 * case["layers"] * case["moved"] * case["page"] * token, "flops": 0.0}
    ctx, qs, r = _contexts(case), _queries(case), case["q_heads"]
    tokens = sum(_needed(case, c - n, c - 1) for c, n in zip(ctx, qs) if n)
    pairs = sum(_visible(case, c - n + i) for c, n in zip(ctx, qs) for i in range(n))
    return {"bytes": float(tokens * token + sum(qs) * r * (4 * d + 4)), "flops": 4.0 * pairs * r * d}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _head_values(shape, generator, dtype):
    """Keys or values as a layer makes them: normal, some channels of a head larger than others."""
    channel = torch.exp(0.4 * torch.randn(shape[1:], generator=generator, device="cuda"))
    return (torch.randn(shape, generator=generator, device="cuda") * channel).to(dtype)


def _new_cache(pages, case, generator):
    """A cache whose memory holds whatever was there before."""
    d = case["head_dim"]
    shape = (pages, case["kv_heads"], case["page"], (d + 8 * d // case["group"]) // 4)
    words = torch.randint(-2**31, 2**31, shape, generator=generator, device="cuda", dtype=torch.int32)
    return words.view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    d, h = case["head_dim"], case["kv_heads"]
    state = {"case": case}
    if case["op"] == "attention":
        dtype, page = TYPES[case["dtype"]], case["page"]
        ctx, qs = _contexts(case), _queries(case)
        width = max(1, -(-max(ctx) // page))
        pages = sum(-(-c // page) for c in ctx) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        table = torch.full((len(ctx), width), -1, dtype=torch.int32, device="cuda")
        cache = _new_cache(pages, case, g)
        at = 0
        for i, c in enumerate(ctx):      # a sequence at a time, to keep the memory of this small
            n = -(-c // page)
            table[i, :n] = order[at:at + n].int()
            at += n
            if c:
                j = torch.arange(c, device="cuda")
                slots = table[i].long()[j // page] * page + j % page
                _store(_head_values((c, h, d), g, dtype), _head_values((c, h, d), g, dtype), slots, cache)
        if case["window"]:               # pages that no query sees any more went back to the pool
            first = torch.tensor([c - n for c, n in zip(ctx, qs)], device="cuda")[:, None]
            start = torch.arange(width, device="cuda")[None] * page
            gone = (start + page - 1 < first - case["window"] + 1) & (start >= case["sinks"])
            table[gone] = -1
        starts = [0]
        for n in qs:
            starts.append(starts[-1] + n)
        # queries of a size that gives scores of a few units
        q = torch.randn((starts[-1], case["q_heads"], d), generator=g, device="cuda") * 1.2
        state.update(q=q.to(dtype), cache=cache, table=table,
                     context=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                     starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), longest=max(qs))
    elif case["op"] == "append":
        n, page = case["tokens"], case["page"]
        dtype = TYPES[case["dtype"]]
        pages = -(-n // page) * (page if n <= 64 else 1) + 5
        if n <= 64:     # a step's tokens: each at the end of a sequence of its own
            at = torch.randperm(pages, generator=g, device="cuda")[:n] * page
            slots = at + torch.randint(0, page, (n,), generator=g, device="cuda")
        else:           # a prompt's tokens: page after page
            j = torch.arange(n, device="cuda")
            slots = torch.randperm(pages, generator=g, device="cuda")[j // page] * page + j % page
        if n > case["padded"] > 0:
            slots[-case["padded"]:] = -1
        state.update(k=_head_values((n, h, d), g, dtype), v=_head_values((n, h, d), g, dtype), slots=slots,
                     cache=_new_cache(pages, case, g))
    elif case["op"] == "rope":
        n, dtype = case["tokens"], TYPES[case["dtype"]]
        half = case["rot"] // 2
        angle = torch.arange(case["positions"], device="cuda", dtype=torch.float64)[:, None] * \
            500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        weight = lambda: (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype) if case["norm"] else None
        state.update(q=_head_values((n, case["q_heads"], d), g, dtype), k=_head_values((n, h, d), g, dtype),
                     positions=torch.randint(0, case["positions"], (n,), generator=g, device="cuda"),
                     table=torch.stack((angle.cos(), angle.sin()), -1).float(), q_weight=weight(), k_weight=weight())
    else:
        cache = torch.stack([_new_cache(case["pages"], case, g) for _ in range(case["layers"])])
        order = torch.randperm(case["pages"], generator=g, device="cuda")
        src, dst = order[:case["moved"]].clone(), order[-case["moved"]:].clone()
        state.update(cache=cache, src=src, dst=dst)
    return state


# ---------------------------------------------------------------------------
# The plain form.
# ---------------------------------------------------------------------------
def _quantize(x, group):
    """Codes, zero-points and scales of x [tokens, heads, channels], group by group."""
    x = x.float().unflatten(-1, (-1, group))
    low, high = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
    # divided by a tensor: a division by a number may be done as a product
    scale = ((high - low) / torch.full_like(low, 15.0)).clamp(max=65504.0).half().float()
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    zero = torch.round(-low / scale).clamp(0, 15)
    code = (torch.round(x / scale[..., None]) + zero[..., None]).clamp(0, 15)
    return code.flatten(-2).int(), zero.int(), scale


def _shifts(device):
    """Places of the eight channels of a code word, in bits."""
    e = torch.arange(8, device=device, dtype=torch.int32)
    return 4 * (e // 2) + 16 * (e % 2)


def _words(code):
    """Code words [..., D/8] of codes [..., D]."""
    return (code.unflatten(-1, (-1, 8)) << _shifts(code.device)).sum(-1, dtype=torch.int32)


def _parts(cache, head_dim):
    """The parts of a cache, as words of 32 bits: K codes [pages, heads, page, 4, D/32], V codes [pages, heads, page/4,
    D/8, 4], K and V params [pages, heads, groups, page]."""
    pages, heads, page, token = cache.shape
    words = cache.view(torch.int32).view(pages, heads, -1)
    groups = (token - head_dim) // 8
    sizes = [page * head_dim // 8, page * head_dim // 8, page * groups, page * groups]
    k, v, kp, vp = words.split(sizes, -1)
    return (k.unflatten(-1, (page, 4, head_dim // 32)), v.unflatten(-1, (page // 4, head_dim // 8, 4)),
            kp.unflatten(-1, (groups, page)), vp.unflatten(-1, (groups, page)))


def _store(k, v, slots, cache):
    """Tokens into the cache; a slot outside of it takes none (one token at least has a slot)."""
    page, d = cache.shape[2], k.shape[-1]
    group = 8 * d // (cache.shape[3] - d)
    k_codes, v_codes, k_params, v_params = _parts(cache, d)
    kept = (slots >= 0) & (slots < cache.shape[0] * page)
    # in the place of a token without a slot the first one that has one, once more
    at = torch.where(kept, torch.arange(len(slots), device=slots.device), kept.int().argmax())
    k, v, slots = k[at], v[at], slots[at]
    p, t = slots // page, slots % page
    code, zero, scale = _quantize(k, group)
    k_codes[p, :, t] = _words(code).unflatten(-1, (-1, 4)).transpose(-1, -2)
    k_params[p, :, :, t] = scale.half().view(torch.int16).int() | (zero << 16)
    code, zero, scale = _quantize(v, group)
    v_codes[p, :, t // 4, :, t % 4] = _words(code)
    v_params[p, :, :, t] = scale.half().view(torch.int16).int() | (zero << 16)


def _values(words, params):
    """fp32 values [..., D] of code words [..., D/8] in the channels' order and params [..., groups]."""
    code = ((words[..., None] >> _shifts(words.device)) & 15).flatten(-2).float()
    scale = (params & 0xFFFF).short().view(torch.float16).float()
    zero = ((params >> 16) & 15).float()
    code = code.unflatten(-1, (params.shape[-1], -1))
    return ((code - zero[..., None]) * scale[..., None]).flatten(-2)


def _fetch(cache, slots, head_dim):
    """fp32 K and V [tokens, heads, D] of slots of the cache; zeros for a slot outside of it."""
    page = cache.shape[2]
    k_codes, v_codes, k_params, v_params = _parts(cache, head_dim)
    kept = ((slots >= 0) & (slots < cache.shape[0] * page))[:, None, None]
    at = slots.clamp(0, cache.shape[0] * page - 1)
    p, t = at // page, at % page
    k = _values(k_codes[p, :, t].transpose(-1, -2).flatten(-2), k_params[p, :, :, t])
    v = _values(v_codes[p, :, t // 4, :, t % 4], v_params[p, :, :, t])
    return torch.where(kept, k, torch.zeros_like(k)), torch.where(kept, v, torch.zeros_like(v))


def _plain_attention(s):
    case, q, table = s["case"], s["q"], s["table"]
    seqs, width = table.shape
    heads, d, page = case["kv_heads"], case["head_dim"], case["page"]
    ratio, most = case["q_heads"] // heads, s["longest"]
    tokens = width * page
    j = torch.arange(tokens, device=q.device)
    here = (table >= 0).repeat_interleave(page, 1)
    slots = torch.where(here, table.long().repeat_interleave(page, 1) * page + j % page, -1)
    k, v = _fetch(s["cache"], slots.reshape(-1), d)
    k = k.view(seqs, tokens, heads, d).permute(0, 2, 3, 1)
    v = v.view(seqs, tokens, heads, d).permute(0, 2, 1, 3)
    # the queries, a sequence to a row, padded to the longest
    i = torch.arange(most, device=q.device)
    count = (s["starts"][1:] - s["starts"][:-1]).long()[:, None]
    row = (s["starts"][:-1].long()[:, None] + i).clamp(max=q.shape[0] - 1)
    qp = q[row].float().view(seqs, most, heads, ratio, d).permute(0, 2, 1, 3, 4).reshape(seqs, heads, most * ratio, d)
    context = s["context"].long()[:, None]
    position = context - count + i
    seen = (j <= position[..., None]) & here[:, None, :]
    if case["window"]:
        seen &= (j > position[..., None] - case["window"]) | (j < case["sinks"])
    seen = seen.repeat_interleave(ratio, 1)[:, None]
    # what lies behind a sequence's end may be anything
    v = torch.where((j < context)[:, None, :, None], v, torch.zeros_like(v))
    score = torch.where(seen, torch.matmul(qp * (1.0 / math.sqrt(d)), k), -math.inf)
    most_of = score.amax(-1, keepdim=True)
    most_of = torch.where(most_of == -math.inf, torch.zeros_like(most_of), most_of)
    p = torch.exp(score - most_of)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = torch.where(total == 0, -math.inf, most_of + torch.log(total))
    r = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(s["starts"].long(), r, right=True) - 1
    r = r - s["starts"].long()[b]
    back = lambda x: x.view(seqs, heads, most, ratio, -1)[b, :, r].flatten(1, 2)
    return {"out": back(o).to(q.dtype), "lse": back(lse)[..., 0]}


def _rotate(x, weight, cos_sin, interleaved):
    dtype, x = x.dtype, x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    cos, sin = cos_sin[:, None, :, 0], cos_sin[:, None, :, 1]
    r = 2 * cos.shape[-1]
    turned = x[..., :r]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :r // 2], turned[..., r // 2:])
    c, e = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((c, e), -1).flatten(-2) if interleaved else torch.cat((c, e), -1)
    return torch.cat((turned, x[..., r:]), -1).to(dtype)


def _plain(s):
    case = s["case"]
    if case["op"] == "attention":
        return _plain_attention(s)
    if case["op"] == "append":
        _store(s["k"], s["v"], s["slots"], s["cache"])
        k, v = _fetch(s["cache"], s["slots"], case["head_dim"])
        return {"k": k.to(s["k"].dtype), "v": v.to(s["v"].dtype)}
    if case["op"] == "rope":
        at = s["table"][s["positions"]]
        return {"q": _rotate(s["q"], s["q_weight"], at, case["interleaved"]),
                "k": _rotate(s["k"], s["k_weight"], at, case["interleaved"])}
    s["cache"][:, s["dst"]] = s["cache"][:, s["src"]]
    return {"cache": s["cache"].view(torch.int32)}


def _own(s):
    import quantized_matmul_quantize_amd as qmm
    case = s["case"]
    if case["op"] == "attention":
        out, lse = qmm.kv4_attention(s["q"], s["cache"], s["table"], s["context"], window=case["window"],
                                     sinks=case["sinks"], return_lse=True,
                                     **({} if case["q_len"] == 1 else {"cu_q": s["starts"], "max_q": s["longest"]}))
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        qmm.kv4_append(s["k"], s["v"], s["slots"], s["cache"])
        k, v = qmm.kv4_read(s["cache"], s["slots"], case["head_dim"], dtype=s["k"].dtype)
        return {"k": k, "v": v}
    if case["op"] == "rope":
        q, k = qmm.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], s["q_weight"], s["k_weight"], eps=1e-6,
                                interleaved=case["interleaved"])
        return {"q": q, "k": k}
    qmm.kv4_copy_pages(s["cache"], s["src"], s["dst"])
    return {"cache": s["cache"].view(torch.int32)}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definition in 64 bits.
# ---------------------------------------------------------------------------
def _value64(page_words, offset_of, params, group):
    """Values of channels through the place of each channel's nibble: page_words [n, words], offset_of [D] word of each
    channel, params [n, groups]."""
    d = offset_of.shape[0]
    c = torch.arange(d, device=page_words.device)
    code = torch.bitwise_right_shift(page_words.long()[:, offset_of], 4 * ((c % 8) // 2) + 16 * (c % 2)) % 16
    bits = params.long()[:, c // group]
    exponent, fraction = bits // 1024 % 32, bits % 1024
    scale = torch.where(exponent == 0, fraction.double() * 2.0**-24,
                        (1.0 + fraction.double() / 1024) * torch.pow(2.0, exponent.double() - 15))
    return (code - bits // 65536 % 16).double() * scale


def _sequence64(s, b, head):
    """K and V [context, D] of one sequence and head in fp64."""
    case = s["case"]
    d, page, group = case["head_dim"], case["page"], case["group"]
    n = int(s["context"][b])
    j = torch.arange(n, device="cuda")
    at = s["table"][b].long()[j // page].clamp(min=0)
    words = s["cache"].view(torch.int32)[:, head].flatten(1)
    c, t = torch.arange(d, device="cuda"), j % page
    w = c // 8
    half, groups = page * d // 8, d // group
    k_at = t[:, None] * (d // 8) + ((w % 4) * (d // 32) + w // 4)[None]
    v_at = half + (t // 4 * (d // 2))[:, None] + 4 * w[None] + (t % 4)[:, None]
    p_at = 2 * half + torch.arange(groups, device="cuda")[None] * page + t[:, None]
    k = _value64(words[at[:, None], k_at], c, words[at[:, None], p_at], group)
    v = _value64(words[at[:, None], v_at], c, words[at[:, None], p_at + groups * page], group)
    return k, v


def _exact_attention(case, seed):
    if sum(_contexts(case)) * case["kv_heads"] * case["head_dim"] > 3e8:
        return None      # too long in 64 bits
    s = prepare(case, seed)
    ratio, d = case["q_heads"] // case["kv_heads"], case["head_dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, (ctx, n) in enumerate(zip(_contexts(case), _queries(case))):
        if not ctx or not n:
            continue
        at = int(s["starts"][b])
        p = torch.arange(ctx - n, ctx, device="cuda")[:, None]
        j = torch.arange(ctx, device="cuda")[None]
        hidden = j > p
        if case["window"]:
            hidden |= (p - j >= case["window"]) & (j >= case["sinks"])
        for head in range(case["kv_heads"]):
            k, v = _sequence64(s, b, head)
            for r in range(head * ratio, (head + 1) * ratio):
                x = (s["q"][at:at + n, r].double() @ k.T) / math.sqrt(d)
                x = x.masked_fill(hidden, -math.inf)
                lse[at:at + n, r] = torch.logsumexp(x, -1)
                out[at:at + n, r] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(case, seed)
    if case["op"] == "copy":
        return None      # bytes moved, nothing computed
    s = prepare(case, seed)
    if case["op"] == "append":
        got = {}
        for name in ("k", "v"):
            x = s[name].double().view(case["tokens"], case["kv_heads"], -1, case["group"])
            low = torch.minimum(x.min(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device="cuda"))
            high = torch.maximum(x.max(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device="cuda"))
            step = ((high - low) / 15).half().double()
            zero = (-low / step).round().clamp(0, 15)
            value = ((x / step).round() + zero).clamp(0, 15).sub(zero).mul(step).reshape(s[name].shape)
            got[name] = value * (s["slots"] >= 0).double()[:, None, None]
        return got
    angle = s["table"][s["positions"]].double()
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        if case["norm"]:
            x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * s[name + "_weight"].double()
        y = x.clone()
        half = case["rot"] // 2
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            cos, sin = angle[:, None, i, 0], angle[:, None, i, 1]
            y[..., a] = x[..., a] * cos - x[..., b] * sin
            y[..., b] = x[..., b] * cos + x[..., a] * sin
        got[name] = y
    return got
