"""Measured cases of decoding several continuations of one prompt over the 4-bit paged key/value cache: attention
that reads a shared prefix once, the append with norms and rotation on the way, the selection of beams, and the
reordering of their cache.

`run` computes a case either with elementary torch operations (the plain form, `own` false) or with this package's
calls (`own` true), on the same inputs.  Both work on the same packed cache:

  cache  uint8 [pages, kv_heads, page, D + 8 D/g], of which the bytes of one (page, head) are
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

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def _prefix(name, dtype, groups, branches, prefix, tail, q_len, q_heads, kv_heads, head_dim, group, page, spread=0.0,
            empty=0):
    return {"name": name, "op": "prefix", "dtype": dtype, "groups": groups, "branches": branches, "prefix": prefix,
            "tail": tail, "q_len": q_len, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "group": group, "page": page, "spread": spread, "empty": empty}


def _append(name, dtype, tokens, q_heads, kv_heads, head_dim, group, page, rot, interleaved, norm, positions, padded=0):
    return {"name": name, "op": "append", "dtype": dtype, "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "group": group, "page": page, "rot": rot, "interleaved": interleaved, "norm": norm,
            "positions": positions, "padded": padded}


def _select(name, dtype, seqs, beams, vocabulary, k, finished=0, banned=0, padded=0):
    return {"name": name, "op": "select", "dtype": dtype, "seqs": seqs, "beams": beams, "vocabulary": vocabulary,
            "k": k, "finished": finished, "banned": banned, "padded": padded}


def _reorder(name, layers, seqs, beams, prompt, generated, kv_heads, head_dim, group, page):
    return {"name": name, "op": "reorder", "layers": layers, "seqs": seqs, "beams": beams, "prompt": prompt,
            "generated": generated, "kv_heads": kv_heads, "head_dim": head_dim, "group": group, "page": page}


def listed():
    return [
        # one user's prompt, four beams a few tokens in: latency counts
        _prefix("prefix_beams", "bf16", 1, 4, 1000, 40, 1, 32, 8, 128, 64, 64),
        # 64 samples of one 4k prompt, some hundred tokens of their own each
        _prefix("prefix_samples", "bf16", 1, 64, 4096, 300, 1, 32, 8, 128, 128, 64, spread=0.5),
        # a batch of prompts with a few branches each, three drafted tokens to verify, small heads, an unused slot
        _prefix("prefix_drafts", "fp16", 12, 9, 6001, 777, 3, 16, 2, 64, 32, 32, spread=0.6, empty=1),
        # many questions on two long documents
        _prefix("prefix_document", "bf16", 2, 24, 100000, 513, 1, 64, 8, 128, 64, 128, spread=0.3),
        # a decode step's heads of 64 sequences, three slots of the batch unused
        _append("append_step", "bf16", 64, 32, 8, 128, 64, 64, 128, False, True, 131072, padded=3),
        # an odd chunk of prompts of an older layout: interleaved pairs, half the head rotated, no norms
        _append("append_odd", "fp16", 1023, 16, 16, 64, 32, 16, 32, True, False, 4096),
        # a prompt's chunk
        _append("append_prompt", "bf16", 8191, 32, 8, 128, 64, 64, 128, False, True, 32768),
        # one user's four beams on a small vocabulary
        _select("select_one", "fp32", 1, 4, 32768, 4),
        # odd vocabulary, some beams finished, banned tokens
        _select("select_odd", "fp16", 7, 5, 100003, 5, finished=1, banned=50),
        # a serving batch: twice as many candidates as beams, so that those that end can be set aside
        _select("select_batch", "bf16", 64, 8, 131072, 16, padded=64),
        # one user's four beams, every layer's cache
        _reorder("reorder_one", 32, 1, 4, 1000, 100, 8, 128, 64, 64),
        # a serving batch of beams
        _reorder("reorder_batch", 16, 16, 8, 2000, 150, 8, 128, 64, 64),
    ]


def _spread_over(rng, low, high):
    """A whole number of [low, high], evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "append", "select", "select", "reorder"])
    head_dim = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if head_dim % g == 0])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "prefix":
        ratio = rng.choice([1, 2, 3, 4, 5, 7, 8])
        branches, groups = _spread_over(rng, 1, 64), _spread_over(rng, 1, 12)
        q_len = rng.choice([1, 1, 1, rng.randint(2, 6)])
        prefix, tail = _spread_over(rng, 16, 100000), _spread_over(rng, q_len, 1000)
        rows = groups * branches * q_len * ratio * kv_heads
        prefix = max(1, min(prefix, int(1.5e11 / (4 * rows * head_dim)), int(2.9e8 / (groups * kv_heads * head_dim)),
                            int(8e8 / rows)))
        c = _prefix("", dtype, groups, branches, prefix, tail, q_len, ratio * kv_heads, kv_heads, head_dim, group,
                    page, spread=round(rng.uniform(0.0, 0.8), 2), empty=1 if branches > 2 and rng.random() < 0.3 else 0)
    elif op == "append":
        rot = rng.choice([r for r in (32, 64, 128, head_dim) if r <= head_dim])
        tokens = _spread_over(rng, 1, 8191)
        q_heads = kv_heads * rng.choice([1, 2, 4])
        tokens = max(1, min(tokens, int(3.5e7 / ((q_heads + kv_heads) * head_dim))))
        c = _append("", dtype, tokens, q_heads, kv_heads, head_dim, group, page, rot, rng.random() < 0.5,
                    rng.random() < 0.7, _spread_over(rng, 64, 131072), padded=rng.choice([0, 0, 1]))
    elif op == "select":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        beams, vocabulary = rng.randint(1, 16), _spread_over(rng, 1000, 131072)
        seqs = max(1, min(_spread_over(rng, 1, 64), int(3.2e7 / (beams * vocabulary))))
        c = _select("", dtype, seqs, beams, vocabulary, rng.choice([beams, 2 * beams, rng.randint(1, 32)]),
                    finished=rng.choice([0, 1]) if beams > 1 else 0, banned=rng.choice([0, 20]),
                    padded=rng.choice([0, 1, 61]))
    else:
        beams, seqs, layers = rng.randint(2, 12), _spread_over(rng, 1, 16), rng.randint(1, 32)
        page_bytes = kv_heads * page * (head_dim + 8 * head_dim // group)
        seqs = max(1, min(seqs, int(4.5e8 / (beams * layers * page_bytes))))
        prompt = _spread_over(rng, 1, 2000)
        prompt = max(1, min(prompt, int(1e9 / (seqs * layers * page_bytes)) * page))
        c = _reorder("", layers, seqs, beams, prompt, _spread_over(rng, 1, 3 * page), kv_heads, head_dim, group, page)
    del c["name"]
    return c


def _branches(case):
    """Per group (tokens of the prefix, tokens of each branch after it); an unused slot of the batch has None."""
    r = random.Random(7919 * case["groups"] + 31 * case["branches"] + case["prefix"])
    less = lambda most: max(1, int(most * (1.0 - case["spread"] * r.random())))
    got = []
    for g in range(case["groups"]):
        n = case["branches"] if g == 0 else less(case["branches"])
        p = case["prefix"] if g == 0 else less(case["prefix"])
        got.append((p, [case["tail"] if i == 0 else max(case["q_len"], less(case["tail"])) for i in range(n)]))
    if case["empty"]:
        got[-1][1][-1] = None
    return got


def _generated(case):
    """Tokens of each sequence of beams: prompt and generated."""
    r = random.Random(104729 * case["seqs"] + case["prompt"])
    return [(max(1, case["prompt"] - r.randint(0, case["prompt"] // 2)), r.randint(1, case["generated"]))
            for _ in range(case["seqs"])]


def _parents(case):
    """The beam that each beam goes on from: about half go on from themselves."""
    r = random.Random(15485863 * case["seqs"] + case["beams"])
    return [[b if r.random() < 0.5 else r.randrange(case["beams"]) for b in range(case["beams"])]
            for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "select":
        rows = case["seqs"] * case["beams"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": float((rows - case["seqs"] * case["finished"]) * case["vocabulary"] * size + 4 * rows +
                               20 * case["seqs"] * case["k"]),
                "flops": 4.0 * (rows - case["seqs"] * case["finished"]) * case["vocabulary"]}
    d, h = case["head_dim"], case["kv_heads"]
    token = h * (d + 8 * d // case["group"])
    if case["op"] == "append":
        n, hq = case["tokens"], case["q_heads"]
        return {"bytes": float(n * (4 * hq * d + 8 * h * d + token + 16 + 4 * case["rot"])),
                "flops": float(n * ((hq + h) * (3 * case["rot"] + 3 * d) + 16 * h * d))}
    if case["op"] == "reorder":
        moved = 0
        for (prompt, generated), parents in zip(_generated(case), _parents(case)):
            filled = (prompt + generated) % case["page"]
            moved += -(-filled // 4) * 4 * sum(b != p for b, p in enumerate(parents))
        slots = case["seqs"] * case["beams"]
        width = -(-max(sum(x) for x in _generated(case)) // case["page"])
        return {"bytes": float(2 * case["layers"] * moved * token + slots * (8 * width + 24)), "flops": 0.0}
    tokens = pairs = rows = 0
    q = case["q_len"]
    for prefix, tails in _branches(case):
        tokens += prefix + sum(t or 0 for t in tails)
        rows += q * len(tails)
        pairs += sum(q * (prefix + t) - q * (q - 1) // 2 for t in tails if t)
    return {"bytes": float(tokens * token + rows * case["q_heads"] * (4 * d + 4)), "flops": 4.0 * pairs * case["q_heads"] * d}


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


def _prepare_prefix(case, g):
    d, h, page, dtype = case["head_dim"], case["kv_heads"], case["page"], TYPES[case["dtype"]]
    plan, q_len = _branches(case), case["q_len"]
    tables, context, sizes, free = [], [], [], 0
    for prefix, tails in plan:
        whole = prefix // page
        shared = list(range(free, free + whole))
        free += whole
        for t in tails:
            total = prefix + t if t else 0
            mine = list(range(free, free + -(-total // page) - whole)) if t else []
            free += len(mine)
            tables.append(shared + mine if t else [])
            context.append(total)
        sizes.append(len(tails))
    width, seqs = max(len(t) for t in tables), len(tables)
    pages = free + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
    for b, t in enumerate(tables):
        if t:
            table[b, :len(t)] = order[torch.tensor(t, device="cuda")]
    cache = _new_cache(pages, case, g)
    b = 0
    for prefix, tails in plan:            # a group at a time, to keep the memory of this small
        k, v = _head_values((prefix, h, d), g, dtype), _head_values((prefix, h, d), g, dtype)
        first = True
        for t in tails:
            if t:
                # the page in which the prefix ends is each branch's own, with the same tokens in it
                start = 0 if first else prefix // page * page
                j = torch.arange(start, prefix + t, device="cuda")
                slots = table[b].long()[j // page] * page + j % page
                _store(torch.cat((k[start:], _head_values((t, h, d), g, dtype))),
                       torch.cat((v[start:], _head_values((t, h, d), g, dtype))), slots, cache)
                first = False
            b += 1
    bounds = [0]
    for n in sizes:
        bounds.append(bounds[-1] + n)
    # queries of a size that gives scores of a few units
    q = torch.randn((seqs * q_len, case["q_heads"], d), generator=g, device="cuda") * 1.2
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return dict(q=q.to(dtype), cache=cache, table=table, context=ints(context), groups=ints(bounds),
                prefix=ints([p for p, _ in plan]), starts=ints([q_len * b for b in range(seqs + 1)]),
                most_group=max(sizes), most_prefix=max(p for p, _ in plan),
                most_tail=max(t or 0 for _, x in plan for t in x))


def _prepare_append(case, g):
    n, h, d, page, dtype = case["tokens"], case["kv_heads"], case["head_dim"], case["page"], TYPES[case["dtype"]]
    pages = -(-n // page) * (page if n <= 64 else 1) + 5
    if n <= 64:         # a step's tokens: each at the end of a sequence of its own
        at = torch.randperm(pages, generator=g, device="cuda")[:n] * page
        slots = at + torch.randint(0, page, (n,), generator=g, device="cuda")
    else:               # a prompt's tokens: page after page
        j = torch.arange(n, device="cuda")
        slots = torch.randperm(pages, generator=g, device="cuda")[j // page] * page + j % page
    if n > case["padded"] > 0:
        slots[-case["padded"]:] = -1
    half = case["rot"] // 2
    angle = torch.arange(case["positions"], device="cuda", dtype=torch.float64)[:, None] * \
        500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    weight = lambda: (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype) if case["norm"] else None
    # queries, keys and values are parts of one projection's output
    qkv = torch.cat([_head_values((n, x, d), g, dtype) for x in (case["q_heads"], h, h)], 1)
    q, k, v = qkv.split([case["q_heads"], h, h], 1)
    return dict(q=q, k=k, v=v, slots=slots, positions=torch.randint(0, case["positions"], (n,), generator=g, device="cuda"),
                table=torch.stack((angle.cos(), angle.sin()), -1).float(), q_weight=weight(), k_weight=weight(),
                cache=_new_cache(pages, case, g))


def _prepare_select(case, g):
    seqs, beams, vocabulary = case["seqs"], case["beams"], case["vocabulary"]
    rows = seqs * beams
    # logits of a model: most tokens are unlikely, a few far above the others
    x = torch.randn((rows, vocabulary + case["padded"]), generator=g, device="cuda") * 2.0
    likely = (torch.randint(0, vocabulary, (rows, 1), generator=g, device="cuda") +
              torch.arange(24, device="cuda") * (vocabulary // 24)) % vocabulary          # distinct ones
    x.scatter_add_(1, likely, 6.0 + 4.0 * torch.rand((rows, 24), generator=g, device="cuda"))
    if case["banned"]:
        x.scatter_(1, torch.randint(0, vocabulary, (rows, case["banned"]), generator=g, device="cuda"), -math.inf)
    scores = -20.0 * torch.rand((seqs, 1), generator=g, device="cuda") - \
        3.0 * torch.rand((seqs, beams), generator=g, device="cuda").cumsum(1)
    finished = torch.zeros((seqs, beams), dtype=torch.bool, device="cuda")
    finished[:, :case["finished"]] = True
    return dict(logits=x.to(TYPES[case["dtype"]])[:, :vocabulary], scores=scores, finished=finished)


def _prepare_reorder(case, g):
    seqs, beams, page = case["seqs"], case["beams"], case["page"]
    plan, free = _generated(case), 0
    rows, tails, context = [], [], []
    r = random.Random(seqs)
    for prompt, generated in plan:
        whole, total = prompt // page, prompt + generated
        shared = list(range(free, free + whole))
        free += whole
        for _ in range(beams):
            full = total // page - whole                     # pages since the prompt that are full
            mine = list(range(free, free + full))
            pair = [free + full, free + full + 1]
            free += full + 2
            rows.append(shared + mine + ([pair[r.randrange(2)]] if total % page else []))
            tails.append(pair)
            context.append(total)
    width = max(len(x) for x in rows)
    cache = torch.stack([_new_cache(free, case, g) for _ in range(case["layers"])])
    order = torch.randperm(free, generator=g, device="cuda").int()
    table = torch.full((len(rows), width), -1, dtype=torch.int32, device="cuda")
    for i, x in enumerate(rows):
        table[i, :len(x)] = order[torch.tensor(x, device="cuda", dtype=torch.int64)]
    return dict(cache=cache, table=table, tails=order[torch.tensor(tails, device="cuda")],
                context=torch.tensor(context, dtype=torch.int32, device="cuda"),
                parents=torch.tensor(_parents(case), dtype=torch.int64, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = {"prefix": _prepare_prefix, "append": _prepare_append, "select": _prepare_select, "reorder": _prepare_reorder}
    return {"case": case, **make[case["op"]](case, g)}


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


def _part_of(q, cache, slots, seen):
    """Maximum, sum and weighted values of rows q [n, heads, rows, D] over the keys in slots [n, keys], where `seen`
    [n, rows, keys]."""
    n, keys = slots.shape
    heads, d = q.shape[1], q.shape[-1]
    k, v = _fetch(cache, slots.reshape(-1), d)
    k = k.view(n, keys, heads, d).permute(0, 2, 3, 1)
    v = v.view(n, keys, heads, d).permute(0, 2, 1, 3)
    seen = seen & (slots >= 0)[:, None, :]
    v = torch.where(seen.any(1)[:, None, :, None], v, torch.zeros_like(v))      # what is hidden may be anything
    score = torch.where(seen[:, None], torch.matmul(q * (1.0 / math.sqrt(d)), k), -math.inf)
    most = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(most == -math.inf, torch.zeros_like(most), most))
    return most, p.sum(-1, keepdim=True), torch.matmul(p, v)


def _plain_prefix(s):
    case, table = s["case"], s["table"].long()
    seqs, width = table.shape
    heads, d, page, n = case["kv_heads"], case["head_dim"], case["page"], case["q_len"]
    ratio, device = case["q_heads"] // heads, table.device
    context, prefix, groups = s["context"].long(), s["prefix"].long(), s["groups"].long()
    slots_of = lambda rows, j: torch.where(
        (j < width * page) & (rows.gather(1, (j // page).clamp(max=width - 1)) >= 0),
        rows.gather(1, (j // page).clamp(max=width - 1)) * page + j % page, -1)
    q = s["q"].float().view(seqs, n, heads, ratio, d).permute(0, 2, 1, 3, 4).reshape(seqs, heads, n * ratio, d)
    position = (context[:, None] - n + torch.arange(n, device=device)).repeat_interleave(ratio, 1)       # [seqs, rows]
    # the prefix: the rows of a group's sequences side by side
    count = groups[1:] - groups[:-1]
    member = torch.arange(s["most_group"], device=device)
    here = member < count[:, None]
    member = torch.where(here, groups[:-1, None] + member, 0)
    j = torch.arange(s["most_prefix"], device=device).expand(len(count), -1)
    rows = q[member].permute(0, 2, 1, 3, 4).flatten(2, 3)
    at = position[member].flatten(1)
    of_group = _part_of(rows, s["cache"], slots_of(table[groups[:-1]], j),
                        (j < prefix[:, None])[:, None] & (j[:, None] <= at[..., None]))
    mine = torch.searchsorted(groups, torch.arange(seqs, device=device), right=True) - 1
    back = lambda x: x.unflatten(2, (s["most_group"], n * ratio))[mine, :, torch.arange(seqs, device=device) - groups[mine]]
    m0, l0, o0 = (back(x) for x in of_group)
    # each sequence's own tokens
    j = prefix[mine][:, None] + torch.arange(max(1, s["most_tail"]), device=device)
    m1, l1, o1 = _part_of(q, s["cache"], slots_of(table, j), j[:, None] <= position[..., None])
    m = torch.maximum(m0, m1)
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)
    f0, f1 = torch.exp(m0 - base), torch.exp(m1 - base)
    total = l0 * f0 + l1 * f1
    o = (o0 * f0 + o1 * f1) / torch.where(total == 0, torch.ones_like(total), total)
    lse = torch.where(total == 0, -math.inf, base + torch.log(total))
    flat = lambda x: x.view(seqs, heads, n, ratio, -1).transpose(1, 2).reshape(seqs * n, heads * ratio, -1)
    return {"out": flat(o).to(s["q"].dtype), "lse": flat(lse)[..., 0]}


def _turned(x, weight, cos_sin, interleaved):
    """Heads x [tokens, heads, D] normed where there is a weight, then their first channels turned, in 64 bits: which
    side of a border a key falls on decides its code."""
    x = x.double()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.double()
    cos, sin = cos_sin[:, None, :, 0], cos_sin[:, None, :, 1]
    r = 2 * cos.shape[-1]
    turned = x[..., :r]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :r // 2], turned[..., r // 2:])
    c, e = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((c, e), -1).flatten(-2) if interleaved else torch.cat((c, e), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _plain_append(s):
    at = s["table"][s["positions"]].double()
    dtype, interleaved = s["q"].dtype, s["case"]["interleaved"]
    _store(_turned(s["k"], s["k_weight"], at, interleaved).float(), s["v"], s["slots"], s["cache"])
    k, v = _fetch(s["cache"], s["slots"], s["case"]["head_dim"])
    return {"q": _turned(s["q"], s["q_weight"], at, interleaved).to(dtype), "k": k.to(dtype), "v": v.to(dtype)}


def _plain_select(s):
    case, x = s["case"], s["logits"].double()          # near ties between beams are decided by their sums
    seqs, beams = s["scores"].shape
    most = x.amax(-1, keepdim=True)
    lse = most + torch.log(torch.exp(x - most).sum(-1, keepdim=True))
    value = (x - lse).view(seqs, beams, -1) + s["scores"].double()[..., None]
    only = torch.where(torch.arange(case["vocabulary"], device=x.device) == 0, s["scores"].double()[..., None], -math.inf)
    value = torch.where(s["finished"][..., None], only, value).flatten(1)
    best, at = torch.sort(value, dim=1, descending=True, stable=True)
    best, at = best[:, :case["k"]], at[:, :case["k"]]
    return {"scores": best.float(), "tokens": at % case["vocabulary"], "parents": at // case["vocabulary"]}


def _plain_reorder(s):
    case, table, context, tails = s["case"], s["table"], s["context"].long(), s["tails"]
    page, d = case["page"], case["head_dim"]
    slots, width = table.shape
    me = torch.arange(slots, device=table.device)
    beams = case["beams"]
    parent = me // beams * beams + s["parents"].flatten()
    column = lambda rows, n: rows.gather(1, (n // page).clamp(max=width - 1)[:, None])[:, 0]
    spare = torch.where(column(table, context) == tails[:, 0], tails[:, 1], tails[:, 0])
    n = context[parent]
    new = table[parent]
    moved = (parent != me) & (n % page != 0)
    source = column(new, n)
    new = torch.where(moved[:, None] & (torch.arange(width, device=table.device) == (n // page)[:, None]),
                      spare[:, None], new)
    # the filled part of a page, in whole fours of tokens; an unmoved slot's page onto itself
    target = torch.where(moved, spare, source).long().clamp(min=0)
    source = source.long().clamp(min=0)
    filled = torch.where(moved, (n % page + 3) // 4 * 4, 0)
    groups = d // case["group"]
    t = torch.arange(page, device=table.device)
    token = torch.cat((t.repeat_interleave(d // 8), t[::4].repeat_interleave(d // 2), t.repeat(2 * groups)))                                # first token of each word of a record
    words = s["cache"].view(torch.int32).flatten(3)
    words[:, target] = torch.where((token < filled[:, None])[:, None], words[:, source], words[:, target])
    return {"table": new, "context": n.int(), "cache": s["cache"].view(torch.int32)}


def _own(s):
    import quantized_matmul_quantize_amd as qmm
    case = s["case"]
    if case["op"] == "prefix":
        ragged = {} if case["q_len"] == 1 else {"cu_q": s["starts"], "max_q": case["q_len"]}
        out, lse = qmm.kv4_prefix_attention(s["q"], s["cache"], s["table"], s["context"], s["groups"], s["prefix"],
                                            max_group=s["most_group"], max_prefix=s["most_prefix"],
                                            max_tail=s["most_tail"], return_lse=True, **ragged)
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        q = qmm.kv4_rope_append(s["q"], s["k"], s["v"], s["slots"], s["cache"], s["positions"], s["table"],
                                s["q_weight"], s["k_weight"], eps=1e-6, interleaved=case["interleaved"])
        k, v = qmm.kv4_read(s["cache"], s["slots"], case["head_dim"], dtype=s["k"].dtype)
        return {"q": q, "k": k, "v": v}
    if case["op"] == "select":
        scores, tokens, parents = qmm.beam_select(s["logits"], s["scores"], case["k"], s["finished"], pad=0)
        return {"scores": scores, "tokens": tokens, "parents": parents}
    table, context = qmm.kv4_beam_reorder(s["cache"], case["head_dim"], s["table"], s["context"], s["tails"], s["parents"])
    return {"table": table, "context": context, "cache": s["cache"].view(torch.int32)}


def run(state):
    if own:
        return _own(state)
    plain = {"prefix": _plain_prefix, "append": _plain_append, "select": _plain_select, "reorder": _plain_reorder}
    return plain[state["case"]["op"]](state)


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
    """K and V [context, D] of one sequence and head in fp64, through the sequence's own pages."""
    case = s["case"]
    d, page, group = case["head_dim"], case["page"], case["group"]
    j = torch.arange(int(s["context"][b]), device="cuda")
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


def _exact_prefix(case, seed):
    total = sum(p + (t or 0) for p, x in _branches(case) for t in x)
    if total * case["kv_heads"] * case["head_dim"] > 3e8 or sum(len(x) for _, x in _branches(case)) * case["q_heads"] > 4096:
        return None      # too long in 64 bits
    s = prepare(case, seed)
    ratio, d, n = case["q_heads"] // case["kv_heads"], case["head_dim"], case["q_len"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, tokens in enumerate(s["context"].tolist()):
        if not tokens:
            continue
        hidden = torch.arange(tokens, device="cuda")[None] > torch.arange(tokens - n, tokens, device="cuda")[:, None]
        for head in range(case["kv_heads"]):
            k, v = _sequence64(s, b, head)
            for r in range(head * ratio, (head + 1) * ratio):
                x = (s["q"][b * n:(b + 1) * n, r].double() @ k.T) / math.sqrt(d)
                x = x.masked_fill(hidden, -math.inf)
                lse[b * n:(b + 1) * n, r] = torch.logsumexp(x, -1)
                out[b * n:(b + 1) * n, r] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}


def _exact_append(case, seed):
    s = prepare(case, seed)
    angle = s["table"][s["positions"]].double()
    half, got = case["rot"] // 2, {}
    for name in ("q", "k"):
        x = s[name].double()
        if case["norm"]:
            x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * s[name + "_weight"].double()
        y = x.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            cos, sin = angle[:, None, i, 0], angle[:, None, i, 1]
            y[..., a] = x[..., a] * cos - x[..., b] * sin
            y[..., b] = x[..., b] * cos + x[..., a] * sin
        got[name] = y
    for name in ("k", "v"):
        x = (got["k"].float() if name == "k" else s["v"]).double().view(case["tokens"], case["kv_heads"], -1, case["group"])
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        low, high = torch.minimum(x.min(-1, keepdim=True).values, zero), torch.maximum(x.max(-1, keepdim=True).values, zero)
        step = ((high - low) / 15).half().double()
        zero = (-low / step).round().clamp(0, 15)
        value = ((x / step).round() + zero).clamp(0, 15).sub(zero).mul(step).reshape(s[name].shape)
        got[name] = value * (s["slots"] >= 0).double()[:, None, None]
    return got


def exact(case, seed):
    if case["op"] == "reorder":
        return None      # bytes moved, nothing computed
    if case["op"] == "prefix":
        return _exact_prefix(case, seed)
    if case["op"] == "append":
        return _exact_append(case, seed)
    s = prepare(case, seed)
    seqs, beams = s["scores"].shape
    best = torch.empty((seqs, case["k"]), dtype=torch.float64, device="cuda")
    for b in range(seqs):
        value = torch.log_softmax(s["logits"][b * beams:(b + 1) * beams].double(), -1) + s["scores"][b].double()[:, None]
        done = s["finished"][b]
        value = torch.cat((value[~done].flatten(), s["scores"][b][done].double()))
        best[b] = value.sort(descending=True).values[:case["k"]]
    return {"scores": best, "tokens": None, "parents": None}
