"""Cases of the operators that surround the quantized linear layers of a decoder.

Four operators, as they follow one another in a decoder layer with 4-bit weights
and a 4-bit key/value cache:

  linear   W4A16 matrix product with bias, activation, gate and residual in its epilogue
  pages    block table, slot map and positions of a step, from the requests' lengths
  store    keys and values quantized into the cache's pages, and read back as stored
  attend   attention over the paged 4-bit cache: single tokens, a few tokens, prompts

``own`` false: the operators in plain torch operations, in 32 bits, rounded once
at the end.  ``own`` true: the framework's calls.  ``exact`` evaluates the
definitions in 64 bits.
"""
import math
import random

import torch

own = False

GROUP = 128     # rows of a weight group
BLOCK = 16      # tokens of a cache block
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode token through the fused QKV projection of a 7B-shaped layer, with its bias
        {"name": "linear qkv bias, 1 token", "op": "linear", "tokens": 1, "k": 4096, "n": 6144, "bias": True,
         "act": "none", "gated": False, "residual": False, "scaled": False},
        # a decode batch of 16 through the gated MLP's first product of a 13B-shaped layer (gate and up interleaved)
        {"name": "linear swiglu, 16 tokens", "op": "linear", "tokens": 16, "k": 5120, "n": 27648, "bias": False,
         "act": "silu", "gated": True, "residual": False, "scaled": False},
        # an odd batch through a non-gated layer with everything in the epilogue and the channel scale in the call
        {"name": "linear gelu, 37 tokens", "op": "linear", "tokens": 37, "k": 5120, "n": 5120, "bias": True,
         "act": "gelu", "gated": False, "residual": True, "scaled": True},
        # a prompt through the down projection of a 7B-shaped layer, added to the residual stream
        {"name": "linear residual, 2048 tokens", "op": "linear", "tokens": 2048, "k": 14336, "n": 4096, "bias": False,
         "act": "none", "gated": False, "residual": True, "scaled": False},
        # one decode step of a full batch: one new token for each of 256 requests
        {"name": "pages, 256 decode tokens", "op": "pages", "requests": 256, "cached": 8191, "new": 1, "page": 16},
        # a batch of prompts admitted at once: ragged lengths from none to a few thousand tokens
        {"name": "pages, 37 prompts", "op": "pages", "requests": 37, "cached": 0, "new": 4099, "page": 64},
        # the new keys and values of a decode batch, taken out of the fused QKV rows
        {"name": "store, 64 tokens", "op": "store", "tokens": 64, "heads": 8, "dim": 128, "page": 16},
        # the keys and values of a prompt batch
        {"name": "store, 16411 tokens", "op": "store", "tokens": 16411, "heads": 8, "dim": 128, "page": 64},
        # one request early in its answer: the smallest call, latency counts (7B shape: 32 query, 8 key/value heads)
        {"name": "attend, 1 x 1037", "op": "attend", "requests": 1, "new": 1, "length": 1037, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0},
        # a serving step of a 70B-shaped layer: ragged requests up to 16 thousand tokens
        {"name": "attend, 48 x 16384", "op": "attend", "requests": 48, "new": 1, "length": 16384, "q_heads": 64,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0},
        # verification of 4 drafted tokens in long contexts with a sliding window, one head per key/value head
        {"name": "attend, 5 x 33001 window", "op": "attend", "requests": 5, "new": 4, "length": 33001, "q_heads": 16,
         "kv_heads": 16, "dim": 64, "page": 32, "window": 8192},
        # prompts with a part already cached (7B shape): the tensor-bound end
        {"name": "attend, 3 prompts of 4001", "op": "attend", "requests": 3, "new": 2900, "length": 4001, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "pages", "store", "attend", "attend", "attend"])
    if op == "linear":
        tokens = _log_int(rng, 1, 4096)
        k, n = 128 * _log_int(rng, 1, 112), 16 * _log_int(rng, 1, 1792)
        while tokens * k * n > 2048 * 14336 * 4096:
            tokens = max(1, tokens // 2)
        return {"op": op, "tokens": tokens, "k": k, "n": n, "bias": rng.random() < 0.5,
                "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), "gated": rng.random() < 0.4,
                "residual": rng.random() < 0.5, "scaled": rng.random() < 0.3}
    if op == "pages":
        return {"op": op, "requests": _log_int(rng, 1, 256), "cached": rng.choice([0, _log_int(rng, 1, 8191)]),
                "new": rng.choice([1, _log_int(rng, 2, 600)]), "page": rng.choice([16, 32, 64, 128])}
    if op == "store":
        return {"op": op, "tokens": _log_int(rng, 1, 16411), "heads": rng.choice([1, 2, 4, 8]),
                "dim": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128])}
    kv = rng.choice([1, 2, 4, 8])
    q = kv * rng.choice([1, 2, 4, 5, 7, 8])
    kind = rng.choice(["decode", "few", "prompt"])
    if kind == "decode":
        new, requests, length = 1, _log_int(rng, 1, 64), _log_int(rng, 1, 12000)
    elif kind == "few":
        new, requests, length = rng.randint(2, 8), _log_int(rng, 1, 16), _log_int(rng, 9, 16000)
    else:
        requests, length = rng.randint(1, 3), _log_int(rng, 65, 4001)
        new = max(9, int(length * rng.uniform(0.05, 1.0)))
        new = min(new, 2900, length)
        q = min(q, 32)
    return {"op": op, "requests": requests, "new": new, "length": length, "q_heads": q, "kv_heads": kv,
            "dim": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]),
            "window": rng.choice([0, 0, _log_int(rng, 1, 8192)])}


def _lengths(case):
    """(cached tokens including the new ones, new tokens) of each request: ragged, the first one the longest."""
    r = random.Random("%d/%d/%d" % (case["requests"], case["length"], case["new"]))
    lens, new = [case["length"]], [case["new"]]
    for _ in range(case["requests"] - 1):
        lens.append(max(case["new"], int(case["length"] * r.uniform(0.05, 1.0))))
        new.append(case["new"] if case["new"] <= 8 else max(1, int(case["new"] * r.uniform(0.2, 1.0))))
    return lens, new


def _page_lengths(case):
    r = random.Random("%d/%d/%d" % (case["requests"], case["cached"], case["new"]))
    old = [int(case["cached"] * r.uniform(0.0, 1.0)) for _ in range(case["requests"])]
    new = [1 if case["new"] == 1 else int(case["new"] * r.uniform(0.0, 1.0)) for _ in range(case["requests"])]
    old[0], new[0] = case["cached"], case["new"]
    return old, new


def _attended(case):
    """(cached tokens that some query reads, query-key pairs), over all requests, for one head."""
    tokens = pairs = 0
    for n, nq in zip(*_lengths(case)):
        w = case["window"] or n
        tokens += min(n, w + nq - 1)
        first = n - nq  # position of the first query
        for_all = nq * first + nq * (nq + 1) // 2
        if case["window"]:
            # positions p with p + 1 > w see w keys
            over = range(max(first, w), n)
            for_all -= sum((over[0] + 1 - w, over[-1] + 1 - w)) * len(over) // 2 if len(over) else 0
        pairs += for_all
    return tokens, pairs


def work(case):
    if case["op"] == "linear":
        m, k, n = case["tokens"], case["k"], case["n"]
        o = n // 2 if case["gated"] else n
        b = k * n // 2 + 2 * (k // GROUP) * n + (k // GROUP) * n // 2 + 2 * m * k + 2 * m * o
        b += 2 * n * case["bias"] + 2 * m * o * case["residual"] + 2 * k * case["scaled"]
        return {"bytes": b, "flops": 2 * m * k * n}
    if case["op"] == "pages":
        old, new = _page_lengths(case)
        pages = sum(-(-(a + b) // case["page"]) - -(-a // case["page"]) for a, b in zip(old, new))
        return {"bytes": 12 * sum(new) + 12 * case["requests"] + 8 * pages + 12, "flops": 0}
    if case["op"] == "store":
        t, d = case["tokens"] * case["heads"], case["dim"]
        return {"bytes": t * (4 * d + d + 8) + t * (4 * d + d + 8) + 16 * case["tokens"], "flops": 0}
    tokens, pairs = _attended(case)
    _, new = _lengths(case)
    b = tokens * case["kv_heads"] * (case["dim"] + 8) + 4 * sum(new) * case["q_heads"] * case["dim"]
    return {"bytes": b + 4 * -(-tokens // case["page"]), "flops": 4 * case["dim"] * case["q_heads"] * pairs}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _quantized_weight(g, k, n):
    """W ~ N(0, 0.02^2) on the 4-bit grid of its groups of 128 rows: packed words, steps, packed zero points."""
    w = _normal(g, k // GROUP, GROUP, n).mul_(0.02)
    lo, hi = w.amin(1), w.amax(1)
    step = ((hi - lo) / 15).half()
    zero = torch.clamp(torch.round(-lo / step.float()), 0, 15)
    q = torch.clamp(torch.round(w / step.float()[:, None]) + zero[:, None], 0, 15).to(torch.int32).reshape(k // 8, 8, n)
    packed = torch.zeros(k // 8, n, dtype=torch.int32, device=DEV)
    zeros = torch.zeros(k // GROUP, n // 8, dtype=torch.int32, device=DEV)
    zi = zero.to(torch.int32).reshape(k // GROUP, n // 8, 8)
    for j in range(8):
        packed |= q[:, j] << (4 * j)
        zeros |= zi[:, :, j] << (4 * j)
    return packed, step, zeros


def _pack_cache(k, v, dim):
    """Cache blocks of 16 tokens [..., 16, dim] -> [..., 16 dim + 128] bytes: codes of k, codes of v, then a word per
    token and tensor with the step (low half, float16) and the zero point (high half)."""
    parts, metas = [], []
    for x in (k, v):
        q, step, zero = _grid(x)
        q = q.to(torch.uint8)
        parts.append((q[..., 0::2] | (q[..., 1::2] << 4)).flatten(-2))
        meta = torch.zeros(*step.shape, 4, dtype=torch.uint8, device=DEV)
        meta[..., :2] = step.contiguous().view(torch.uint8).reshape(*step.shape, 2)
        meta[..., 2] = zero.to(torch.uint8)
        metas.append(meta.flatten(-2))
    return torch.cat(parts + metas, -1)


def _grid(x):
    """Codes, step (float16) and zero point of x's 4-bit grid over its last dimension; the grid contains zero."""
    x = x.float()
    lo, hi = x.amin(-1).clamp_max(0), x.amax(-1).clamp_min(0)
    step = ((hi - lo).clamp_min(1e-5) / 15).half()
    s = step.float()
    zero = torch.round(-lo / s).clamp(0, 15)
    q = (torch.round(x * (1 / s)[..., None]) + zero[..., None]).clamp(0, 15)
    return q, step, zero


def _key_values(g, *shape):
    """Keys with a few outlier channels, and values, as float16."""
    k = _normal(g, *shape)
    k[..., ::37] *= 4
    return k.half(), _normal(g, *shape).half()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "linear":
        m, k, n = case["tokens"], case["k"], case["n"]
        s["Q"], s["scales"], s["zeros"] = _quantized_weight(g, k, n)
        x = _normal(g, m, k)
        x[:, torch.randperm(k, generator=g, device=DEV)[: -(-k // 100)]] *= 20   # 1% outlier channels
        s["x"] = x.half()
        s["s"] = torch.exp(_normal(g, k) * 0.3).half() if case["scaled"] else None
        s["b"] = _normal(g, n).half() if case["bias"] else None
        s["r"] = _normal(g, m, n // 2 if case["gated"] else n).half() if case["residual"] else None
        if own:
            import weight_only_quantization_quantize_b200 as awq
            s["layer"] = awq.QuantLinear(s["Q"], s["scales"], s["zeros"], s["s"], bias=s["b"], act=case["act"],
                                         gated=case["gated"])
        return s
    page = case["page"]
    if case["op"] == "pages":
        old, new = _page_lengths(case)
        held = [-(-a // page) for a in old]
        most = max(-(-(a + b) // page) for a, b in zip(old, new)) + 1
        total = sum(held) + sum(-(-(a + b) // page) for a, b in zip(old, new)) + 7
        order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = torch.full((len(old), most), -1, dtype=torch.int32, device=DEV)
        place = torch.arange(most, device=DEV)[None] < torch.tensor(held, device=DEV)[:, None]
        table[place] = order[: sum(held)]
        s["table"], s["free"] = table, torch.cat([order[sum(held):], order.new_full((sum(held),), -1)])
        s["free_count"] = torch.tensor([total - sum(held)], dtype=torch.int32, device=DEV)
        s["old"] = torch.tensor(old, dtype=torch.int32, device=DEV)
        s["new_lens"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        s["total"] = sum(new) + 3   # rows of the step, the last ones padding
        s["next"], s["next_free"] = torch.empty_like(s["old"]), torch.empty_like(s["free_count"])
        if own:
            import weight_only_quantization_quantize_b200 as awq
            s["pages"] = awq.KV4Pages(total, page, len(old), most, block_table=s["table"], lens=s["old"],
                                      free_pages=s["free"], free_count=s["free_count"])
        return s
    heads, dim = case.get("heads", case.get("kv_heads")), case["dim"]
    size = page // BLOCK * (BLOCK * dim + 128)   # bytes of a page, for one head
    if case["op"] == "store":
        t = case["tokens"]
        count = -(-t // page) + 3
        k, v = _key_values(g, t, heads, dim)
        row = torch.randn(t, 4 * heads * dim, generator=g, device=DEV).half()   # a fused projection's rows
        row[:, 2 * heads * dim: 3 * heads * dim], row[:, 3 * heads * dim:] = k.flatten(1), v.flatten(1)
        s["k"] = row[:, 2 * heads * dim: 3 * heads * dim].unflatten(1, (heads, dim))
        s["v"] = row[:, 3 * heads * dim:].unflatten(1, (heads, dim))
        order = torch.randperm(count, generator=g, device=DEV)
        at = torch.arange(t, device=DEV)
        s["slots"] = order[at // page] * page + at % page
        if t > 1:
            s["slots"][t // 2] = -1   # a padded row, stored nowhere
        s["cache"] = torch.zeros(count, heads, size, dtype=torch.uint8, device=DEV)
        if own:
            import weight_only_quantization_quantize_b200 as awq
            s["layer"] = awq.KV4Cache(awq.KV4Pages(count, page, 1, count), heads, dim, data=s["cache"])
        return s
    lens, new = _lengths(case)
    held = [-(-n // page) for n in lens]
    order = torch.randperm(sum(held) + 5, generator=g, device=DEV).to(torch.int32)
    s["cache"] = torch.empty(len(order), heads, size, dtype=torch.uint8, device=DEV)
    for at in range(0, len(order), 4096):
        part = s["cache"][at: at + 4096]
        k, v = _key_values(g, len(part), heads, page // BLOCK, BLOCK, dim)
        part.copy_(_pack_cache(k, v, dim).flatten(2))
    s["table"] = torch.full((len(lens), max(held)), -1, dtype=torch.int32, device=DEV)
    place = torch.arange(max(held), device=DEV)[None] < torch.tensor(held, device=DEV)[:, None]
    s["table"][place] = order[: sum(held)]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["cu"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    s["q"] = _normal(g, sum(new), case["q_heads"], dim).half()
    s["most"] = max(new)
    if own:
        import weight_only_quantization_quantize_b200 as awq
        pages = awq.KV4Pages(len(order), page, len(lens), max(held), block_table=s["table"], lens=s["lens"])
        s["layer"] = awq.KV4Cache(pages, heads, dim, data=s["cache"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        if s["op"] == "linear":
            return s["layer"](s["x"], residual=s["r"])
        if s["op"] == "pages":
            slots, positions, cu = s["pages"].reserve(s["new_lens"], s["total"], next_lens=s["next"],
                                                      next_free=s["next_free"])
            return {"slots": slots, "positions": positions, "cu": cu, "lens": s["next"], "free": s["next_free"],
                    "table": s["table"]}
        if s["op"] == "store":
            s["layer"].append(s["k"], s["v"], s["slots"])
            return s["layer"].load(s["slots"])
        return s["layer"].attention(s["q"], cu=s["cu"], max_new=s["most"], window=s["window"])
    return {"linear": _linear, "pages": _pages, "store": _store, "attend": _attend}[s["op"]](s)


def _act(t, act):
    if act == "relu":
        return t.clamp_min(0)
    if act == "silu":
        return t / (1 + torch.exp(-t))
    if act == "gelu":
        return 0.5 * t * (1 + torch.erf(t * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t * t * t)))
    return t


def _linear(s):
    k, n = s["k"], s["n"]
    at = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    q = ((s["Q"][:, None] >> at[:, None]) & 15).reshape(k // GROUP, GROUP, n)
    z = ((s["zeros"][:, :, None] >> at) & 15).reshape(k // GROUP, 1, n)
    w = ((q - z).float() * s["scales"].float()[:, None]).reshape(k, n)
    x = s["x"].float()
    if s["s"] is not None:
        x = (x / s["s"].float()).half().float()   # X / s is a float16 operand of the product
    t = x @ w
    if s["b"] is not None:
        t = t + s["b"].float()
    t = _act(t[:, 0::2], s["act"]) * t[:, 1::2] if s["gated"] else _act(t, s["act"])
    if s["r"] is not None:
        t = t + s["r"].float()
    return t.half()


def _pages(s):
    page, old, new = s["page"], s["old"], s["new_lens"]
    cu = torch.zeros(len(old) + 1, dtype=torch.int32, device=DEV)
    cu[1:] = new.cumsum(0)
    held = (old + page - 1) // page
    need = (old + new + page - 1) // page - held
    first = need.cumsum(0) - need
    col = torch.arange(s["table"].shape[1], device=DEV)[None]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    pick = s["free_count"] - 1 - (first[:, None] + col - held[:, None])
    table = torch.where(fresh, s["free"][torch.where(fresh, pick, 0)], s["table"])
    row = torch.arange(s["total"], device=DEV)
    b = (row[:, None] >= cu[None, 1:]).sum(1)
    real = b < len(old)
    b = b.clamp_max(len(old) - 1)
    position = torch.where(real, old[b] + row - cu[b], -1).to(torch.int32)
    at = position.clamp_min(0)
    slots = torch.where(real, table[b, at // page].long() * page + at % page, -1)
    return {"slots": slots, "positions": position, "cu": cu, "lens": old + new,
            "free": s["free_count"] - need.sum().to(torch.int32), "table": table}


def _unpack(block, dim):
    """Keys and values of cache blocks [..., 16 dim + 128] as float32 [..., 16, dim]."""
    half = BLOCK * dim // 2
    out = []
    for i in range(2):   # keys, values
        b = block[..., i * half: (i + 1) * half].unflatten(-1, (BLOCK, dim // 2))
        meta = block[..., 2 * half + 64 * i: 2 * half + 64 * (i + 1)].unflatten(-1, (BLOCK, 4))
        step = meta[..., :2].contiguous().view(torch.float16).float()
        q = torch.stack([b & 15, b >> 4], -1).flatten(-2)
        out.append((q.float() - meta[..., 2:3].float()) * step)
    return out


def _store(s):
    dim, page, slots = s["dim"], s["page"], s["slots"]
    heads, half = s["heads"], BLOCK * dim // 2
    real = slots >= 0
    at = slots[real]
    blocks = s["cache"].view(-1, heads, page // BLOCK, BLOCK * dim + 128)
    p, j, i = at // page, at % page // BLOCK, at % BLOCK
    head = torch.arange(heads, device=DEV)
    values = []
    for n, x in enumerate((s["k"], s["v"])):
        q, step, zero = _grid(x[real])
        q = q.to(torch.uint8)
        meta = torch.cat([step.view(torch.uint8).unflatten(-1, (heads, 2)), zero.to(torch.uint8)[..., None],
                          torch.zeros_like(zero, dtype=torch.uint8)[..., None]], -1)
        codes = blocks[..., n * half: (n + 1) * half].unflatten(-1, (BLOCK, dim // 2))
        metas = blocks[..., 2 * half + 64 * n: 2 * half + 64 * (n + 1)].unflatten(-1, (BLOCK, 4))
        codes[p[:, None], head, j[:, None], i[:, None]] = q[..., 0::2] | (q[..., 1::2] << 4)
        metas[p[:, None], head, j[:, None], i[:, None]] = meta
        b, m = codes[p, :, j, i], metas[p, :, j, i]
        got = torch.stack([b & 15, b >> 4], -1).flatten(-2).float() - m[..., 2:3].float()
        out = torch.zeros(len(slots), heads, dim, dtype=torch.float16, device=DEV)
        out[real] = (got * m[..., :2].contiguous().view(torch.float16).float()).half()
        values.append(out)
    return tuple(values)


def _attend(s):
    page, dim, hk = s["page"], s["dim"], s["kv_heads"]
    group, most = s["q_heads"] // hk, s["most"]
    lens, cu = s["lens"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    blocks = s["cache"].view(len(s["cache"]), hk, page // BLOCK, BLOCK * dim + 128)[s["table"].clamp_min(0).long()]
    k, v = _unpack(blocks, dim)                                         # [requests, pages, heads, blocks, 16, dim]
    k = k.transpose(1, 2).flatten(2, 4)                                 # [requests, heads, tokens, dim]
    v = v.transpose(1, 2).flatten(2, 4)
    i = torch.arange(most, device=DEV)
    real = i < new[:, None]
    row = torch.where(real, cu[:-1, None] + i, 0)
    q = s["q"].float()[row].unflatten(2, (hk, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [requests, heads, group x new, dim]
    pos = ((lens - new)[:, None] + i)[:, None, None, :, None]
    j = torch.arange(k.shape[2], device=DEV)
    seen = j <= pos
    if s["window"]:
        seen &= j > pos - s["window"]
    t = (q @ k.transpose(2, 3)).mul_(dim ** -0.5).unflatten(2, (group, most))
    t.masked_fill_(~seen, -math.inf)
    top = t.amax(-1, keepdim=True).clamp_min(-1e30)
    e = t.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e.flatten(2, 3) @ v).unflatten(2, (group, most)) / torch.where(total > 0, total, 1)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                          # [requests, new, heads, dim]
    out = torch.zeros(s["q"].shape, dtype=torch.float16, device=DEV)
    out[row[real]] = o[real].half()
    return out


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return None   # whole numbers only
    if case["op"] == "linear":
        k, n = case["k"], case["n"]
        w = torch.empty(k, n, dtype=torch.float64, device=DEV)
        for j in range(8):   # row 8 i + j sits in bits 4 j .. 4 j + 3 of word i
            w[j::8] = s["Q"] >> (4 * j) & 15
        zero = torch.stack([s["zeros"] >> (4 * j) & 15 for j in range(8)], -1).flatten(1).double()
        for g in range(k // GROUP):
            w[g * GROUP: (g + 1) * GROUP].sub_(zero[g]).mul_(s["scales"][g].double())
        x = s["x"].double()
        if s["s"] is not None:
            x = (x / s["s"].double()).half().double()
        t = x.matmul(w)
        if s["b"] is not None:
            t += s["b"].double()
        gate = t[:, ::2] if case["gated"] else t
        a = {"none": lambda u: u, "relu": lambda u: u.clamp(min=0), "silu": lambda u: u * torch.sigmoid(u),
             "gelu": lambda u: u * 0.5 * torch.erfc(-u / math.sqrt(2)),
             "gelu_tanh": lambda u: u * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3))}[case["act"]](gate)
        if case["gated"]:
            a = a * t[:, 1::2]
        return a if s["r"] is None else a + s["r"].double()
    if case["op"] == "store":
        out = []
        for x in (s["k"].double(), s["v"].double()):
            x = torch.where((s["slots"] >= 0)[:, None, None], x, 0.0)
            lo, hi = x.min(2, keepdim=True).values.clamp(max=0), x.max(2, keepdim=True).values.clamp(min=0)
            step = ((hi - lo).clamp(min=1e-5) / 15).half().double()
            zero = (-lo / step).round().clamp(0, 15)
            out.append((((x / step).round() + zero).clamp(0, 15) - zero) * step)
        return tuple(out)
    dim, page, hk = case["dim"], case["page"], case["kv_heads"]
    lens, new = _lengths(case)
    group, at = case["q_heads"] // hk, 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    if sum(n * m for n, m in zip(lens, new)) * case["q_heads"] * dim > 4e12:
        return None
    for b, (n, m) in enumerate(zip(lens, new)):
        rec = s["cache"][s["table"][b, : -(-n // page)].long()].transpose(0, 1).reshape(hk, -1, BLOCK * dim + 128)
        words = rec[..., : BLOCK * dim].reshape(hk, -1, 2, BLOCK, dim // 2)
        q4 = torch.empty(*words.shape[:-1], dim, dtype=torch.float64, device=DEV)
        q4[..., ::2], q4[..., 1::2] = words % 16, words // 16
        tail = rec[..., BLOCK * dim:].contiguous().view(torch.float16).reshape(hk, -1, 2, BLOCK, 2)
        zero = tail[..., 1].contiguous().view(torch.int16).double()
        x = (q4 - zero[..., None]) * tail[..., :1].double()
        k, v = (x[:, :, i].reshape(hk, -1, dim)[:, :n] for i in (0, 1))
        pos = torch.arange(n - m, n, device=DEV)[:, None]
        key = torch.arange(n, device=DEV)[None]
        hidden = (key > pos) | (key <= pos - (case["window"] or n + 1))
        for h in range(hk):
            q = s["q"][at: at + m, h * group: (h + 1) * group].double().transpose(0, 1)
            p = torch.softmax((q @ k[h].T / math.sqrt(dim)).masked_fill(hidden, -math.inf), -1)
            out[at: at + m, h * group: (h + 1) * group] = (p @ v[h]).transpose(0, 1)
        at += m
    return out
