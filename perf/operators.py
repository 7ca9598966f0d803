"""Measured cases of the 4-bit KV cache operators: block tables and slot maps built from
request lengths, the append that quantizes new keys and values into the paged cache (with the
read that gives the stored values back), and attention over the cache for single tokens,
drafts and prompts.

`run` computes each operator in a plain form (elementary torch operations), or, with `own`
set, calls the framework. The cache's byte layout is the framework's: block `n`, head `h` is
one chunk [K codes | V codes | K scales | V scales] of `block` tokens. A token's 4-bit codes
are packed two per byte in the order of its dimensions; the 32-bit words of a K row and the
bytes of a V row are then transposed into the order in which the tensor-core fragments take
them, and the two halves of a 64-byte V row change places on tokens 2 and 3 of every four.
A scale word holds S and Z of one group as two binary16 values.
"""
import math
import random

import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------- cases

def listed():
    """Head layouts: 32 heads of 128 and 64 query heads over 8 KV heads of 128, as in the 7B-
    and 70B-class layers (4096 and 8192 wide) of the matmul benchmark; 2048 prompt tokens as in
    its prefill; the others are generic."""
    att = {"kind": "attend", "window": 0, "causal": True}
    return [
        # one decode step's bookkeeping: every request of a batch gets one more token
        {"name": "tables_step", "kind": "tables", "requests": 256, "budget": 256, "ctx": 8192, "block": 64},
        # admission of many prompts at once, most blocks newly taken, a padded token budget
        {"name": "tables_prompts", "kind": "tables", "requests": 700, "budget": 131072, "ctx": 1500, "block": 16},
        # the keys and values of one decode step
        {"name": "append_step", "kind": "append", "tokens": 64, "padded": 0, "kv_heads": 8, "dim": 128, "group": 128, "block": 64, "dtype": "bf16", "fused": False},
        # a long prompt's keys and values, as slices of a fused projection's output, padded rows behind
        {"name": "append_prompt", "kind": "append", "tokens": 16384, "padded": 111, "kv_heads": 8, "dim": 128, "group": 128, "block": 64, "dtype": "bf16", "fused": True},
        # small heads with fine groups
        {"name": "append_fine_groups", "kind": "append", "tokens": 4099, "padded": 0, "kv_heads": 6, "dim": 64, "group": 32, "block": 16, "dtype": "fp16", "fused": False},
        # one user's next token after a short chat: latency
        {"name": "decode_one_short", **att, "requests": 1, "new": 1, "ctx": 997, "ragged": False, "heads": 32, "kv_heads": 32, "dim": 128, "group": 128, "block": 64, "dtype": "bf16"},
        # one user's next token in a very long document: the long axis has to be split
        {"name": "decode_one_long", **att, "requests": 1, "new": 1, "ctx": 131071, "ragged": False, "heads": 64, "kv_heads": 8, "dim": 128, "group": 128, "block": 64, "dtype": "bf16"},
        # a serving batch of requests of all lengths, one of its places empty
        {"name": "decode_batch", **att, "requests": 64, "new": 1, "ctx": 8192, "ragged": True, "heads": 64, "kv_heads": 8, "dim": 128, "group": 128, "block": 16, "dtype": "bf16"},
        # drafted tokens to be verified: three queries a request, small heads, fine groups
        {"name": "decode_drafts", **att, "requests": 48, "new": 3, "ctx": 3001, "ragged": True, "heads": 24, "kv_heads": 6, "dim": 64, "group": 32, "block": 32, "dtype": "fp16"},
        # a fresh prompt of a 7B-class layer
        {"name": "prompt_2048", **att, "requests": 1, "new": 2048, "ctx": 0, "ragged": False, "heads": 32, "kv_heads": 32, "dim": 128, "group": 128, "block": 64, "dtype": "bf16"},
        # a chunk of a long prompt of a 70B-class layer, after what is cached already
        {"name": "prompt_chunk", **att, "requests": 1, "new": 1024, "ctx": 15360, "ragged": False, "heads": 64, "kv_heads": 8, "dim": 128, "group": 128, "block": 64, "dtype": "bf16"},
        # several prompts of odd lengths at once, an odd number of heads to a KV head, two groups a head
        {"name": "prompts_ragged", **att, "requests": 7, "new": 1111, "ctx": 900, "ragged": True, "heads": 28, "kv_heads": 4, "dim": 128, "group": 64, "block": 32, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tables", "append", "append", "decode", "decode", "decode", "prompt", "prompt", "prompt"])
    block = rng.choice([16, 32, 64, 128])
    if kind == "tables":
        n = _log(rng, 1, 1024)
        return {"kind": kind, "requests": n, "budget": _log(rng, n, 131072), "ctx": _log(rng, 1, 8192), "block": block}
    dim = rng.choice([64, 128, 128])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim] + [dim, dim])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if kind == "append":
        return {"kind": kind, "tokens": _log(rng, 1, 16384), "padded": rng.choice([0, 0, 1, 77]), "kv_heads": rng.choice([1, 2, 4, 5, 8]), "dim": dim, "group": group,
                "block": block, "dtype": dtype, "fused": rng.random() < 0.5}
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    ratio = rng.choice([1, 2, 3, 4, 4, 7, 8, 8, 16])
    base = {"kind": "attend", "ragged": rng.random() < 0.6, "heads": kv_heads * ratio, "kv_heads": kv_heads, "dim": dim, "group": group, "block": block, "dtype": dtype}
    if kind == "decode":
        n = _log(rng, 1, 128)
        ctx = _log(rng, 1, max(2, min(131072, (1 << 22) // (n * kv_heads))))
        return {**base, "requests": n, "new": rng.choice([1, 1, 1, 2, 4, 5]), "ctx": ctx, "window": rng.choice([0, 0, 0, 100, 1024]), "causal": True}
    n = _log(rng, 1, 8)
    new = _log(rng, 16, 2048 // n)
    ctx = _log(rng, 1, max(2, min(16384, (1 << 30) // (n * new * base["heads"]))))
    return {**base, "requests": n, "new": new, "ctx": ctx, "window": rng.choice([0, 0, 0, 500]), "causal": rng.random() < 0.8}


def _spread(n, most, ragged):
    """n lengths up to `most`: all of them `most`, or spread evenly below it, the first one 0."""
    if not ragged or n == 1:
        return [most] * n
    return [0] + [max(1, most * i // (n - 1)) for i in range(1, n)]


def _lengths(case):
    """(tokens in the cache with this call's, this call's) of each request: the same ones for
    every seed, which only orders them."""
    n = case["requests"]
    if case["kind"] == "tables":
        share = case["budget"] // n
        new = [1] * n if share <= 1 else [max(1, share * (1 + i * 7 % 16) // 17) for i in range(n)]
        return [(c + k, k) for c, k in zip(_spread(n, case["ctx"], True), new)]
    if case["new"] <= 8:  # decode: the same number of queries each; a padded place holds nothing
        return [(kv, case["new"]) for kv in _spread(n, case["ctx"] + case["new"], case["ragged"])]
    new = _spread(n, case["new"], case["ragged"])
    return [(c + k, k) for c, k in zip(_spread(n, case["ctx"], case["ragged"])[::-1], new)]


def _attended(case):
    """Number of (query, key) pairs of one head."""
    total, w = 0, case["window"]
    for kv, new in _lengths(case):
        for i in range(new):
            last = kv - new + i if case["causal"] else kv - 1
            if last >= 0:
                total += min(last + 1, w) if w else last + 1
    return total


def _row_bytes(case):
    return case["dim"] // 2 + 4 * (case["dim"] // case["group"])  # one token of one head, K or V


def work(case):
    if case["kind"] == "tables":
        lens = _lengths(case)
        b = case["block"]
        taken = sum(-(-kv // b) - -(-(kv - n) // b) for kv, n in lens)
        return {"bytes": 4 * (2 * len(lens) + 2 * taken + 2 * case["budget"] + 2 * len(lens)), "flops": 0}
    if case["kind"] == "append":
        n = case["tokens"] * case["kv_heads"] * case["dim"] * 2
        rows = case["tokens"] * case["kv_heads"] * 2
        padded = case["padded"] * case["kv_heads"] * case["dim"] * 2 * 4
        # read the inputs, write the stored rows, read them back, write their values
        return {"bytes": 2 * n + 2 * rows * _row_bytes(case) + 4 * n + padded, "flops": 6 * n}
    lens = _lengths(case)
    queries = sum(n for _, n in lens)
    w = case["window"]
    cached = sum(min(kv, w + n - 1 if case["causal"] else w) if w else kv for kv, n in lens)
    return {"bytes": cached * case["kv_heads"] * 2 * _row_bytes(case) + queries * case["heads"] * (4 * case["dim"] + 4),
            "flops": 4 * _attended(case) * case["heads"] * case["dim"]}


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pack_rows(codes, key):
    """Codes [..., block, dim] -> bytes [..., block, dim / 2] in the cache's order."""
    block, dim = codes.shape[-2:]
    b = codes[..., 0::2] | codes[..., 1::2] << 4
    if key:  # words 4 j + c -> place c * (dim / 32) + j
        b = b.unflatten(-1, (dim // 32, 4, 4)).transpose(-3, -2)
        return b.reshape(*codes.shape[:-1], dim // 2)
    b = b.unflatten(-1, (dim // 16, 8)).transpose(-2, -1).reshape(*codes.shape[:-1], dim // 2)
    if dim == 128:
        b = b.unflatten(-2, (block // 4, 4)).clone()
        b[..., 2:, :] = b[..., 2:, :].roll(32, -1)
        b = b.flatten(-3, -2)
    return b


def _quantize_quick(x, group):
    """Codes and S, Z of x [..., dim] for the making of a cache (any valid ones do)."""
    x = x.unflatten(-1, (-1, group))
    lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    s = ((hi - lo) / 15).half().float().clamp(min=2.0**-14)
    z = (-lo / s).round().clamp(0, 15)
    q = ((x / s[..., None]).round() + z[..., None]).clamp(0, 15).to(torch.uint8)
    return q.flatten(-2), torch.stack((s, z), -1).half()


def _make_cache(case, blocks, seed):
    """A cache filled with quantized keys and values: keys with some strong channels, values
    whose size differs from token to token."""
    g = _gen(seed)
    shape = (blocks, case["kv_heads"], case["block"], case["dim"])
    parts = []
    for key in (True, False):
        x = torch.randn(shape, generator=g, device=DEV)
        if key:
            x *= 1 + 3 * (torch.rand(case["kv_heads"], 1, case["dim"], generator=g, device=DEV) < 0.04)
        else:
            x *= 0.5 + torch.rand(*shape[:3], 1, generator=g, device=DEV)
        q, sz = _quantize_quick(x, case["group"])
        del x
        parts.append((_pack_rows(q, key).flatten(-2), sz.flatten(-3).contiguous().view(torch.uint8)))
    return torch.cat((parts[0][0], parts[1][0], parts[0][1], parts[1][1]), -1).contiguous()


def prepare(case, seed):
    rng = random.Random(seed)
    g = _gen(seed)
    block = case["block"]
    if case["kind"] == "append":
        t, p, h, d = case["tokens"], case["padded"], case["kv_heads"], case["dim"]
        wide = 3 * h * d if case["fused"] else 2 * h * d  # queries beside them in a fused projection
        x = torch.randn(t + p, wide, generator=g, device=DEV)
        x[:, -2 * h * d: -h * d] *= 1 + 3 * (torch.rand(h * d, generator=g, device=DEV) < 0.04)
        x = x.to(DTYPES[case["dtype"]])
        k, v = x[:, -2 * h * d: -h * d].unflatten(-1, (h, d)), x[:, -h * d:].unflatten(-1, (h, d))
        if not case["fused"]:
            k, v = k.contiguous(), v.contiguous()
        blocks = -(-(t + p) // block) + 3
        order = torch.randperm(blocks, generator=g, device=DEV)
        at = torch.arange(t + p, device=DEV) + rng.randrange(2 * block)
        slots = order[at // block] * block + at % block
        slots[t:] = -1
        chunk = 2 * block * _row_bytes(case)
        return {"case": case, "k": k, "v": v, "slots": slots.int(), "cache": torch.zeros(blocks, h, chunk, dtype=torch.uint8, device=DEV)}
    lens = _lengths(case)
    rng.shuffle(lens)
    kv, new = [k for k, _ in lens], [n for _, n in lens]
    need = [-(-n // block) for n in kv]
    if case["kind"] == "tables":
        ctx = [k - n for k, n in lens]
        held = [-(-c // block) for c in ctx]
        pool = torch.randperm(sum(need) + 5, generator=g, device=DEV).int()
        table = torch.full((len(lens), max(need) + 2), -1, dtype=torch.int32)
        host, at = pool.tolist(), 0
        for i, n in enumerate(held):
            table[i, :n] = torch.tensor(host[at: at + n], dtype=torch.int32)
            at += n
        return {"case": case, "ctx_lens": _ints(ctx), "new_lens": _ints(new), "tables": table.to(DEV), "free": pool[at:].clone()}
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    host, at = torch.randperm(sum(need) + 2, generator=g, device=DEV).tolist(), 0
    for i, n in enumerate(need):
        table[i, :n] = torch.tensor(host[at: at + n], dtype=torch.int32)
        at += n
    starts = [sum(new[:i]) for i in range(len(new) + 1)]
    q = torch.randn(starts[-1], case["heads"], case["dim"], generator=g, device=DEV).to(DTYPES[case["dtype"]])
    return {"case": case, "q": q, "cache": _make_cache(case, sum(need) + 2, seed), "tables": table.to(DEV), "q_starts": _ints(starts), "kv_lens": _ints(kv),
            "max_q": max(new), "max_kv": max(kv + [1])}


# ------------------------------------------------------------------------- plain forms

def _to_half(x):
    """float64 x >= 0 rounded once to binary16 (half to even), as float64."""
    step = torch.exp2(torch.frexp(x).exponent.clamp(min=-13).double() - 11)
    return torch.round(x / step) * step


def _stored(x, group):
    """The values S' (q - Z) that a row is stored as: range with zero, S' the binary16 rounding
    of a fifteenth of it, codes half to even on the exact quotient. Roundings next to a border
    need 64 bits."""
    w = x.double().unflatten(-1, (-1, group))
    lo, hi = w.amin(-1, keepdim=True).clamp(max=0), w.amax(-1, keepdim=True).clamp(min=0)
    s = _to_half((hi - lo) / 15)
    s = torch.where(s == 0, 1.0, s)
    z = torch.round(-lo / s).clamp(0, 15)
    q = (torch.round(w / s) + z).clamp(0, 15)
    return (s * (q - z)).flatten(-2).float()


def _plain_tables(st):
    block, budget = st["case"]["block"], st["case"]["budget"]
    ctx, new, free = st["ctx_lens"].long(), st["new_lens"].long(), st["free"]
    kv = ctx + new
    held, need = (ctx + block - 1) // block, (kv + block - 1) // block
    starts = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    ends = (need - held).cumsum(0)
    place = torch.arange(st["tables"].shape[1], device=DEV)
    fresh = (place >= held[:, None]) & (place < need[:, None])
    which = (ends - need)[:, None] + place  # the request's first free block, less what it holds
    tables = torch.where(fresh, free[which.clamp(0, free.numel() - 1)], st["tables"])
    token = torch.arange(budget, device=DEV)
    row = torch.searchsorted(starts[1:], token, right=True)
    live = row < len(ctx)
    row = row.clamp(max=len(ctx) - 1)
    pos = ctx[row] + token - starts[row]
    block_of = tables[row, (pos // block).clamp(0, tables.shape[1] - 1)]
    slots = torch.where(live, block_of * block + pos % block, -1)
    return {"tables": tables, "slots": slots.int(), "q_starts": starts.int(), "kv_lens": kv.int(), "taken": ends[-1:].int()}


def _codes(b, key):
    """Bytes [..., block, dim / 2] in the cache's order -> codes [..., block, dim]."""
    block, dim = b.shape[-2], 2 * b.shape[-1]
    if key:
        b = b.unflatten(-1, (4, dim // 32, 4)).transpose(-3, -2).flatten(-3)
    else:
        if dim == 128:
            turned = (torch.arange(block, device=b.device) & 2).bool()[:, None]
            b = torch.where(turned, b.roll(32, -1), b)
        b = b.unflatten(-1, (8, dim // 16)).transpose(-2, -1).flatten(-2)
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _values(chunks, case):
    """Chunks [..., bytes] -> keys and values [..., block, dim] in 32 bits (exact)."""
    block, dim, groups = case["block"], case["dim"], case["dim"] // case["group"]
    n = block * dim // 2
    parts = chunks.split([n, n, 4 * block * groups, 4 * block * groups], -1)

    def one(b, sz, key):
        q = _codes(b.unflatten(-1, (block, dim // 2)), key).unflatten(-1, (groups, -1)).float()
        sz = sz.contiguous().view(torch.float16).float().unflatten(-1, (block, groups, 2))
        return (sz[..., :1] * (q - sz[..., 1:])).flatten(-2)

    return one(parts[0], parts[2], True), one(parts[1], parts[3], False)


def _plain_attend(st):
    case = st["case"]
    tables, starts, kv_lens = st["tables"].long().clamp(min=0), st["q_starts"].long(), st["kv_lens"].long()
    q, n, h, ratio = st["q"], len(kv_lens), case["kv_heads"], case["heads"] // case["kv_heads"]
    k, v = _values(st["cache"][tables], case)  # [n, blocks, h, block, dim]
    k, v = (x.transpose(1, 2).flatten(2, 3)[:, :, : st["max_kv"]] for x in (k, v))
    lens = starts[1:] - starts[:-1]
    i = torch.arange(st["max_q"], device=DEV)
    source = (starts[:-1, None] + i).clamp(max=max(0, q.shape[0] - 1))
    x = q.float()[source].unflatten(2, (h, ratio)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [n, h, ratio * max_q, dim]
    s = x @ k.transpose(-1, -2) * (case["dim"] ** -0.5)
    j = torch.arange(k.shape[2], device=DEV)
    last = (kv_lens - lens)[:, None] + i if case["causal"] else (kv_lens - 1)[:, None].expand(-1, st["max_q"])
    seen = (j <= last[..., None]) & (j < kv_lens[:, None, None])
    if case["window"]:
        seen &= j > last[..., None] - case["window"]
    s = s.unflatten(2, (ratio, -1)).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.clamp(min=torch.finfo(torch.float32).min))
    del s
    total = p.sum(-1, keepdim=True)
    o = p.flatten(2, 3) @ v
    o = o.unflatten(2, (ratio, -1)) / total.clamp(min=torch.finfo(torch.float32).tiny)
    lse = (m + total.log())[..., 0]
    token = torch.arange(q.shape[0], device=DEV)
    row = torch.searchsorted(starts[1:], token, right=True)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[row, token - starts[row]]
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)[row, token - starts[row]]
    return {"out": o.to(q.dtype), "lse": lse}


# ----------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if case["kind"] == "tables":
        if own:
            import w4a16_dequant_matmul_b200 as wq

            slots, starts, kv_lens, taken = wq.wq_kv4_block_tables(state["ctx_lens"], state["new_lens"], state["free"], state["tables"], case["block"], case["budget"])
            return {"tables": state["tables"], "slots": slots, "q_starts": starts, "kv_lens": kv_lens, "taken": taken}
        return _plain_tables(state)
    if case["kind"] == "append":
        if own:
            import w4a16_dequant_matmul_b200 as wq

            wq.wq_kv4_append(state["k"], state["v"], state["slots"], state["cache"], group=case["group"])
            k, v = wq.wq_kv4_read(state["cache"], state["slots"], case["dim"], group=case["group"])
            return {"k": k, "v": v}
        live = (state["slots"] >= 0)[:, None, None]
        return {"k": torch.where(live, _stored(state["k"], case["group"]), 0), "v": torch.where(live, _stored(state["v"], case["group"]), 0)}
    if own:
        import w4a16_dequant_matmul_b200 as wq

        out, lse = wq.wq_kv4_attention(state["q"], state["cache"], state["tables"], state["q_starts"], state["kv_lens"], state["max_q"], group=case["group"],
                                       causal=case["causal"], window=case["window"], return_lse=True)
        return {"out": out, "lse": lse}
    return _plain_attend(state)


# -------------------------------------------------------------------------------- exact

def _exact_rows(raw, dim, groups, block, n, h, t, key):
    """Rows t of block n, head h of the cache `raw`, by the layout's definition, in 64 bits."""
    half = block * dim // 2
    place = torch.empty(dim // 2, dtype=torch.long)  # where byte b of the natural order is stored
    for b in range(dim // 2):
        word, inside = divmod(b, 4)
        place[b] = ((word % 4) * (dim // 32) + word // 4) * 4 + inside if key else (b % 8) * (dim // 16) + b // 8
    place = place.to(raw.device)[None, :].expand(len(t), -1)
    if not key and dim == 128:
        place = place ^ (32 * (t // 2 % 2))[:, None]
    base = (0 if key else half) + t[:, None] * (dim // 2)
    b = raw[n[:, None], h, base + place]
    q = torch.empty(len(t), dim, dtype=torch.float64, device=raw.device)
    q[:, 0::2], q[:, 1::2] = (b % 16).double(), (b // 16).double()
    words = 2 * half + (0 if key else 4 * block * groups) + t[:, None] * 4 * groups + torch.arange(4 * groups, device=raw.device)
    sz = raw[n[:, None], h, words].view(torch.float16).double().reshape(len(t), groups, 2)
    sz = sz.repeat_interleave(dim // groups, 1)
    return sz[..., 0] * (q - sz[..., 1])


def exact(case, seed):
    if case["kind"] == "tables":
        return None
    st = prepare(case, seed)
    if case["kind"] == "append":
        out = {}
        for name in ("k", "v"):
            w = st[name].double().reshape(-1, case["group"])
            top, low = torch.clamp(w.max(1).values, min=0.0), torch.clamp(w.min(1).values, max=0.0)
            s = (top - low) / 15.0
            # the binary16 neighbours of s are found by exponent; the nearer one is taken, on a tie the even one
            e = torch.floor(torch.log2(torch.clamp(s, min=2.0**-24)))
            e = torch.where(torch.exp2(e) > s, e - 1, e)
            e = torch.where(torch.exp2(e + 1) <= s, e + 1, e).clamp(min=-14.0)
            unit = torch.exp2(e - 10)
            down = torch.floor(s / unit)
            rest = s / unit - down
            down = down + ((rest > 0.5) | ((rest == 0.5) & (down % 2 == 1))).double()
            s = torch.where(down == 0, torch.ones_like(s), down * unit)[:, None]
            z = torch.round(-low[:, None] / s).clamp(0, 15)
            level = torch.clamp(torch.round(w / s), min=-z, max=15 - z)
            out[name] = (level * s).reshape(st[name].shape)
            out[name][case["tokens"]:] = 0.0
        return out
    if 4 * _attended(case) * case["heads"] * case["dim"] > 2e12:
        return None
    q, raw, block = st["q"].double(), st["cache"], case["block"]
    ratio = case["heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    starts, kv_lens = st["q_starts"].tolist(), st["kv_lens"].tolist()
    for b, kv in enumerate(kv_lens):
        lo, hi = starts[b], starts[b + 1]
        if kv == 0 or hi == lo:
            continue
        at = torch.arange(kv, device=DEV)
        n, t = st["tables"][b].long()[at // block], at % block
        last = torch.arange(hi - lo, device=DEV)[:, None] + (kv - (hi - lo)) if case["causal"] else torch.full((hi - lo, 1), kv - 1, device=DEV)
        hidden = at[None, :] > last
        if case["window"]:
            hidden |= at[None, :] <= last - case["window"]
        for h in range(case["kv_heads"]):
            k = _exact_rows(raw, case["dim"], case["dim"] // case["group"], block, n, h, t, True)
            v = _exact_rows(raw, case["dim"], case["dim"] // case["group"], block, n, h, t, False)
            for head in range(h * ratio, (h + 1) * ratio):
                s = (q[lo:hi, head] @ k.T) / math.sqrt(case["dim"])
                s[hidden] = -math.inf
                lse[lo:hi, head] = torch.logsumexp(s, 1)
                some = ~hidden.all(1)
                out[lo:hi, head][some] = torch.softmax(s[some], 1) @ v
    return {"out": out, "lse": lse}
