"""The operators of a key/value cache held in MXFP4, as cases to time and to compare.

What stands before a tensor-parallel block's first all-reduce: a paged cache of keys and
values in 4 bits, written as tokens come and read by attention.

* "append": q and k of new tokens are rotated by their positions, k and v quantized into
  the cache's pages; the rows' values are then read back as the cache holds them;
* "attention": queries over the pages of their sequences: one token of each, a few (a
  draft to be verified), a chunk behind a long context, whole prompts.

A cache is pages x kv_heads x (page * d / 2048) MXFP4 tiles (1024 bytes of codes, 64 E8M0
scales), ``table`` lists every sequence's pages, ``lengths`` its tokens with the new ones,
``offsets`` the rows that are new.  ``run`` computes a case in elementary torch operations
(``own`` false) or with the framework's calls (``own`` true); ``exact`` in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
TILE, TILE_BYTES = 2048, 1088            # an MXFP4 tile: 1024 bytes of codes, 64 E8M0 scales
BASE = 10000.0                           # of the rotation's angles


def _append(name, dtype, seqs, new, context, **more):
    c = {"name": name, "op": "append", "dtype": dtype, "seqs": seqs, "new": new, "context": context, "ragged": 0.5,
         "heads": 32, "kv": 8, "d": 128, "page": 16, "rot": 128, "interleaved": False}
    return {**c, **more}


def _attention(name, dtype, seqs, new, context, **more):
    c = {"name": name, "op": "attention", "dtype": dtype, "seqs": seqs, "new": new, "context": context, "ragged": 0.5,
         "heads": 32, "kv": 8, "d": 128, "page": 16, "causal": True, "window": 0, "lse": False}
    return {**c, **more}


def listed():
    return [
        # one generated token of one sequence: the latency of a serving step
        _append("append_token", "bf16", 1, 1, 4000),
        # a decoding batch: one token of each of 64 sequences, contexts of all lengths
        _append("append_batch", "bf16", 64, 1, 2000),
        # prompts of a few sequences, 16384 tokens: bound by memory
        _append("append_prompt", "bf16", 4, 4096, 0, page=64),
        # chunks in fp32, heads of 96 of which 64 values are rotated, neighbours paired, as many kv heads as heads
        _append("append_odd_fp32", "fp32", 3, 259, 700, heads=5, kv=5, d=96, page=64, rot=64, interleaved=True),
        # one generated token of one sequence
        _attention("attend_token", "bf16", 1, 1, 4000),
        # a decoding batch with contexts of all lengths
        _attention("attend_batch", "bf16", 32, 1, 4000, ragged=0.9),
        # the same of long contexts: gigabytes of cache
        _attention("attend_long", "bf16", 64, 1, 16000, page=64),
        # a few tokens of a draft verified at once in fp16, narrow heads, sliding window
        _attention("attend_draft_fp16", "fp16", 16, 5, 5000, heads=16, kv=4, d=64, page=32, window=2048, lse=True),
        # a chunk of a prompt behind a long context
        _attention("attend_chunk", "bf16", 2, 512, 30000, page=64),
        # whole prompts, causal: bound by the matrix cores
        _attention("attend_prompt", "bf16", 2, 6000, 0, page=64),
        # a long prompt of wide heads, few of them
        _attention("attend_wide", "bf16", 1, 8192, 0, heads=16, kv=2, d=256, ragged=0.0),
        # odd sizes in fp32, one kv head a head, every query over all keys, with the log-sum-exp
        _attention("attend_odd_fp32", "fp32", 5, 37, 777, heads=7, kv=7, d=192, page=32, causal=False, lse=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    d = rng.choice([64, 96, 128, 128, 128, 192, 256])
    least = {64: 32, 96: 64, 128: 16, 192: 32, 256: 16}[d]
    kv = rng.choice([1, 2, 3, 4, 5, 8])
    c = {"dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "seqs": _log(rng, 1, 64), "d": d, "kv": kv,
         "heads": kv * rng.choice([1, 2, 4, 5, 8]), "page": least * rng.choice([1, 2, 4]),
         "ragged": rng.choice([0.0, 0.5, 0.9])}
    if rng.random() < 0.4:
        c.update(op="append", new=_log(rng, 1, 4096), context=rng.choice([0, _log(rng, 1, 16384)]),
                 rot=rng.choice([0, d // 2, d, d]) // 16 * 16, interleaved=rng.random() < 0.3)
        while c["seqs"] * c["new"] * (c["heads"] + 2 * kv) * d > 1 << 26:
            c["seqs"], c["new"] = c["seqs"] // 2 + 1, c["new"] // 2 + 1
        return c
    c.update(op="attention", new=rng.choice([1, 1, 1, _log(rng, 2, 16), _log(rng, 16, 4096)]),
             context=_log(rng, 1, 32768), causal=rng.random() < 0.8, lse=rng.random() < 0.3)
    c["window"] = _log(rng, 16, 8192) if c["causal"] and rng.random() < 0.3 else 0
    passes = {"bf16": 1, "fp16": 4, "fp32": 9}[c["dtype"]]
    while c["seqs"] * (c["context"] + c["new"]) * kv * d > 1 << 29 or \
            c["seqs"] * c["new"] * (c["context"] + c["new"]) * c["heads"] * d * passes > 1 << 37:
        c["seqs"], c["new"], c["context"] = -(-c["seqs"] // 2), -(-c["new"] // 2), -(-c["context"] // 2)
    return c


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 7919 + 29)


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(*shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(dtype)


def _channels(g, d):
    """How large each value of a head is: alike, but for a few channels that keys have."""
    size = torch.ones(d, device=DEV)
    size[torch.randint(0, d, (max(1, d // 32),), device=DEV, generator=g)] = 5.0
    return size


def _spread(most, ragged, count):
    """Sizes from `most` down to the share of it that `ragged` leaves, evenly."""
    return [int(most * (1 - ragged * (i + 0.5) / count)) for i in range(count)]


def _sizes(case, seed):
    """(new tokens, length in the cache with them) of every sequence, in an order that the seed gives."""
    g = torch.Generator().manual_seed(seed * 31 + 7)
    new, context = ([sizes[i] for i in torch.randperm(case["seqs"], generator=g).tolist()] for sizes in _parts(case))
    return new, [n + c for n, c in zip(new, context)]


def _parts(case):
    return ([max(1, n) for n in _spread(case["new"], case["ragged"], case["seqs"])],
            _spread(case["context"], case["ragged"], case["seqs"]))


def _filled(g, pages, kv, page, d, size):
    """A cache of normal values, quantized 2^26 at a time."""
    tiles = page * d // TILE
    cache = torch.empty(pages, kv, tiles * TILE_BYTES, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (kv * page * d))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        _pack((_randn(g, b - a, kv, page, d) * size).view(-1, 32), cache[a:b].view(-1, TILE_BYTES))
    return cache


def _pack(x, tiles):
    """Blocks of 32 values into MXFP4 tiles: 2^e, e = floor(log2 max) - 2, and the nearest codes, ties to even ones."""
    top = x.abs().amax(1)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)
    e = torch.where(top == 0, -127, e)
    v = torch.ldexp(x, -e[:, None])
    a = v.abs()
    code = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += a >= mid if i % 2 else a > mid
    code += torch.signbit(v).to(torch.uint8) << 3
    tiles[:, :1024] = (code[:, 0::2] | code[:, 1::2] << 4).view(-1, 1024)
    tiles[:, 1024:] = (e + 127).to(torch.uint8).view(-1, 64)


def prepare(case, seed):
    g = _gen(seed + 1)
    s = dict(case)
    dt, d, kv, page, seqs = DT[case["dtype"]], case["d"], case["kv"], case["page"], case["seqs"]
    new, length = _sizes(case, seed)
    s["new_of"], s["length_of"] = new, length
    tokens, width = sum(new), -(-max(length) // page)
    # append touches the pages of new tokens only: the others are not made
    first = [(n - m) // page if case["op"] == "append" else 0 for n, m in zip(length, new)]
    used = [range(a, -(-n // page)) for a, n in zip(first, length)]
    pages = sum(map(len, used)) + 3
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    table = torch.zeros(seqs, width, dtype=torch.int32, device=DEV)
    at = 0
    for i, r in enumerate(used):
        table[i, r.start:r.stop] = order[at:at + len(r)]
        at += len(r)
    s["table"] = table
    s["lengths"] = torch.tensor(length, dtype=torch.int32, device=DEV)
    s["offsets"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    size = _channels(g, d)
    s["k_cache"], s["v_cache"] = _filled(g, pages, kv, page, d, size), _filled(g, pages, kv, page, d, 1.0)
    if case["op"] == "attention":
        s["q"] = _randn(g, tokens, case["heads"], d, std=1.2, dtype=dt)
        return s
    # the three parts of one fused projection's output, as they lie there
    qkv = _randn(g, tokens, case["heads"] + 2 * kv, d)
    qkv[:, case["heads"]:case["heads"] + kv] *= size
    s["qkv"] = qkv.to(dt)
    s["rotation"] = None
    if case["rot"]:
        half = case["rot"] // 2
        angle = torch.arange(width * page, device=DEV).double()[:, None] * BASE ** (
            -torch.arange(half, device=DEV).double() / half)
        s["rotation"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return s


# --------------------------------------------------------------- the calls ----

def run(s):
    return (OWN if own else PLAIN)[s["op"]](s)


def _own_append(s):
    import reduction_codec_amd as rca
    q, k, v = s["qkv"].split([s["heads"], s["kv"], s["kv"]], 1)
    q = rca.mxfp4_cache_append(k, v, s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["offsets"], q=q,
                               rotation=s["rotation"], interleaved=s["interleaved"])
    k, v = rca.mxfp4_cache_read(s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["offsets"], k.shape[0], s["d"],
                                dtype=k.dtype)
    return {"q": q, "k": k, "v": v}


def _own_attention(s):
    import reduction_codec_amd as rca
    r = rca.mxfp4_cache_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["offsets"],
                                  causal=s["causal"], window=s["window"], max_query=s["new"], lse=s["lse"])
    return {"out": r[0], "lse": r[1]} if s["lse"] else {"out": r, "lse": None}


OWN = {"append": _own_append, "attention": _own_attention}


# --------------------------------------------------------- the plain forms ----

def _decode(tiles):
    """Values of MXFP4 tiles (..., 1088) -> (..., 2048) in fp32."""
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    byte = torch.arange(256, device=DEV)
    pairs = torch.stack([one[byte & 15], one[byte >> 4]], 1)
    codes = pairs[tiles[..., :1024].int()].view(*tiles.shape[:-1], 64, 32)
    return (codes * torch.exp2(tiles[..., 1024:].float() - 127)[..., None]).flatten(-2)


def _places(s):
    """Position, and page and place in it, of every row."""
    off, length = s["offsets"].long(), s["lengths"].long()
    at = torch.arange(sum(s["new_of"]), device=DEV)
    seq = torch.searchsorted(off[1:].contiguous(), at, right=True)
    pos = length[seq] - off[seq + 1] + at
    return pos, s["table"][seq, pos // s["page"]].long(), pos % s["page"]


def _rotate(x, turn, half, interleaved):
    """Rows (tokens, heads, d) turned by their tokens' angles; in 64 bits, as the codes of what lies next to the
    border between two of them hang on the last bit."""
    x = x.double()
    cos, sin = turn[:, None, :half].double(), turn[:, None, half:].double()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    y = x.clone()
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    else:
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_append(s):
    q, k, v = s["qkv"].split([s["heads"], s["kv"], s["kv"]], 1)
    dt, d, kv, page, n = k.dtype, s["d"], s["kv"], s["page"], k.shape[0]
    pos, pages, place = _places(s)
    if s["rot"]:
        turn = s["rotation"][pos]
        q = _rotate(q, turn, s["rot"] // 2, s["interleaved"]).to(dt)
        k = _rotate(k, turn, s["rot"] // 2, s["interleaved"])
    else:
        q = q.clone()
    out = {"q": q}
    # block b of a head's page: its codes' and its scale's first byte
    block = place[:, None] * (d // 32) + torch.arange(d // 32, device=DEV)
    base = ((pages[:, None] * kv + torch.arange(kv, device=DEV)) * (page * d // TILE))[:, :, None]
    tile = (base + block[:, None] // 64) * TILE_BYTES
    codes_at = ((tile + block[:, None] % 64 * 16)[..., None] + torch.arange(16, device=DEV)).flatten()
    scale_at = (tile + 1024 + block[:, None] % 64).flatten()
    blocks = n * kv * d // 32
    for name, x, cache in (("k", k, s["k_cache"]), ("v", v, s["v_cache"])):
        packed = torch.zeros(-(-blocks // 64), TILE_BYTES, dtype=torch.uint8, device=DEV)
        rows = torch.zeros(packed.shape[0] * 64, 32, dtype=x.dtype if x.dtype == torch.float64 else torch.float32,
                           device=DEV)
        rows[:blocks] = x.reshape(-1, 32)
        _pack(rows, packed)
        flat = cache.view(-1)
        flat[codes_at] = packed[:, :1024].reshape(-1)[:blocks * 16]
        flat[scale_at] = packed[:, 1024:].reshape(-1)[:blocks]
        again = torch.zeros_like(packed)
        again[:, :1024].view(-1, 1024)[:] = torch.nn.functional.pad(flat[codes_at], (0, -blocks * 16 % 1024)).view(-1, 1024)
        again[:, 1024:] = torch.nn.functional.pad(flat[scale_at], (0, -blocks % 64)).view(-1, 64)
        out[name] = _decode(again).view(-1)[:n * kv * d].view(n, kv, d).to(dt)
    return out


def _plain_attention(s):
    """Sequence by sequence: its pages decoded, all scores, their softmax."""
    q, d, kv, page = s["q"], s["d"], s["kv"], s["page"]
    group = s["heads"] // kv
    outs, lses, a = [], [], 0
    for i, (m, n) in enumerate(zip(s["new_of"], s["length_of"])):
        pages = s["table"][i, :-(-n // page)].long()
        k, v = [_decode(c[pages].view(len(pages), kv, -1, TILE_BYTES)).view(len(pages), kv, page, d).transpose(0, 1)
                .reshape(kv, -1, d)[:, :n] for c in (s["k_cache"], s["v_cache"])]
        rows = q[a:a + m].float().view(m, kv, group, d).transpose(0, 1).reshape(kv, m * group, d)
        score = torch.matmul(rows, k.transpose(1, 2).contiguous()) * d ** -0.5
        if s["causal"]:
            key = torch.arange(n, device=DEV)
            pos = torch.arange(n - m, n, device=DEV).repeat_interleave(group)[:, None]
            hidden = key > pos
            if s["window"]:
                hidden = hidden | (key <= pos - s["window"])
            score.masked_fill_(hidden, -math.inf)
        top = score.amax(2, keepdim=True)
        p = torch.exp(score - top)
        total = p.sum(2, keepdim=True)
        out = torch.matmul(p, v.contiguous()) / total
        outs.append(out.view(kv, m, group, d).transpose(0, 1).reshape(m, -1, d).to(q.dtype))
        lses.append((top + total.log()).view(kv, m, group).transpose(0, 1).reshape(m, -1))
        a += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses) if s["lse"] else None}


PLAIN = {"append": _plain_append, "attention": _plain_attention}


# ------------------------------------------------------------ what it needs ----

def work(case):
    b, d, kv, heads = SIZE[case["dtype"]], case["d"], case["kv"], case["heads"]
    new, context = _parts(case)
    tokens, mean = sum(new), sum(context) / case["seqs"]
    cell = 2 * kv * d * 17 / 32                                        # a token's keys and values in the cache
    if case["op"] == "append":
        # rows in, q out, the cache written, and read again to values; the rows' angles
        return {"bytes": tokens * ((2 * heads + 4 * kv) * d * b + 2 * cell + case["rot"] * 4),
                "flops": tokens * (heads + kv) * case["rot"] * 3 + tokens * 2 * kv * d * 4}
    keys = pairs = 0
    for n in new:                                                      # behind contexts of the mean length
        if case["window"]:
            keys += min(mean + n, case["window"] + n - 1)
            pairs += sum(min(case["window"], mean + i + 1) for i in range(n))
        else:
            keys += mean + n
            pairs += n * mean + (n * (n + 1) / 2 if case["causal"] else n * n)
    return {"bytes": keys * cell + tokens * heads * (2 * d * b + 4 * int(case["lse"])), "flops": pairs * heads * d * 4}


# ------------------------------------------------------------- in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _exact_append(s):
    """The rows alone: what a value turned and rounded to its block's grid is. The grid's step at x is 2^(e-1) up to
    2 * 2^e and twice and four times that above, and half to even steps is half to even codes."""
    q, k, v = (t.double() for t in s["qkv"].split([s["heads"], s["kv"], s["kv"]], 1))
    r = s["rot"]
    if r:
        start = [n - m for n, m in zip(s["length_of"], s["new_of"])]
        pos = torch.cat([torch.arange(b, b + m, device=DEV) for b, m in zip(start, s["new_of"])])
        turn = torch.complex(s["rotation"][pos, :r // 2].double(), s["rotation"][pos, r // 2:].double())[:, None]
        done = []
        for x in (q, k):
            pairs = x[..., :r].unflatten(-1, (-1, 2) if s["interleaved"] else (2, -1))
            pairs = pairs if s["interleaved"] else pairs.transpose(-1, -2)
            z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * turn)
            z = z if s["interleaved"] else z.transpose(-1, -2)
            done.append(torch.cat([z.flatten(-2), x[..., r:]], -1))
        q, k = done
    grid = []
    for x in (k, v):
        blocks = x.reshape(-1, 32)
        top = blocks.abs().amax(1, keepdim=True)
        e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
        step = torch.ldexp(torch.ones_like(blocks), e - 1)
        size = blocks.abs() / step                                     # in steps of 0.5: 0 .. 16
        code = torch.where(size < 4, size.round(), torch.where(size < 8, (size / 2).round() * 2, (size / 4).round() * 4))
        grid.append((code.clamp(max=12) * step * blocks.sign()).view(x.shape))
    return {"q": q, "k": grid[0], "v": grid[1]}


def _exact_attention(s):
    """Head by head: nibble values by bits, e^x of 64-bit scores."""
    d, kv, page = s["d"], s["kv"], s["page"]
    group = s["heads"] // kv
    tokens = s["q"].shape[0]
    out = torch.zeros(tokens, s["heads"], d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(tokens, s["heads"], dtype=torch.float64, device=DEV)

    def values(cache, pages, head, n):
        t = cache[pages, head].view(-1, TILE_BYTES)
        nib = torch.stack([t[:, :1024] & 15, t[:, :1024] >> 4], 2).reshape(-1, 64, 32)
        frac, ex = (nib & 1).double(), ((nib >> 1) & 3).double()
        x = torch.where(ex == 0, frac / 2, (1 + frac / 2) * torch.exp2(ex - 1)) * (1.0 - 2.0 * (nib >> 3).double())
        return (x * torch.exp2(t[:, 1024:].double() - 127)[..., None]).reshape(-1, d)[:n]

    a = 0
    for i, (m, n) in enumerate(zip(s["new_of"], s["length_of"])):
        pages = s["table"][i, :-(-n // page)].long()
        seen = torch.ones(m, n, dtype=torch.bool, device=DEV)
        if s["causal"]:
            back = torch.arange(n - m, n, device=DEV)[:, None] - torch.arange(n, device=DEV)
            seen = (back >= 0) & (back < s["window"]) if s["window"] else back >= 0
        for head in range(kv):
            k, v = values(s["k_cache"], pages, head, n), values(s["v_cache"], pages, head, n)
            for h in range(head * group, (head + 1) * group):
                score = (s["q"][a:a + m, h].double() @ k.T / math.sqrt(d)).where(seen, -math.inf)
                lse[a:a + m, h] = torch.logsumexp(score, 1)
                out[a:a + m, h] = torch.exp(score - lse[a:a + m, h, None]) @ v
        a += m
    return {"out": out, "lse": lse if s["lse"] else None}
