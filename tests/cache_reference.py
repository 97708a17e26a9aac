"""Plain statements, in binary64, of a paged cache held in MXFP4, for the tests:
where a row stands, what the cache holds of it, the bytes that appending writes,
and attention with a bound of its rounding."""
import math

import numpy as np
import torch

import oracle

TILE, TILE_BYTES = 2048, 1088
NAN_SCALE = 255                     # the E8M0 byte that makes every value of a block NaN
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
# the weights' rounding: to bfloat16, or to two or three terms of it
WEIGHT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -16, torch.float32: 2.0 ** -23}


def stream_bytes(page, d):
    return page * d // TILE * TILE_BYTES


def values(stream):
    """Decoded values, in binary64, of whole tiles (uint8, any shape; flat)."""
    flat = np.ascontiguousarray(stream.cpu().numpy().reshape(-1))
    return torch.from_numpy(oracle.unpack_dequant(oracle.MXFP4, flat, flat.size // TILE_BYTES * TILE)).double()


def pack(x):
    """MXFP4 tiles of binary64 values (a multiple of 2048): scale 2^(floor(log2 max) - 2), nearest code, ties to even."""
    b = np.asarray(x, dtype=np.float64).reshape(-1, 32)
    top = np.abs(b).max(1)
    e = np.where(top > 0, np.frexp(top)[1] - 3, -127).clip(-127, 127)
    a = np.ldexp(np.abs(b), -e[:, None])
    code = sum(((a >= m) if i % 2 else (a > m)).astype(np.uint8) for i, m in enumerate(MIDS))
    code = code | (np.signbit(b).astype(np.uint8) << 3)
    out = np.empty((b.shape[0] // 64, TILE_BYTES), np.uint8)
    out[:, :1024] = (code[:, 0::2] | code[:, 1::2] << 4).reshape(-1, 1024)
    out[:, 1024:] = (e + 127).astype(np.uint8).reshape(-1, 64)
    return torch.from_numpy(out.reshape(-1))


def narrow(x, dtype):
    """Binary64 values rounded once to dtype: torch goes by way of binary32 and would round twice, so the first
    step is to the neighbour towards zero, its last bit set where anything is lost."""
    if dtype == torch.float32:
        return x.float()
    a = x.numpy()
    f = a.astype(np.float32)
    over = np.abs(f.astype(np.float64)) > np.abs(a)
    bits = f.view(np.uint32) - over.astype(np.uint32)
    bits = bits | (f.astype(np.float64) != a).astype(np.uint32)
    return torch.from_numpy(bits.view(np.float32)).to(dtype)


def positions(lengths, offsets, tokens, capacity):
    """[(sequence, position) or None] of every row; lengths count within [0, capacity]."""
    out = [None] * tokens
    for s, n in enumerate(lengths):
        a, b = (min(max(o, 0), tokens) for o in offsets[s:s + 2])
        for i in range(a, b):
            out[i] = (s, min(max(n, 0), capacity) - b + i)
    return out


def turn(x, rotation, pos, interleaved):
    """Rows (heads x d, binary64) turned by the angles of position pos."""
    if rotation is None:
        return x
    r = rotation.shape[1]
    c, s = rotation[pos, :r // 2].double(), rotation[pos, r // 2:].double()
    y = x.clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return y


class Plan:
    """Sequences of (new tokens, length), their pages dealt at random among `spare` more."""

    def __init__(self, spec, page, seed=0, spare=3, wider=2, before=0, behind=0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.new, self.lengths = page, [a for a, _ in spec], [n for _, n in spec]
        need = [-(-max(n, 0) // page) for n in self.lengths]
        self.pages = sum(need) + spare
        self.max_pages = max(need, default=0) + wider
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = [[order.pop() for _ in range(n)] + [(-1, 1 << 30, -7)[i % 3] for i in range(self.max_pages - n)]
                      for n in need]
        self.offsets = [before]
        for a in self.new:
            self.offsets.append(self.offsets[-1] + a)
        self.tokens = self.offsets[-1] + behind

    def tensors(self, dev):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        return i32(self.table).view(len(self.lengths), self.max_pages), i32(self.lengths), i32(self.offsets)

    def rows(self):
        return positions(self.lengths, self.offsets, self.tokens, self.max_pages * self.page)

    def page_at(self, s, pos):
        p = self.table[s][pos // self.page] if 0 <= pos < self.max_pages * self.page else -1
        return p if 0 <= p < self.pages else -1


def random_cache(plan, kv, d, seed, exponents=(-3, 1), poison=True):
    """(k bytes, v bytes, k values, v values): pages x kv x bytes, and pages x kv x page x d. What no token is
    in has NaN scales."""
    g = torch.Generator().manual_seed(seed)
    page, out, vals = plan.page, [], []
    for _ in range(2):
        tiles = page * d // TILE
        c = torch.randint(0, 256, (plan.pages, kv, tiles, TILE_BYTES), generator=g, dtype=torch.uint8)
        c[..., 1024:] = torch.randint(127 + exponents[0], 128 + exponents[1], c[..., 1024:].shape, generator=g,
                                      dtype=torch.uint8)
        if poison:
            used = torch.zeros(plan.pages, page, dtype=torch.bool)
            for s, n in enumerate(plan.lengths):
                for pos in range(min(max(n, 0), plan.max_pages * page)):
                    if plan.page_at(s, pos) >= 0:
                        used[plan.page_at(s, pos), pos % page] = True
            bad = (~used).repeat_interleave(d // 32, 1).view(plan.pages, 1, tiles, 64).expand(-1, kv, -1, -1)
            c[..., 1024:][bad] = NAN_SCALE
        out.append(c.view(plan.pages, kv, -1))
        vals.append(values(c).view(plan.pages, kv, page, d))
    return out[0], out[1], vals[0], vals[1]


def appended(plan, cache, x, d, rotation=None, interleaved=False):
    """The cache's bytes after rows x (tokens x kv x d) are written to it."""
    kv, nb = x.shape[1], d // 32
    c = cache.clone().view(plan.pages, kv, -1, TILE_BYTES)
    for i, at in enumerate(plan.rows()):
        if at is None or at[1] < 0:
            continue
        p = plan.page_at(*at)
        if p < 0:
            continue
        y = turn(x[i].double(), rotation, at[1], interleaved)
        packed = pack(torch.cat([y.reshape(-1), torch.zeros(-y.numel() % TILE, dtype=torch.float64)]).numpy()).view(-1, TILE_BYTES)
        for h in range(kv):
            for b in range(nb):
                src, dst = h * nb + b, at[1] % plan.page * nb + b
                t = c[p, h, dst // 64]
                t[dst % 64 * 16:dst % 64 * 16 + 16] = packed[src // 64, src % 64 * 16:src % 64 * 16 + 16]
                t[1024 + dst % 64] = packed[src // 64, 1024 + src % 64]
    return c.view(cache.shape)


def attention(plan, q, kvals, vvals, scale, causal=True, window=0):
    """(out, lse, bound of out, bound of lse) in binary64, None rows' places left NaN. The bounds: a score of d
    products is off by (d + 8) 2^-23 of their magnitudes and by 2^-22 of its own size and the maximum's (the
    multiplication by the scale, the difference, the power's argument); a weight by that and WEIGHT, and by 2^-126
    of the largest, 1, where binary32 and the terms it is cut into end (exp(-88) is below that, and a weight's third
    term lies 2^-16 under it); a sum of n terms by (n + 8) 2^-23 of theirs, and by 2^-149, binary32's smallest, for
    each of the up to three products that a term is formed of, and for the division."""
    tokens, heads, d = q.shape
    group = heads // kvals.shape[1]
    out = torch.full((tokens, heads, d), math.nan, dtype=torch.float64)
    lse = torch.full((tokens, heads), math.nan, dtype=torch.float64)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    of = {}
    for i, at in enumerate(plan.rows()):
        if at is None:
            continue
        s, pos = at
        n = min(max(plan.lengths[s], 0), plan.max_pages * plan.page)
        if s not in of:
            there = [j for j in range(n) if plan.page_at(s, j) >= 0]
            pages, places = [plan.page_at(s, j) for j in there], [j % plan.page for j in there]
            of[s] = torch.tensor(there, dtype=torch.long), kvals[pages, :, places], vvals[pages, :, places]
        at_j, k, v = of[s]
        seen = torch.ones_like(at_j, dtype=torch.bool)
        if causal:
            seen = at_j <= pos
            if window:
                seen &= at_j > pos - window
        if not seen.any():
            out[i], lse[i] = 0, -math.inf
            continue
        k, v = (x[seen].repeat_interleave(group, 1) for x in (k, v))                # keys x heads x d
        qi = q[i].double()
        score = scale * (k * qi).sum(2)
        top = score.max(0).values
        e = torch.exp(score - top)
        total = e.sum(0)
        w = e / total
        out[i], lse[i] = (w[..., None] * v).sum(0), top + total.log()
        off = (d + 8) * 2.0 ** -23 * abs(scale) * (k * qi).abs().sum(2) + 2.0 ** -22 * (score.abs() + top.abs())
        count = float(seen.sum())
        rel = torch.expm1(off) + WEIGHT[q.dtype] + (count + 8) * 2.0 ** -23
        tol[i] = (w[..., None] * v.abs() * rel[..., None]).sum(0) + out[i].abs() * (w * rel).sum(0)[:, None]
        tol[i] += 2.0 ** -126 * (v.abs().sum(0) + count * out[i].abs()) + (3 * count + 1) * 2.0 ** -149
        lse_tol[i] = (w * rel).sum(0) + 2.0 ** -22 * (lse[i].abs() + 1)
    return out, lse, tol, lse_tol
