"""The large-language-model operators of this framework, as cases to time and to compare.

Three operators meet at a tensor-parallel block whose collectives are quantized:

* "experts": products grouped by expert, with ragged groups of rows, on MXFP4-packed
  weights (E experts of n x k, one packed stream of E*n*k elements), forward, and
  backward to the rows and to the weights (dense, straight through the cast);
* "norm": what stands between one block and the next: norm of the block's output, its
  gate, the scaled residual, and the norm before the next block, forward and backward;
* "clip": the global norm of many gradient tensors, and clipping by it.

``run`` computes a case in elementary torch operations in 32 bits (``own`` false) or
with the framework's calls (``own`` true); ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
TILE, TILE_BYTES = 2048, 1088            # an MXFP4 tile: 1024 bytes of codes, 64 E8M0 scales
EPS = 1e-6


def listed():
    return [
        # one generated token: its two experts of eight, the latency of a serving step
        {"name": "experts_token", "op": "experts", "dir": "fwd", "dtype": "bf16", "tokens": 1, "top": 2, "experts": 8,
         "n": 4096, "k": 4096, "skew": 0.5},
        # a decoding batch over many small experts: a few rows each, the weights' bytes count
        {"name": "experts_batch", "op": "experts", "dir": "fwd", "dtype": "bf16", "tokens": 48, "top": 4, "experts": 32,
         "n": 2048, "k": 4096, "skew": 1.0},
        # a batch of prompts: thousands of rows per expert, bound by the matrix cores
        {"name": "experts_prompt", "op": "experts", "dir": "fwd", "dtype": "bf16", "tokens": 8192, "top": 2,
         "experts": 8, "n": 8192, "k": 4096, "skew": 0.3},
        # a short prompt in fp16 with widths off every power of two
        {"name": "experts_odd_fp16", "op": "experts", "dir": "fwd", "dtype": "fp16", "tokens": 777, "top": 3,
         "experts": 12, "n": 1000, "k": 2080, "skew": 1.0},
        # the backward pass of a training step: gradients of the rows and of the weights
        {"name": "experts_train", "op": "experts", "dir": "bwd", "dtype": "bf16", "tokens": 4096, "top": 2,
         "experts": 16, "n": 2048, "k": 4096, "skew": 0.5},
        # one generated token between two blocks
        {"name": "norm_token", "op": "norm", "dir": "fwd", "dtype": "bf16", "rows": 1, "d": 4096, "post": True,
         "gate": "channel", "scale": 1.0, "save": False},
        # the rows of a batch of prompts, widest residual stream
        {"name": "norm_prompt", "op": "norm", "dir": "fwd", "dtype": "bf16", "rows": 16384, "d": 8192, "post": True,
         "gate": "channel", "scale": 0.5, "save": True},
        # a training step's backward, gate of one value per channel (its gradient is a sum over rows)
        {"name": "norm_train", "op": "norm", "dir": "bwd", "dtype": "bf16", "rows": 8192, "d": 4096, "post": True,
         "gate": "channel", "scale": 1.0, "save": True},
        # a gate of its own for every value, in fp32, at an odd width
        {"name": "norm_gated_fp32", "op": "norm", "dir": "bwd", "dtype": "fp32", "rows": 2500, "d": 1999, "post": True,
         "gate": "full", "scale": 0.7, "save": True},
        # adapters: few layers of narrow fp32 gradients, mostly latency
        {"name": "clip_small", "op": "clip", "dtype": "fp32", "layers": 6, "width": 256, "ff": 64, "max_norm": 1.0,
         "scale": 1.0},
        # odd sizes, under the limit: the averaged gradients come through scaled only
        {"name": "clip_odd", "op": "clip", "dtype": "fp16", "layers": 13, "width": 501, "ff": 1301, "max_norm": 1e9,
         "scale": 0.125},
        # a model's bf16 gradients and fp32 vectors, clipped
        {"name": "clip_model", "op": "clip", "dtype": "bf16", "layers": 16, "width": 2048, "ff": 8192, "max_norm": 1.0,
         "scale": 1.0},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + step))) // step * step)))


def draw(rng):
    c = _drawn(rng)
    while 3 * 1024 in [*c.values(), c.get("tokens", 0) * c.get("top", 0)]:
        c = _drawn(rng)
    return c


def _drawn(rng):
    op = rng.choice(["experts", "experts", "norm", "norm", "clip"])
    if op == "experts":
        c = {"op": op, "dir": rng.choice(["fwd", "fwd", "bwd"]), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
             "tokens": _log(rng, 1, 8192), "experts": _log(rng, 2, 64), "n": _log(rng, 128, 8192, 8),
             "k": _log(rng, 128, 8192, 32), "skew": rng.choice([0.0, 0.5, 1.0])}
        c["top"] = rng.randint(1, min(8, c["experts"]))
        passes = 1 if c["dir"] == "fwd" else 2
        while c["experts"] * c["n"] * c["k"] * passes > 1 << 28:
            c["n"] = max(128, c["n"] // 2 // 8 * 8)
        while c["tokens"] * c["top"] * c["n"] * c["k"] * passes > 1 << 37:
            c["tokens"] = c["tokens"] // 2 + 1
        return c
    if op == "norm":
        c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
             "rows": _log(rng, 1, 16384), "d": _log(rng, 64, 16384, rng.choice([1, 8, 64])),
             "post": rng.random() < 0.75, "gate": rng.choice(["none", "channel", "full"]),
             "scale": rng.choice([1.0, 0.5, 0.7])}
        c["save"] = c["dir"] == "bwd" or rng.random() < 0.5
        while c["rows"] * c["d"] > 1 << 26:
            c["rows"] = c["rows"] // 2 + 1
        return c
    return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "layers": _log(rng, 1, 16),
            "width": _log(rng, 64, 2048, rng.choice([1, 8])), "ff": _log(rng, 64, 4096, rng.choice([1, 8])),
            "max_norm": rng.choice([1.0, 1.0, 1e9]), "scale": rng.choice([1.0, 0.125])}


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(*shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(dtype)


def _activations(g, rows, k, dtype):
    """Rows as a residual stream has them: normal, with a few channels 20 times as large."""
    x = _randn(g, rows, k)
    big = torch.randint(0, k, (max(1, k // 512),), device=DEV, generator=g)
    x[:, big] *= 20.0
    return x.to(dtype)


def _packed_weights(g, count):
    """An MXFP4 stream of `count` weights N(0, 0.02) cast directly: blocks of 32 share 2^floor(log2 max - 2)."""
    tiles = -(-count // TILE)
    w = _randn(g, tiles, 64, 32, std=0.02)
    e = torch.floor(torch.log2(w.abs().amax(-1, keepdim=True).clamp_min(1e-30))) - 2
    v = w * torch.exp2(-e)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    q = torch.bucketize(v.abs(), mids, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    q = q.view(tiles, 1024, 2)
    return torch.cat([q[..., 0] | (q[..., 1] << 4), (e.view(tiles, 64) + 127).to(torch.uint8)], 1).reshape(-1)


def _routing(case, seed):
    """Offsets of the experts' groups of rows: every token goes to its `top` best experts, some liked more."""
    g = _gen(seed)
    liked = _randn(g, case["experts"], std=case["skew"])
    noise = torch.empty(case["tokens"], case["experts"], device=DEV).exponential_(generator=g)
    chosen = (liked - noise.log()).topk(case["top"], dim=1).indices.reshape(-1)
    counts = torch.bincount(chosen, minlength=case["experts"])
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32), int(counts.max())


def _grad_sizes(case):
    w, f = case["width"], case["ff"]
    return [(w * w, False), (w * w, False), (w * w, False), (w * w, False), (w * f, False), (w * f, False),
            (w, True), (w, True)] * case["layers"]


def prepare(case, seed):
    g = _gen(seed + 1)
    dt = DT[case["dtype"]]
    s = dict(case)
    if case["op"] == "experts":
        rows, n, k = case["tokens"] * case["top"], case["n"], case["k"]
        s["offsets"], s["most"] = _routing(case, seed)
        s["w"] = _packed_weights(g, case["experts"] * n * k)
        s["x"] = _activations(g, rows, k, dt)
        if case["dir"] == "bwd":
            s["dy"] = _randn(g, rows, n, std=1e-2, dtype=dt)
    elif case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        wt = torch.float32 if case["dtype"] == "fp32" else dt
        s["y"], s["r"] = _randn(g, rows, d, std=0.5, dtype=dt), _activations(g, rows, d, dt)
        s["pre_w"] = (1 + _randn(g, d, std=0.1)).to(wt)
        s["post_w"] = (1 + _randn(g, d, std=0.1)).to(wt) if case["post"] else None
        s["g"] = (None if case["gate"] == "none" else (0.5 + _randn(g, d, std=0.2)).to(wt) if case["gate"] == "channel"
                  else (0.5 + _randn(g, rows, d, std=0.2)).to(dt))
        if case["dir"] == "bwd":
            # what the forward pass left: h as stored, and 1 / rms of y's rows (1 without a post norm) and of h's
            y = s["y"].float()
            rstd_y = torch.rsqrt(y.square().mean(1) + EPS) if case["post"] else torch.ones(rows, device=DEV)
            u = y * rstd_y[:, None] * (s["post_w"].float() if case["post"] else 1.0)
            h = case["scale"] * s["r"].float() + u * (1.0 if s["g"] is None else s["g"].float())
            s["h"], rstd_h = h.to(dt), torch.rsqrt(h.square().mean(1) + EPS)
            s["stats"] = torch.stack([rstd_y, rstd_h])
            s["dz"], s["dh"] = _randn(g, rows, d, std=1e-2, dtype=dt), _randn(g, rows, d, std=1e-2, dtype=dt)
            del s["r"]
    else:
        sizes = _grad_sizes(case)
        mats, vecs = sum(c for c, v in sizes if not v), sum(c for c, v in sizes if v)
        flat = {False: _randn(g, mats, std=1e-3, dtype=dt), True: _randn(g, vecs, std=1e-2)}
        out = {v: torch.empty_like(t) for v, t in flat.items()}
        # one buffer per type, as collectives have them; the tensors are its parts, at whatever place they fall
        at, s["grads"], s["clipped"] = {False: 0, True: 0}, [], []
        for c, v in sizes:
            s["grads"].append(flat[v][at[v]:at[v] + c])
            s["clipped"].append(out[v][at[v]:at[v] + c])
            at[v] += c
        s["flat"], s["out"] = [flat[False], flat[True]], [out[False], out[True]]
    return s


# --------------------------------------------------------------- the calls ----

def run(s):
    return OWN[s["op"]](s) if own else PLAIN[s["op"]](s)


def _own_experts(s):
    import reduction_codec_amd as rca
    if s["dir"] == "fwd":
        return rca.mxfp4_grouped_matmul(s["x"], s["w"], s["offsets"], s["n"])
    return (rca.mxfp4_grouped_matmul_dx(s["dy"], s["w"], s["offsets"], s["k"]),
            rca.grouped_matmul_dw(s["dy"], s["x"], s["offsets"]))


def _own_norm(s):
    import reduction_codec_amd as rca
    if s["dir"] == "fwd":
        h, z, stats = rca.block_norm(s["y"], s["r"], s["pre_w"], post_weight=s["post_w"], gate=s["g"],
                                     residual_scale=s["scale"], eps=EPS, stats=s["save"])
        return {"h": h, "z": z, "stats": stats}
    dy, dr, dpre, dpost, dgate = rca.block_norm_backward(
        s["dz"], s["dh"], s["h"], s["stats"], s["y"], s["pre_w"], post_weight=s["post_w"], gate=s["g"],
        residual_scale=s["scale"])
    return {"dy": dy, "dr": dr, "dpre": dpre, "dpost": dpost, "dgate": dgate}


def _own_clip(s):
    import reduction_codec_amd as rca
    norm = rca.grad_norm_clip(s["grads"], s["max_norm"], scale=s["scale"], eps=EPS, out=s["clipped"])
    return [norm] + s["out"]


OWN = {"experts": _own_experts, "norm": _own_norm, "clip": _own_clip}


# --------------------------------------------------------- the plain forms ----

def _decode(w):
    """Values of MXFP4 tiles (..., tiles, 1088 bytes) -> (..., tiles * 2048) in fp32."""
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    byte = torch.arange(256, device=DEV)
    pairs = torch.stack([one[byte & 15], one[byte >> 4]], 1)
    codes = pairs[w[..., :1024].int()].view(*w.shape[:-1], 64, 32)
    return (codes * torch.exp2(w[..., 1024:].float() - 127)[..., None]).flatten(-3)


def _plain_experts(s):
    """Rows laid out by expert with room for the largest group, one batched product, rows back. Fewer rows than
    experts: each row with its own expert's weights."""
    n, k, off, x = s["n"], s["k"], s["offsets"].long(), s["x"]
    rows, E = x.shape[0], off.numel() - 1
    at = torch.arange(rows, device=DEV)
    expert = torch.searchsorted(off[1:].contiguous(), at, right=True)
    tiles = s["w"].view(-1, TILE_BYTES)
    if s["dir"] == "fwd" and rows < E and (n * k) % TILE == 0:
        w = _decode(tiles.view(E, -1, TILE_BYTES)[expert]).view(rows, n, k)
        return torch.matmul(w, x.float()[:, :, None])[..., 0].to(x.dtype)
    w = _decode(tiles)[:E * n * k].view(E, n, k)
    place = expert * s["most"] + at - off[expert]
    xs = torch.zeros(E * s["most"], k, device=DEV).index_copy_(0, place, x.float()).view(E, s["most"], k)
    if s["dir"] == "fwd":
        return torch.matmul(xs, w.transpose(1, 2)).view(-1, n)[place].to(x.dtype)
    dys = torch.zeros(E * s["most"], n, device=DEV).index_copy_(0, place, s["dy"].float()).view(E, s["most"], n)
    return torch.matmul(dys, w).view(-1, k)[place].to(x.dtype), torch.matmul(dys.transpose(1, 2), xs)


def _plain_norm(s):
    y, dt = s["y"].float(), s["y"].dtype
    gate = 1.0 if s["g"] is None else s["g"].float()
    pre, post = s["pre_w"].float(), s["post_w"].float() if s["post"] else 1.0
    if s["dir"] == "fwd":
        rstd_y = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) if s["post"] else torch.ones_like(y[:, :1])
        h = s["scale"] * s["r"].float() + gate * (y * rstd_y * post)
        rstd_h = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        stats = torch.stack([rstd_y[:, 0], rstd_h[:, 0]]) if s["save"] else None
        return {"h": h.to(dt), "z": (h * rstd_h * pre).to(dt), "stats": stats}
    rstd_y, rstd_h = s["stats"][0, :, None], s["stats"][1, :, None]
    dz, hn = s["dz"].float(), s["h"].float() * rstd_h
    a = dz * pre
    dh = s["dh"].float() + rstd_h * (a - hn * (a * hn).mean(1, keepdim=True))
    yn = y * rstd_y
    du = dh * gate
    b = du * post
    dy = rstd_y * (b - yn * (b * yn).mean(1, keepdim=True)) if s["post"] else b
    dgate = dh * yn * post
    return {"dy": dy.to(dt), "dr": (s["scale"] * dh).to(dt), "dpre": (dz * hn).sum(0),
            "dpost": (du * yn).sum(0) if s["post"] else None,
            "dgate": None if s["gate"] == "none" else dgate.sum(0) if s["gate"] == "channel" else dgate.to(dt)}


def _plain_clip(s):
    """On the two buffers that the tensors are parts of, so that their number costs nothing here."""
    mats, vecs = s["flat"]
    norm = (mats.float().square().sum() + vecs.square().sum()).sqrt() * s["scale"]
    factor = (s["max_norm"] / (norm + EPS)).clamp(max=1.0) * s["scale"]
    s["out"][0].copy_(mats.float() * factor)
    s["out"][1].copy_(vecs * factor)
    return [norm.reshape(1)] + s["out"]


PLAIN = {"experts": _plain_experts, "norm": _plain_norm, "clip": _plain_clip}


# ------------------------------------------------------------ what it needs ----

def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] == "experts":
        rows, E, n, k = case["tokens"] * case["top"], case["experts"], case["n"], case["k"]
        # experts that some row goes to, were every expert liked alike
        active = E * (1 - (1 - case["top"] / E) ** case["tokens"])
        weights = active * n * k * TILE_BYTES / TILE
        if case["dir"] == "fwd":
            return {"bytes": weights + rows * (n + k) * b, "flops": 2 * rows * n * k}
        return {"bytes": weights + rows * (n + 2 * k) * b + E * n * k * 4, "flops": 4 * rows * n * k}
    if case["op"] == "norm":
        each = case["rows"] * case["d"]
        full = 1 if case["gate"] == "full" else 0
        vectors = 1 + int(case["post"]) + int(case["gate"] == "channel")
        wb = 4 if case["dtype"] == "fp32" else 2
        if case["dir"] == "fwd":
            return {"bytes": (4 + full) * each * b + vectors * case["d"] * wb, "flops": 12 * each}
        return {"bytes": (6 + 2 * full) * each * b + vectors * case["d"] * (wb + 4) + 8 * case["rows"],
                "flops": 25 * each}
    sizes = _grad_sizes(case)
    total = sum(c * (4 if v else b) for c, v in sizes)
    return {"bytes": 2 * total + 4, "flops": 3 * sum(c for c, _ in sizes)}


# ------------------------------------------------------------- in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    return {"experts": _exact_experts, "norm": _exact_norm, "clip": _exact_clip}[case["op"]](s)


def _exact_experts(s):
    n, k = s["n"], s["k"]
    off = s["offsets"].tolist()
    E = len(off) - 1
    tiles = s["w"].view(-1, TILE_BYTES)
    x = s["x"]
    y = torch.zeros(x.shape[0], n, dtype=torch.float64, device=DEV)
    dx = torch.zeros(x.shape[0], k, dtype=torch.float64, device=DEV)
    dw = torch.zeros(E, n, k, dtype=torch.float64, device=DEV) if s["dir"] == "bwd" else None
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        first, last = e * n * k // TILE, -(-(e + 1) * n * k // TILE)
        t = tiles[first:last]
        nib = torch.stack([t[:, :1024] & 15, t[:, :1024] >> 4], 2).reshape(-1, 2048)
        mag, ex = (nib & 1).double(), ((nib >> 1) & 3).double()
        v = torch.where(ex == 0, mag / 2, (1 + mag / 2) * torch.exp2(ex - 1)) * (1.0 - 2.0 * (nib >> 3).double())
        v = v.view(-1, 64, 32) * torch.exp2(t[:, 1024:].double() - 127)[..., None]
        w = v.reshape(-1)[e * n * k - first * TILE:][:n * k].view(n, k)
        xe = x[a:b].double()
        if s["dir"] == "fwd":
            y[a:b] = xe @ w.T
        else:
            dye = s["dy"][a:b].double()
            dx[a:b] = dye @ w
            dw[e] = dye.T @ xe
    return y if s["dir"] == "fwd" else (dx, dw)


def _exact_norm(s):
    d = s["d"]
    y = s["y"].double()
    g = torch.ones(d, dtype=torch.float64, device=DEV) if s["g"] is None else s["g"].double()
    w2 = s["pre_w"].double()
    w1 = s["post_w"].double() if s["post"] else None
    if s["dir"] == "fwd":
        ry = torch.ones_like(y[:, 0]) if w1 is None else 1 / ((y * y).sum(1) / d + EPS).sqrt()
        u = y if w1 is None else y * ry[:, None] * w1
        h = s["r"].double() * s["scale"] + g * u
        rh = 1 / ((h * h).sum(1) / d + EPS).sqrt()
        return {"h": h, "z": h * rh[:, None] * w2, "stats": torch.stack([ry, rh]) if s["save"] else None}
    ry, rh = s["stats"].double()
    h, dz = s["h"].double(), s["dz"].double()
    # z = w2 h rh with rh = (mean h^2 + eps)^(-1/2): dz/dh = w2 rh - w2 h rh^3 h / d
    dh = s["dh"].double() + dz * w2 * rh[:, None] - h * (rh ** 3 / d * (dz * w2 * h).sum(1))[:, None]
    du = dh * g
    out = {"dr": s["scale"] * dh, "dpre": (dz * h * rh[:, None]).sum(0), "dpost": None, "dgate": None}
    u = y
    if w1 is None:
        out["dy"] = du
    else:
        out["dy"] = du * w1 * ry[:, None] - y * (ry ** 3 / d * (du * w1 * y).sum(1))[:, None]
        out["dpost"] = (du * y * ry[:, None]).sum(0)
        u = y * ry[:, None] * w1
    if s["gate"] != "none":
        out["dgate"] = (dh * u).sum(0) if s["gate"] == "channel" else dh * u
    return out


def _exact_clip(s):
    norm = math.sqrt(sum(float((t.double() ** 2).sum()) for t in s["grads"])) * s["scale"]
    factor = min(1.0, s["max_norm"] / (norm + EPS)) * s["scale"]
    mats = [t for t, (_, v) in zip(s["grads"], _grad_sizes(s)) if not v]
    vecs = [t for t, (_, v) in zip(s["grads"], _grad_sizes(s)) if v]
    return [torch.tensor([norm], dtype=torch.float64), torch.cat(mats).double() * factor,
            torch.cat(vecs).double() * factor]
