"""Plain statements, in binary64, of the operators around the codec, for the
tests: products grouped by expert on decoded MXFP4 weights, the norms around a
block with their gradients, and clipping by the global norm."""
import torch

import oracle

# half an ulp of the type's 1.0 (unit roundoff) and half its smallest subnormal
ROUND = {torch.bfloat16: (2.0 ** -9, 2.0 ** -134), torch.float16: (2.0 ** -12, 2.0 ** -25),
         torch.float32: (2.0 ** -25, 2.0 ** -150)}
U32 = 2.0 ** -24                    # unit roundoff of binary32


def rounding(ref: torch.Tensor, dtype) -> torch.Tensor:
    """How far rounding to `dtype` may move a value at most (twice the half ulp
    covers the value's own error moving it to the next binade)."""
    u, s = ROUND[dtype]
    return ref.abs() * 2 * u + s


def random_packed(experts, n, k, seed, exponents=(-6, 1), special=()):
    """(packed bytes, decoded values in binary64) of random codes with block
    scales 2^e, e in the given range; `special` sets scale bytes by block."""
    count = experts * n * k
    tiles = -(-count // 2048)
    g = torch.Generator().manual_seed(seed)
    p = torch.empty(tiles, 1088, dtype=torch.uint8)
    p[:, :1024] = torch.randint(0, 256, (tiles, 1024), generator=g, dtype=torch.uint8)
    p[:, 1024:] = torch.randint(127 + exponents[0], 127 + exponents[1] + 1, (tiles, 64), generator=g, dtype=torch.uint8)
    for block, byte in special:
        p[block // 64, 1024 + block % 64] = byte
    w = torch.from_numpy(oracle.unpack_dequant(oracle.MXFP4, p.reshape(-1).numpy(), count))
    return p.reshape(-1), w.double().view(experts, n, k)


def segments(offsets, rows):
    """[(expert or None, first row, end)], all rows in order."""
    out = [(None, 0, offsets[0])] + [(e, offsets[e], offsets[e + 1]) for e in range(len(offsets) - 1)]
    return out + [(None, offsets[-1], rows)]


def grouped(x, w, offsets):
    """(y, sum of the products' magnitudes)."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(y)
    for e, a, b in segments(offsets, x.shape[0]):
        if e is not None and b > a:
            y[a:b] = x[a:b].double() @ w[e].T
            mag[a:b] = x[a:b].double().abs() @ w[e].abs().T
    return y, mag


def grouped_dx(dy, w, offsets):
    return grouped(dy, w.transpose(1, 2), offsets)


def grouped_dw(dy, x, offsets):
    experts = len(offsets) - 1
    dw = torch.zeros(experts, dy.shape[1], x.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(dw)
    for e, a, b in segments(offsets, x.shape[0]):
        if e is not None:
            dw[e] = dy[a:b].double().T @ x[a:b].double()
            mag[e] = dy[a:b].double().abs().T @ x[a:b].double().abs()
    return dw, mag


def block_norm(y, r, pre, post, gate, alpha, eps):
    """h, z, (ry, rh), in binary64."""
    y, r, pre = y.double(), r.double(), pre.double()
    ry = torch.ones_like(y[:, 0]) if post is None else (y.square().mean(1) + eps).rsqrt()
    u = y if post is None else y * ry[:, None] * post.double()
    h = alpha * r + (u if gate is None else gate.double() * u)
    rh = (h.square().mean(1) + eps).rsqrt()
    return h, h * rh[:, None] * pre, torch.stack([ry, rh])


def block_norm_backward(dz, dh, h, stats, y, pre, post, gate, alpha):
    """{name: (value, sum of the magnitudes of what is added up for it)}."""
    dz, h, y, pre = dz.double(), h.double(), y.double(), pre.double()
    ry, rh = stats.double()[:, :, None]
    d = y.shape[1]
    hn, yn = h * rh, y * ry
    t = dz * pre
    dh = torch.zeros_like(dz) if dh is None else dh.double()
    e = dh + rh * (t - hn * (t * hn).sum(1, keepdim=True) / d)
    e_mag = dh.abs() + rh * (t.abs() + hn.abs() * (t * hn).abs().sum(1, keepdim=True) / d)
    g = torch.ones(d, dtype=torch.float64) if gate is None else gate.double()
    w = torch.ones(d, dtype=torch.float64) if post is None else post.double()
    b, b_mag = e * g * w, e_mag * (g * w).abs()
    out = {"dr": (alpha * e, abs(alpha) * e_mag), "dpre": ((dz * hn).sum(0), (dz * hn).abs().sum(0))}
    if post is None:
        out["dy"] = (b, b_mag)
    else:
        out["dy"] = (ry * (b - yn * (b * yn).sum(1, keepdim=True) / d),
                     ry * (b_mag + yn.abs() * (b_mag * yn.abs()).sum(1, keepdim=True) / d))
        out["dpost"] = ((e * g * yn).sum(0), (e_mag * (g * yn).abs()).sum(0))
    if gate is not None:
        v, m = e * w * yn, e_mag * (w * yn).abs()
        out["dgate"] = (v, m) if gate.dim() == 2 else (v.sum(0), m.sum(0))
    return out


def clip(grads, scale, max_norm, eps):
    """(norm, factor) in binary64."""
    total = sum(float(g.double().square().sum()) for g in grads)
    norm = abs(scale) * total ** 0.5
    return norm, min(1.0, max_norm / (norm + eps)) * scale
