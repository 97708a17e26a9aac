"""The norms around a block, forward and backward, against binary64.

Tolerances: a row's sum of squares goes through at most 32 + 6 + 16 additions
of binary32 and the products around it through fewer than 10 roundings, so
every value is held to 64 units of 2^-24 of the magnitudes added up for it,
plus one rounding to its type; sums over rows to (rows + 64) such units."""
import pytest
import torch

import reduction_codec_amd as rca
from tests import op_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 1), (3, 7), (1, 64), (2, 129), (5, 1000), (4, 2048), (3, 4096), (2, 4097), (70, 333), (2, 8192),
          (3, 10001), (2, 16384), (2, 20000), (1, 32768), (1025, 72), (700, 1024)]
EPS = 1e-6


def inputs(rows, d, dtype, wtype, gate, post, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g) * std + mean  # noqa: E731
    y, r = rn(rows, d, std=0.5).to(dtype), rn(rows, d).to(dtype)
    r[:, :: max(1, d // 3)] *= 20
    pre = rn(d, std=0.2, mean=1.0).to(wtype)
    w = rn(d, std=0.2, mean=1.0).to(wtype) if post else None
    ga = None if gate == "none" else rn(d, std=0.3, mean=0.5).to(wtype) if gate == "channel" else rn(rows, d, std=0.3, mean=0.5).to(dtype)
    return y, r, pre, w, ga


def gpu(t):
    return None if t is None else t.to(DEV)


def within(got, want, mag, units, dtype, what):
    tol = units * ref.U32 * mag + ref.rounding(want, dtype)
    off = (got.cpu().double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp_min(1e-300)).max()))


def check_forward(y, r, pre, w, ga, alpha, dtype, what):
    h, z, st = rca.block_norm(gpu(y), gpu(r), gpu(pre), post_weight=gpu(w), gate=gpu(ga), residual_scale=alpha,
                              eps=EPS, stats=True)
    alpha32, eps32 = float(torch.tensor(alpha)), float(torch.tensor(EPS))
    hr, zr, sr = ref.block_norm(y, r, pre, w, ga, alpha32, eps32)
    gu = (hr - alpha32 * r.double()).abs()
    mag = (alpha32 * r.double()).abs() + gu
    within(st, sr, sr, 64, torch.float32, what + " stats")
    within(h, hr, mag, 64, dtype, what + " h")
    within(z, zr, mag * sr[1][:, None] * pre.double().abs(), 128, dtype, what + " z")
    return h, st


def check_backward(dz, dh, h, st, y, pre, w, ga, alpha, dtype, what):
    out = rca.block_norm_backward(gpu(dz), gpu(dh), h, st, gpu(y), gpu(pre), post_weight=gpu(w), gate=gpu(ga),
                                  residual_scale=alpha)
    want = ref.block_norm_backward(dz, dh, h.cpu(), st.cpu(), y, pre, w, ga, float(torch.tensor(alpha)))
    rows = y.shape[0]
    for name, got in zip(("dy", "dr", "dpre", "dpost", "dgate"), out):
        if name not in want:
            assert got is None, name
            continue
        v, m = want[name]
        if got.dim() == 2:
            within(got, v, m, 160, dtype, f"{what} {name}")
        else:
            assert got.dtype == torch.float32
            within(got, v, m, rows + 224, torch.float32, f"{what} {name}")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward_and_backward(rows, d, dtype):
    for gate, post, wtype, alpha in (("channel", True, dtype, 0.5), ("full", True, torch.float32, 0.7),
                                     ("none", False, torch.float16, 1.0), ("full", False, dtype, -1.0),
                                     ("channel", False, torch.bfloat16, 0.0)):
        what = f"{rows}x{d} {dtype} gate={gate} post={post}"
        print("case " + what, flush=True)
        y, r, pre, w, ga = inputs(rows, d, dtype, wtype, gate, post, seed=rows + d)
        h, st = check_forward(y, r, pre, w, ga, alpha, dtype, what)
        g = torch.Generator().manual_seed(3)
        dz, dh = (torch.randn(rows, d, generator=g) * 0.1).to(dtype), (torch.randn(rows, d, generator=g) * 0.1).to(dtype)
        check_backward(dz, dh if post else None, h, st, y, pre, w, ga, alpha, dtype, what)


def test_in_place():
    y, r, pre, w, ga = (gpu(t) for t in inputs(37, 520, torch.bfloat16, torch.bfloat16, "full", True))
    h, z, st = rca.block_norm(y, r, pre, post_weight=w, gate=ga, stats=True)
    y2, r2 = y.clone(), r.clone()
    rca.block_norm(y2, r2, pre, post_weight=w, gate=ga, h=r2, z=y2)
    assert torch.equal(r2, h) and torch.equal(y2, z)
    dz, dh = torch.randn_like(y), torch.randn_like(y)
    a = rca.block_norm_backward(dz, dh, h, st, y, pre, post_weight=w, gate=ga)
    dz2, dh2 = dz.clone(), dh.clone()
    b = rca.block_norm_backward(dz2, dh2, h, st, y, pre, post_weight=w, gate=ga, dy=dz2, dresidual=dh2)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_zero_rows_and_rows_of_zeros():
    pre = torch.ones(24, device=DEV)
    y = torch.zeros(5, 24, device=DEV)
    h, z, st = rca.block_norm(y, y, pre, post_weight=pre, stats=True)
    assert not h.any() and not z.any() and torch.allclose(st, torch.full_like(st, 1000.0), rtol=1e-6)
    out = rca.block_norm_backward(y, None, h, st, y, pre, post_weight=pre)
    assert all(not t.any() for t in out if t is not None)
    e = torch.empty(0, 24, device=DEV)
    h, z, st = rca.block_norm(e, e, pre, stats=True)
    assert h.shape == e.shape
    dy, dr, dpre, dpost, dgate = rca.block_norm_backward(e, e, h, st, e, pre, post_weight=pre, gate=pre)
    assert not dpre.any() and not dpost.any() and not dgate.any() and dy.shape == e.shape


def test_large_and_tiny_values():
    """Rows whose squares leave binary32's range come out as the formula in
    binary32 gives them (the norm of an overflowing sum is infinite: z = 0); a
    row of small normal values is scaled up."""
    pre = torch.ones(512, device=DEV)
    r = torch.zeros(3, 512, device=DEV)
    r[0], r[1], r[2] = 1e25, 1e-15, 3.0
    h, z, _ = rca.block_norm(torch.zeros_like(r), r, pre)
    assert torch.equal(h, r) and not z[0].any()
    assert torch.allclose(z[2], torch.ones(512, device=DEV), rtol=1e-5)
    x = torch.full((2, 64), 1.0, device=DEV)
    x[0, 5] = float("nan")
    h, z, _ = rca.block_norm(x, x, torch.ones(64, device=DEV), post_weight=torch.ones(64, device=DEV))
    assert z[0].isnan().all() and z[1].isfinite().all()


@pytest.mark.parametrize("gate", ["none", "channel", "full"])
def test_gradients_against_differences(gate):
    """Directional derivatives of a loss in binary64 (the formula's gradients,
    checked to 1e-7), and the kernels' fp32 gradients along the same
    directions, within the error bounds above."""
    rows, d = 6, 40
    y, r, pre, w, ga = inputs(rows, d, torch.float32, torch.float32, gate, True, seed=5)
    g = torch.Generator().manual_seed(9)
    cz, ch = torch.randn(rows, d, generator=g), torch.randn(rows, d, generator=g)
    alpha = 0.75
    leaves = {"y": y, "r": r, "pre": pre, "post": w, "gate": ga}

    def loss(v):
        h, z, _ = ref.block_norm(v["y"], v["r"], v["pre"], v["post"], v["gate"], alpha, EPS)
        return float((h * ch.double()).sum() + (z * cz.double()).sum())

    h, z, st = rca.block_norm(gpu(y), gpu(r), gpu(pre), post_weight=gpu(w), gate=gpu(ga), residual_scale=alpha,
                              eps=EPS, stats=True)
    dy, dr, dpre, dpost, dgate = rca.block_norm_backward(gpu(cz), gpu(ch), h, st, gpu(y), gpu(pre),
                                                         post_weight=gpu(w), gate=gpu(ga), residual_scale=alpha)
    hr, _, sr = ref.block_norm(y, r, pre, w, ga, alpha, EPS)
    formula = ref.block_norm_backward(cz, ch, hr, sr, y, pre, w, ga, alpha)
    names = {"y": ("dy", dy), "r": ("dr", dr), "pre": ("dpre", dpre), "post": ("dpost", dpost), "gate": ("dgate", dgate)}
    for leaf, (name, got) in names.items():
        if leaves[leaf] is None:
            continue
        value, mag = formula[name]
        for seed in range(3):
            step = torch.randn(leaves[leaf].shape, generator=torch.Generator().manual_seed(seed)).double()
            at = lambda s: loss({**leaves, leaf: leaves[leaf].double() + s * 1e-5 * step})  # noqa: E731
            slope = (at(1) - at(-1)) / 2e-5
            assert abs(slope - float((value * step).sum())) <= 1e-7 * float((mag * step.abs()).sum()), (name, seed)
            along = float((got.cpu().double() * step).sum())
            assert abs(slope - along) <= (1e-7 + (rows + 400) * ref.U32) * float((mag * step.abs()).sum()), (name, seed)


def test_repeats_bit_for_bit():
    y, r, pre, w, ga = (gpu(t) for t in inputs(3000, 1024, torch.bfloat16, torch.bfloat16, "channel", True))
    h, z, st = rca.block_norm(y, r, pre, post_weight=w, gate=ga, stats=True)
    run = lambda: rca.block_norm_backward(z, r, h, st, y, pre, post_weight=w, gate=ga)  # noqa: E731
    first = run()
    for _ in range(3):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


def test_more_than_2_to_32_elements():
    rows, d = 131200, 32768                            # 4.3e9 elements
    print("case large", flush=True)
    y = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)
    y[-5:] = torch.randn(5, d, device=DEV).to(torch.bfloat16)
    r = torch.zeros_like(y)
    r[-5:] = torch.randn(5, d, device=DEV).to(torch.bfloat16)
    pre = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    h, z, st = rca.block_norm(y, r, pre, post_weight=pre, stats=True)
    hs, zs, ss = rca.block_norm(y[-5:], r[-5:], pre, post_weight=pre, stats=True)
    assert torch.equal(h[-5:], hs) and torch.equal(z[-5:], zs) and torch.equal(st[:, -5:], ss)
    dy, dr, *_ = rca.block_norm_backward(z, h, h, st, y, pre, post_weight=pre)
    dys, drs, *_ = rca.block_norm_backward(zs, hs, hs, ss.contiguous(), y[-5:], pre, post_weight=pre)
    assert torch.equal(dy[-5:], dys) and torch.equal(dr[-5:], drs)
