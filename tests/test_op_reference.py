"""The binary64 statements that the operators are compared with, pinned on the
CPU: gradients against central differences, the grouped product against single
products, and clipping against its definition."""
import pytest
import torch

from tests import op_reference as ref


def rn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("gate", ["none", "channel", "full"])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_gradients_against_differences(gate, post):
    rows, d, alpha, eps = 4, 9, 0.6, 1e-6
    v = {"y": rn(rows, d, seed=1), "r": rn(rows, d, seed=2), "pre": rn(d, seed=3), "post": rn(d, seed=4) if post else None,
         "gate": None if gate == "none" else rn(d, seed=5) if gate == "channel" else rn(rows, d, seed=5)}
    cz, ch = rn(rows, d, seed=6), rn(rows, d, seed=7)

    def loss(v):
        h, z, _ = ref.block_norm(v["y"], v["r"], v["pre"], v["post"], v["gate"], alpha, eps)
        return float((h * ch).sum() + (z * cz).sum())

    h, _, st = ref.block_norm(v["y"], v["r"], v["pre"], v["post"], v["gate"], alpha, eps)
    grads = ref.block_norm_backward(cz, ch, h, st, v["y"], v["pre"], v["post"], v["gate"], alpha)
    for leaf, name in (("y", "dy"), ("r", "dr"), ("pre", "dpre"), ("post", "dpost"), ("gate", "dgate")):
        if v[leaf] is None:
            assert name not in grads
            continue
        value, mag = grads[name]
        assert (value.abs() <= mag * (1 + 1e-12) + 1e-300).all()
        for seed in range(3):
            step = rn(*v[leaf].shape, seed=20 + seed)
            slope = (loss({**v, leaf: v[leaf] + 1e-5 * step}) - loss({**v, leaf: v[leaf] - 1e-5 * step})) / 2e-5
            assert abs(slope - float((value * step).sum())) <= 1e-8 * float((mag * step.abs()).sum())


def test_grouped_products_row_by_row():
    off, rows = [1, 3, 3, 6], 8
    packed, w = ref.random_packed(3, 8, 32, 1)
    x, dy = rn(rows, 32, seed=1), rn(rows, 8, seed=2)
    y, _ = ref.grouped(x, w, off)
    dx, _ = ref.grouped_dx(dy, w, off)
    dw, _ = ref.grouped_dw(dy, x, off)
    expert = [None, 0, 0, 2, 2, 2, None, None]
    want = torch.zeros_like(dw)
    for i, e in enumerate(expert):
        if e is None:
            assert not y[i].any() and not dx[i].any()
            continue
        assert torch.allclose(y[i], w[e] @ x[i], rtol=1e-13) and torch.allclose(dx[i], w[e].T @ dy[i], rtol=1e-13)
        want[e] += torch.outer(dy[i], x[i])
    assert torch.allclose(dw, want, rtol=1e-12, atol=1e-13) and not dw[1].any()


def test_clip():
    grads = [rn(7, seed=1), rn(2, 3, seed=2)]
    norm, factor = ref.clip(grads, -2.0, 0.1, 0.0)
    whole = torch.cat([g.reshape(-1) for g in grads]) * -2.0
    assert abs(norm - float(whole.norm())) < 1e-12
    scaled = torch.cat([g.reshape(-1) for g in grads]) * factor
    assert abs(float(scaled.norm()) - 0.1) < 1e-12
    assert ref.clip(grads, 0.5, 1e9, 1e-6)[1] == 0.5
