"""Clipping without a limit: max_norm = infinity gives the norm and applies the scale, for any gradients."""
import math

import pytest
import torch

import reduction_codec_amd as rca

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("scale", [1.0, 0.5])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 3e38])
def test_no_limit_scales_whatever_the_norm_is(bad, scale):
    """3e38 twice: finite values whose norm is beyond binary32."""
    for dtype in (torch.float32, torch.bfloat16):
        print(f"case no limit {bad} {scale} {dtype}", flush=True)
        grads = [torch.linspace(-4, 4, 9001, device=DEV).to(dtype), torch.ones(70, device=DEV, dtype=dtype)]
        grads[1][3] = grads[1][4] = bad
        want = [(g.float() * scale).to(dtype) for g in grads]
        outs = [torch.full_like(g, 7.0) for g in grads]
        norm = rca.grad_norm_clip(grads, math.inf, scale=scale, out=outs)
        assert not math.isfinite(float(norm)) or scale < 1
        rca.grad_norm_clip(grads, math.inf, scale=scale)
        for w, o, g in zip(want, outs, grads):
            assert torch.equal(o.nan_to_num(nan=123.0), w.nan_to_num(nan=123.0)) and torch.equal(o.isnan(), w.isnan())
            assert torch.equal(g.nan_to_num(nan=123.0), w.nan_to_num(nan=123.0)) and torch.equal(g.isnan(), w.isnan())
