"""Clipping into outputs that lie right behind their gradients in one buffer."""
import pytest
import torch

import reduction_codec_amd as rca

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("lead", range(1, 8))
def test_wider_output_behind_its_gradient_is_written(lead, dtype):
    """A gradient `lead` elements past a 16-byte boundary and its fp32 output
    `lead` elements after it: counted back by `lead` elements of their types,
    both lie at the boundary.  Under the limit the factor is one, and every
    value has to arrive all the same."""
    for n in range(1, lead + 1):
        print(f"case neighbours lead={lead} n={n} {dtype}", flush=True)
        buf = torch.full((256,), 0x55, dtype=torch.uint8, device=DEV)
        grad = buf[2 * lead:2 * lead + 2 * n].view(dtype)
        out = buf[4 * lead:4 * lead + 4 * n].view(torch.float32)
        grad.copy_(torch.arange(1, n + 1, device=DEV))
        norm = rca.grad_norm_clip([grad], 1e9, out=[out])
        assert torch.equal(out, torch.arange(1, n + 1, device=DEV, dtype=torch.float32))
        assert torch.equal(grad.float(), out) and float(norm) > 0
        assert (buf[4 * lead + 4 * n:] == 0x55).all() and (buf[:2 * lead] == 0x55).all()
