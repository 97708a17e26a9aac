"""The serving example refuses what it cannot share or serve before it touches a GPU, and runs without steps."""
import pytest
import torch

from examples import serving_block


@pytest.mark.parametrize("bad", [{"ranks": 3}, {"ranks": 0}, {"heads": 16, "kv_heads": 4, "ranks": 8}, {"prompts": ()},
                                 {"prompts": (5, 0)}], ids=str)
def test_refusals(bad):
    with pytest.raises(ValueError):
        serving_block.serve(steps=1, **bad)


@pytest.mark.gpu
def test_without_steps_and_with_a_prompt_that_fills_its_pages():
    out = serving_block.serve(steps=0, prompts=(64, 3), ranks=1, width=256, heads=4, kv_heads=2, d=64, page=32, log=lambda s: None)
    assert len(out) == 1 and all(t.shape == (67, 256) and torch.isfinite(t.float()).all() for t in out[0])
