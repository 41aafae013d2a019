"""The layers' buffers hold all that they allocate (CPU)."""
import pytest
import torch

import fp8_block_scaled_bias_amd as M
from fp8_block_scaled_bias_amd import layer as ML


@pytest.mark.parametrize("cls", [ML.Buffers, ML.Int8Buffers])
def test_nothing_is_allocated_twice(cls, monkeypatch):
    made, empty = [], torch.empty

    def counting(*a, **kw):
        made.append(empty(*a, **kw))
        return made[-1]

    monkeypatch.setattr(torch, "empty", counting)
    b = cls(M.LayerShape(256, 16, 4, 2, 4, 128), 24, "cpu")
    held = [t for t in vars(b).values() if isinstance(t, torch.Tensor)]
    assert sum(t.nbytes for t in made) == sum(t.nbytes for t in held)
    assert b.xq.shape == (24, 256) and b.hq.shape == (b.R, 128)
    assert b.hq.dtype == (torch.uint8 if cls is ML.Buffers else torch.int8)
