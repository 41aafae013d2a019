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


def test_balance_buffers_of_a_seq_len_stay():
    """A captured graph writes the buffers of its own seq_len after forwards of
    another one: they are not freed, nor is that one's given out in their place."""
    b = ML.Buffers(M.LayerShape(256, 16, 4, 2, 4, 128), 24, "cpu")
    names = ("scores", "score_sums", "seq_f", "seq_p", "seq_loss", "seq_ws")
    first = [getattr(b.balance(8), n) for n in names]
    assert b.seq_f.shape == (3, 16)
    other = [getattr(b.balance(24), n) for n in names]
    assert b.seq_f.shape == (1, 16) and all(o is not t for o, t in zip(other, first))
    assert all(getattr(b.balance(8), n) is t for n, t in zip(names, first))
