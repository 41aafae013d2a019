"""A layer with a Gate refuses what it does not do before it launches anything."""
import dataclasses

import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
import synth
from gpu_common import bf16_dev, host
from test_gpu_gate_int8_layers import GATES, build

pytestmark = pytest.mark.gpu


def marked(obj):
    """Fill an object's device tensors with a mark; a check that it is still there."""
    mine = {k: t for k, t in vars(obj).items() if isinstance(t, torch.Tensor)}
    for t in mine.values():
        t.view(-1).view(torch.uint8).fill_(0x5A)

    def unchanged():
        torch.cuda.synchronize()
        return [k for k, t in mine.items() if not (host(t.view(-1).view(torch.uint8)) == 0x5A).all()]
    return unchanged


def test_balance_term_refused_first():
    cfg = synth.CONFIGS["tiny"]
    layer, _, _ = build(M.MoELayer, cfg, GATES[0])
    x = bf16_dev(synth.gen_x(cfg))
    check = marked(layer.buffers(cfg.T))
    with pytest.raises(ValueError, match="Gate"):
        layer.forward(x, seq_len=16)
    assert check() == []
    layer.forward(x)
    check = marked(layer.backward_buffers(cfg.T))
    with pytest.raises(ValueError, match="Gate"):
        layer.backward(x, x, seq_len=16)
    assert check() == []


@pytest.mark.parametrize("cls", [M.MoELayer, M.Int8MoELayer])
def test_experts_not_a_multiple_of_16(cls):
    """Forward for any number of experts; the backward refuses before it starts."""
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], E=12, n_group=4, topk_group=2, k=3)
    layer, _, _ = build(cls, cfg, GATES[1])
    x = bf16_dev(synth.gen_x(cfg))
    y = layer.forward(x)
    assert np.isfinite(host(y.float())).all()
    assert host(layer.buffers(cfg.T).counts).sum() == cfg.T * cfg.k
    if cls is M.MoELayer:
        check = marked(layer.backward_buffers(cfg.T))
        with pytest.raises(ValueError, match="E is 12"):
            layer.backward(x, x)
        assert check() == []
