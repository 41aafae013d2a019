"""Inputs that the layers refuse before they look for a GPU or a stream (CPU):
the kernels take a tensor's sizes from the layer's shape, and would read or write
past one of another."""
import pytest
import torch

import fp8_block_scaled_bias_amd as M

S = M.LayerShape(256, 16, 4, 2, 4, 128)
T = 24


@pytest.fixture(params=[M.MoELayer, M.Int8MoELayer, M.Bf16MoELayer])
def layer(request):
    cls = request.param
    return cls(S, torch.zeros(S.E, S.H), torch.zeros(S.E), *cls.empty_weights(S, "cpu"))


def rows(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("x", [rows(T, S.H // 2), rows(T, 2 * S.H), rows(T * S.H), rows(T, 1, S.H)], ids=lambda x: str(list(x.shape)))
def test_other_shapes(layer, x):
    with pytest.raises(ValueError, match="H"):
        layer.forward(x)
    if not isinstance(layer, M.Int8MoELayer):
        for dy, v in ((x, rows(T, S.H)), (rows(T, S.H), x)):
            with pytest.raises(ValueError, match="H"):
                layer.backward(dy, v)


def test_other_buffers(layer):
    x = rows(T, S.H)
    with pytest.raises(ValueError, match="in buffers of"):
        layer.forward(x, layer.buffers(T - 1))
    if not isinstance(layer, M.Int8MoELayer):
        with pytest.raises(ValueError, match="in buffers of"):
            layer.backward(x, x, layer.buffers(T - 1))
        with pytest.raises(ValueError, match="in buffers of"):
            layer.backward(x, rows(T - 1, S.H))


def test_other_types_and_places(layer, monkeypatch):
    """(what stands in for a GPU's number is the CPU's, so that the type is what
    is looked at)"""
    with pytest.raises(ValueError, match="GPU"):
        monkeypatch.setattr(M.layer.L, "_device", lambda: 0)
        layer.forward(rows(T, S.H))
    monkeypatch.setattr(M.layer.L, "_device", lambda: -1)
    monkeypatch.setattr(M.layer.L, "_dev", lambda t: None)
    with pytest.raises(TypeError, match="bfloat16"):
        layer.forward(rows(T, S.H).float())
    if not isinstance(layer, M.Int8MoELayer):
        with pytest.raises(TypeError, match="bfloat16"):
            layer.backward(rows(T, S.H).float(), rows(T, S.H))
        with pytest.raises(ValueError, match="tokens"):
            layer.backward(rows(T, S.H), rows(T, S.H), bwd=layer.backward_buffers(T + 1))


def test_new_weights(layer):
    gu, dn = torch.zeros(S.G, 2 * S.I, S.H), torch.zeros(S.G, S.H, S.I)
    before = layer.w_gu.clone()
    for a, b in ((gu[:1], dn), (gu, dn[:1]), (gu[:, :1], dn), (gu, dn.transpose(1, 2).contiguous()), (gu[0], dn)):
        with pytest.raises(ValueError, match="weights"):
            layer.requantize_from_fp32(a, b)
    for a, b in ((gu.double(), dn), (gu, dn.bfloat16())):
        with pytest.raises(TypeError, match="float32"):
            layer.requantize_from_fp32(a, b)
    assert torch.equal(layer.w_gu.view(torch.uint8), before.view(torch.uint8))
