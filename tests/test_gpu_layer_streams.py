"""Layers and blocks called with a stream that is not the current one, which is
busy: what a first call allocates and fills (the unit weights of the backward's
gather, the buffers) is in the order of the stream that was given."""
import gc

import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
import synth
from bf16_cases import up, values
from gpu_common import dev, host
from test_gpu_bf16_layer import bf16_layer
from test_gpu_gate_int8_layers import build
from test_gpu_norm import EPS

pytestmark = pytest.mark.gpu

CFG = synth.CONFIGS["mid"]


def busy():
    """Work of some 200 ms on the current stream."""
    torch.cuda._sleep(5_000_000_000)


def poison():
    """Small blocks that are handed out next hold NaN."""
    gc.collect()
    torch.cuda.empty_cache()
    t = [torch.full((4096,), float("nan"), device="cuda") for _ in range(2000)]
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("what", ["layer", "block"])
def test_first_calls_on_another_stream(kind, what):
    make = (lambda: bf16_layer(CFG)[0]) if kind == "bf16" else (lambda: build(M.MoELayer, CFG, None)[0])
    rng = np.random.default_rng(1)
    x, dy = up(values(rng, (CFG.T, CFG.H))), up(values(rng, (CFG.T, CFG.H), 0.02))
    w = dev((1 + 0.1 * rng.standard_normal(CFG.H)).astype(np.float32))

    def run(st):
        layer = make()
        torch.cuda.synchronize()
        poison()
        if st is not None:
            busy()
        if what == "layer":
            y = layer.forward(x, stream=st)
            bb = layer.backward(dy, x, stream=st)
            out = (y, bb.dx_total)
        else:
            block = M.MoEBlock(layer, w, EPS)
            y = block.forward(x, stream=st)
            f, bb = block.backward(dy, x, stream=st)
            out = (y, f.dx)
        (st or torch.cuda.current_stream()).synchronize()
        assert st is None or not torch.cuda.current_stream().query(), "the current stream is not busy any more"
        with torch.cuda.stream(st):
            return [host(t.float()).copy() for t in (*out, bb.dC, bb.dW_dn)]
    want = run(None)
    st = torch.cuda.Stream()
    for g, v in zip(run(st), want):
        assert np.array_equal(g, v)


def test_positional_stream():
    layer = bf16_layer(CFG)[0]
    x = up(values(np.random.default_rng(1), (CFG.T, CFG.H)))
    want = host(layer.forward(x).float()).copy()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = layer.forward(x, None, st)
    st.synchronize()
    assert np.array_equal(host(y.float()), want)
    assert torch.cuda.current_stream() != st
