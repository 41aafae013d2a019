"""A layer with a Gate captured as HIP graphs, forward and backward, replayed
between eager calls; two gates at once on two streams."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
import synth
from gpu_common import bf16_dev, dev, host
from oracle import gate as OG
from test_gpu_gate import check
from test_gpu_gate_int8_layers import GATES, build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", GATES, ids=["softmax", "softmax-raw", "sigmoid"])
def test_forward_and_backward_graphs(gate):
    cfg = synth.CONFIGS["mid"]
    layer, _, _ = build(M.MoELayer, cfg, gate)
    xs = [synth.gen_x(cfg, seed=s) for s in (31, 32)]
    dy = bf16_dev(synth.gen_dy(cfg))
    b, bb = layer.buffers(cfg.T), layer.backward_buffers(cfg.T)
    outs = lambda: [host(t.view(torch.uint8)).copy() for t in (b.y, b.topk_idx, b.topk_w, bb.dx_total, bb.dC, bb.dw)]
    x_in = bf16_dev(xs[0])
    eager = []
    for v in xs:
        x_in.copy_(bf16_dev(v))
        layer.forward(x_in)
        layer.backward(dy, x_in)
        eager.append(outs())
    fwd = layer.capture(x_in)
    bwd = torch.cuda.CUDAGraph()
    with torch.cuda.graph(bwd):
        layer.backward(dy, x_in, stream=torch.cuda.current_stream())
    for rep in range(3):
        for i, v in enumerate(xs):
            x_in.copy_(bf16_dev(v))
            fwd.replay()
            bwd.replay()
            torch.cuda.synchronize()
            for got, want in zip(outs(), eager[i]):
                assert np.array_equal(got, want), (rep, i)
        layer.forward(x_in)
        layer.backward(dy, x_in)
        torch.cuda.synchronize()


def test_two_gates_at_once():
    rng = np.random.default_rng(5)
    E, k = 256, 8
    bias = rng.uniform(-0.01, 0.01, E).astype(np.float32)
    jobs = []
    for T, stream in ((4001, torch.cuda.Stream()), (130, torch.cuda.Stream())):
        l = rng.standard_normal((T, E)).astype(np.float32)
        jobs.append((l, dev(l), stream, torch.empty((T, k), dtype=torch.int32, device="cuda"),
                     torch.empty((T, k), device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda")))
    b = dev(bias)
    args = (OG.SIGMOID, 8, 4, 2, k, 1, 2.5)
    torch.cuda.synchronize()
    for _ in range(6):
        for l, logits, stream, idx, w, counts in jobs:
            M.moe_gate(logits, l.shape[0], E, b, *args, idx, w, counts, stream)
    torch.cuda.synchronize()
    for l, _, _, idx, w, counts in jobs:
        check(l.astype(np.float64), bias, (host(idx), host(w), host(counts), None), args, str(l.shape))
