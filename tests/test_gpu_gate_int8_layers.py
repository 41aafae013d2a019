"""The layers that use the gate and the int8 products: MoELayer with a Gate
(forward and backward), Int8MoELayer, and their graphs, against the oracles."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
import synth
from gpu_common import bf16_dev, bf16_values_host, dev, host, log, rel_l2
from oracle import backward as OB
from oracle import gate as OG
from oracle import int8 as OI
from oracle import layer as OL
from oracle.formats import bf16_round, bf16_value_from_bits
from oracle.permute import permute
from test_gpu_layer import oracle_weights, shape_of

pytestmark = pytest.mark.gpu

GATES = [M.Gate(M.SCORE_SOFTMAX, False, 1, True, 1.0), M.Gate(M.SCORE_SOFTMAX, True, 2, False, 16.0),
         M.Gate(M.SCORE_SIGMOID, True, 2, True, 2.5)]


def build(cls, cfg, gate):
    C, b = synth.gen_centroids(cfg), synth.gen_bias(cfg)
    layer = cls.from_fp32_experts(
        shape_of(cfg), torch.from_numpy(C).cuda(), torch.from_numpy(b).cuda(),
        synth.gen_all_expert_weights(cfg, "gu"), synth.gen_all_expert_weights(cfg, "dn"), gate=gate)
    return layer, C, b


def gate_oracle(layer, cfg, b, logits):
    """The oracle's routing of the GPU's own fp32 logits (which are compared
    with the exact ones apart)."""
    g = layer.gate
    r = OG.gate(logits, b if g.use_bias else None, g.score, cfg.n_group, cfg.topk_group, g.group_top,
                cfg.k, g.renormalize, g.scale)
    r["w32"] = r["w"].astype(np.float32)
    return r


def check_logits(logits, x, C):
    xv, Cv = bf16_value_from_bits(x).astype(np.float64), C.astype(np.float64)
    size = np.abs(xv) @ np.abs(Cv).T
    assert (np.abs(logits - xv @ Cv.T) <= 64 * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("name", ["tiny", "mid"])
@pytest.mark.parametrize("gate", GATES, ids=["softmax", "softmax-raw", "sigmoid"])
def test_layer_with_gate(name, gate, monkeypatch):
    cfg = synth.CONFIGS[name]
    layer, C, b = build(M.MoELayer, cfg, gate)
    x, dy = synth.gen_x(cfg), synth.gen_dy(cfg)
    log(f"[gate layer] {name} {gate}")
    y = bf16_values_host(layer.forward(bf16_dev(x)))
    bufs = layer.buffers(cfg.T)
    logits = host(bufs.logits).astype(np.float64)
    check_logits(logits, x, C)
    r = gate_oracle(layer, cfg, b, logits)
    assert np.array_equal(host(bufs.topk_idx), r["idx"]) and np.array_equal(host(bufs.counts), r["counts"])
    monkeypatch.setattr(OL, "route", lambda *a: r)
    wts = oracle_weights(cfg)
    ref = OL.layer(x, C, b, wts, cfg.n_group, cfg.topk_group, cfg.k, cfg.I)
    assert rel_l2(y, ref["y"]) <= 2e-3            # the layer's bar with moe_route
    bb = layer.backward(bf16_dev(dy), bf16_dev(x))
    eb = OB.expert_backward(dy, ref, wts, x, cfg.T, cfg.k, cfg.I, cfg.n_shared)
    assert rel_l2(host(bb.dw), eb["dw"]) <= 5e-3
    dl = OG.gate_backward(logits, gate.score, gate.renormalize, gate.scale, r["idx"], eb["dw"])
    xv = bf16_value_from_bits(x).astype(np.float64)
    dx = bf16_round(eb["dx"] + dl @ C.astype(np.float64))
    assert rel_l2(host(bb.dlogit), dl) <= 5e-3
    assert rel_l2(bf16_values_host(bb.dx_total), dx) <= 5e-3
    assert rel_l2(host(bb.dC), dl.T @ xv) <= 5e-3
    with pytest.raises(ValueError, match="Gate"):
        layer.forward(bf16_dev(x), seq_len=16)


def int8_reference(layer, cfg, x, r):
    """The int8 layer in whole numbers and FP64, rounded where it stores."""
    xv = bf16_value_from_bits(x).astype(np.float32)
    xq, xs = OI.quant_rows(xv)
    offsets, perm_src, inv_perm = permute(r["idx"], cfg.E, cfg.n_shared)
    w = [OI.quant_rows(np.stack([synth.gen_expert_weight(cfg, n, e) for e in range(cfg.G)]))
         for n in ("gu", "dn")]
    for (q, s), (gq, gs) in zip(w, ((layer.w_gu, layer.w_gu_s), (layer.w_dn, layer.w_dn_s))):
        assert np.array_equal(host(gq), q) and np.array_equal(host(gs), s)
    h = bf16_round(OI.swiglu(OI.products(xq, xs, *w[0], offsets, np.asarray(perm_src))))
    hq, hs = OI.quant_rows(h.astype(np.float32))
    D = bf16_round(OI.products(hq, hs, *w[1], offsets))
    R = cfg.T * cfg.k
    rows = np.asarray(inv_perm)[:R].reshape(cfg.T, cfg.k)
    y = (D[rows] * r["w32"].astype(np.float64)[:, :, None]).sum(axis=1)
    return bf16_round(y + D[R:R + cfg.T]) if cfg.n_shared else bf16_round(y)


@pytest.mark.parametrize("name,T", [("tiny", 64), ("mid", 200), ("mid", 3)])
@pytest.mark.parametrize("gate", [GATES[1], GATES[2]], ids=["softmax", "sigmoid"])
def test_int8_layer(name, T, gate):
    cfg = synth.CONFIGS[name].with_(T=T)
    layer, C, b = build(M.Int8MoELayer, cfg, gate)
    x = synth.gen_x(cfg)
    log(f"[int8 layer] {name} T={T} {gate}")
    y = bf16_values_host(layer.forward(bf16_dev(x)))
    bufs = layer.buffers(T)
    r = gate_oracle(layer, cfg, b, host(bufs.logits).astype(np.float64))
    assert np.array_equal(host(bufs.topk_idx), r["idx"])
    # both round at the same places; an element of h next to a border of bf16
    # may round the other way (2^-8 of itself) and then change its code by one
    assert rel_l2(y, int8_reference(layer, cfg, x, r)) <= 2e-3
    with pytest.raises(NotImplementedError):
        layer.backward(bf16_dev(x), bf16_dev(x))


def test_int8_layer_without_gate_graph_and_empty():
    """moe_route in front, captured and replayed; an empty batch; new weights."""
    cfg = synth.CONFIGS["mid"]
    layer, C, b = build(M.Int8MoELayer, cfg, None)
    xs = [synth.gen_x(cfg, seed=s) for s in (21, 22)]
    eager = [bf16_values_host(layer.forward(bf16_dev(v))).copy() for v in xs]
    r = dict(idx=host(layer.buffers(cfg.T).topk_idx), w32=host(layer.buffers(cfg.T).topk_w))
    assert rel_l2(eager[1], int8_reference(layer, cfg, xs[1], r)) <= 2e-3
    x_in = bf16_dev(xs[0])
    g = layer.capture(x_in)
    for rep in range(3):
        for i, v in enumerate(xs):
            x_in.copy_(bf16_dev(v))
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(bf16_values_host(layer.buffers(cfg.T).y), eager[i]), (rep, i)
        layer.forward(bf16_dev(xs[0]))
    assert layer.forward(bf16_dev(np.zeros((0, cfg.H), np.uint16))).shape == (0, cfg.H)
    assert (host(layer.buffers(0).counts) == 0).all()
    gu = torch.from_numpy(np.stack([synth.gen_expert_weight(cfg, "gu", e) for e in range(cfg.G)])).cuda()
    dn = torch.from_numpy(np.stack([synth.gen_expert_weight(cfg, "dn", e) for e in range(cfg.G)])).cuda()
    old = host(layer.w_gu_s).copy()
    layer.requantize_from_fp32(2 * gu, dn)
    assert np.array_equal(host(layer.w_gu_s), 2 * old)


def test_gate_layer_empty_batch():
    cfg = synth.CONFIGS["tiny"]
    layer, C, b = build(M.MoELayer, cfg, GATES[0])
    e = bf16_dev(np.zeros((0, cfg.H), np.uint16))
    assert layer.forward(e).shape == (0, cfg.H)
    bb = layer.backward(e, e)
    assert (host(bb.dC) == 0).all() and (host(bb.dW_gu) == 0).all()


def test_bindings_refuse_wrong_tensors():
    x = torch.zeros((4, 64), device="cuda")
    i = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w, c = torch.zeros((4, 2), device="cuda"), torch.zeros(64, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        M.moe_gate(x.half(), 4, 64, None, 0, 1, 1, 1, 2, 1, 1.0, i, w, c)
    with pytest.raises(TypeError):
        M.moe_gate(x, 4, 64, None, 0, 1, 1, 1, 2, 1, 1.0, i.long(), w, c)
    with pytest.raises(TypeError):
        M.moe_gate_backward(x, 4, 64, 0, 2, 1, 1.0, i, w, x.bfloat16())
    with pytest.raises(ValueError):
        M.moe_gate(x.cpu(), 4, 64, None, 0, 1, 1, 1, 2, 1, 1.0, i, w, c)
    with pytest.raises(ValueError):
        M.moe_gate(torch.zeros((64, 4), device="cuda").t(), 4, 64, None, 0, 1, 1, 1, 2, 1, 1.0, i, w, c)
    with pytest.raises(TypeError):
        M.int8_quant_rows(x, 4, 64, 64, x.to(torch.int8), w)
    q, s = x.to(torch.int8), x[:, 0].contiguous()
    with pytest.raises(TypeError):
        M.grouped_int8_gemm(q, s, None, q.to(torch.uint8)[None], s[None], c[:2], 1, 4, 4, 64, x.bfloat16())
