"""Bf16MoELayer and MoEBlock (a layer between its norms): forward and backward
against FP64 compositions, as graphs, in the forms that the layers have."""
import dataclasses

import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
import synth
from bf16_cases import U, check, up, values
from gpu_common import bf16_dev, bf16_values_host, dev, host, log, rel_l2
from oracle import backward as OBW
from oracle import bf16 as OB
from oracle import gate as OG
from oracle import norm as ON
from oracle.formats import bf16_bits_from_value, bf16_round, bf16_value_from_bits
from oracle.permute import permute
from test_gpu_gate_int8_layers import GATES, build
from test_gpu_layer import shape_of
from test_gpu_norm import EPS, check_as, check_e4m3, get, stream

pytestmark = pytest.mark.gpu


def bf16_layer(cfg, gate=None, act=M.ACT_SILU):
    C, b = synth.gen_centroids(cfg), synth.gen_bias(cfg)
    layer = M.Bf16MoELayer.from_fp32_experts(
        shape_of(cfg), dev(C), dev(b), synth.gen_all_expert_weights(cfg, "gu"),
        synth.gen_all_expert_weights(cfg, "dn"), gate=gate, act=act)
    w = [bf16_round(np.stack([synth.gen_expert_weight(cfg, n, e) for e in range(cfg.G)])).astype(np.float64)
         for n in ("gu", "dn")]
    return layer, C, w


class Reference:
    """The bf16 layer in FP64 for the GPU's routing, rounded where it stores."""

    def __init__(self, cfg, C, w, act, x, bufs):
        self.cfg, self.C, self.w, self.act, self.x = cfg, C.astype(np.float64), w, act, x
        self.idx, self.gate = host(bufs.topk_idx), host(bufs.topk_w).astype(np.float64)
        self.offs, src, inv = permute(self.idx, cfg.E, cfg.n_shared)
        self.src, R = np.asarray(src), cfg.T * cfg.k
        self.inv = np.asarray(inv)[:R]
        self.GU = OB.products(x, w[0], self.offs, self.src)[0]
        self.h = bf16_round(OB.glu(self.GU, act))
        self.D = bf16_round(OB.products(self.h, w[1], self.offs)[0])

    def rows(self, shared_w=None):
        sw = np.ones(self.cfg.T) if shared_w is None else shared_w
        return ON.gather(self.D, self.inv, self.gate, sw if self.cfg.n_shared else None, self.cfg.T, self.cfg.k)

    def y(self):
        rows, w = self.rows()
        return bf16_round((rows * w[:, :, None]).sum(axis=1))

    def backward(self, dD, dw, dlogit):
        """From the gradient of the experts' rows; dlogit(dw): the gate's."""
        cfg, x = self.cfg, self.x
        R = cfg.T * cfg.k
        dh = OB.dgrad(dD, self.w[1], self.offs)[0]
        dgu = bf16_round(OB.glu_backward(bf16_round(self.GU), dh, self.act))
        dX = bf16_round(OB.dgrad(dgu, self.w[0], self.offs)[0])
        dx = dX[self.inv].reshape(cfg.T, cfg.k, -1).sum(axis=1)
        if cfg.n_shared:
            dx = dx + dX[R:]
        dl = dlogit(dw)
        return dict(dW_dn=OB.wgrad(dD, self.h, self.offs)[0], dW_gu=OB.wgrad(dgu, x, self.offs, self.src)[0],
                    dC=dl.T @ x, dx_total=bf16_round(bf16_round(dx) + dl @ self.C))

    def dlogit(self, layer, bufs):
        """Dense gradient of the router's logits for dw [T, k]."""
        cfg = self.cfg

        def route(dw):
            r = OBW.router_backward(bf16_bits_from_value(self.x), self.C, self.idx, dw)
            dl = np.zeros((cfg.T, cfg.E))
            np.put_along_axis(dl, self.idx.astype(np.int64), r["dlogit"], axis=1)
            return dl

        def gate(dw):
            g = layer.gate
            return OG.gate_backward(host(bufs.logits).astype(np.float64), g.score, g.renormalize, g.scale, self.idx, dw)
        return gate if layer.gate is not None else route


def compare(bb, ref):
    for name, want in ref.items():
        t = getattr(bb, name)
        got = get(t) if t.dtype == torch.bfloat16 else host(t)
        err = rel_l2(got, want)
        log(f"[bf16 layer] {name} rel L2 {err:.2e}")
        assert err <= 5e-3, name


@pytest.mark.parametrize("name,T", [("tiny", 64), ("mid", 200), ("mid", 1)])
@pytest.mark.parametrize("gate,act", [(None, M.ACT_SILU), (GATES[1], M.ACT_GELU)], ids=["route", "gate"])
def test_layer(name, T, gate, act):
    cfg = synth.CONFIGS[name].with_(T=T)
    layer, C, w = bf16_layer(cfg, gate, act)
    x, dy = synth.gen_x(cfg), synth.gen_dy(cfg)
    xv, dyv = (bf16_value_from_bits(v).astype(np.float64) for v in (x, dy))
    b = layer.buffers(T)
    for keep in (True, False):   # (the second backward forms gate and up again)
        log(f"[bf16 layer] {name} T={T} keep={keep}")
        y = bf16_values_host(layer.forward(bf16_dev(x), keep_gu=keep))
        ref = Reference(cfg, C, w, act, xv, b)
        assert rel_l2(y, ref.y()) <= 2e-3
        bb = layer.backward(bf16_dev(dy), bf16_dev(x))
        rows, ws = ref.rows()
        cb = OBW.combine_backward(dyv, ref.D, ref.inv, ref.gate, T, cfg.k, cfg.n_shared)
        assert rel_l2(host(bb.dw), cb["dw"]) <= 5e-3
        compare(bb, ref.backward(cb["dD"].astype(np.float64), cb["dw"], ref.dlogit(layer, b)))


def test_layer_against_differences():
    """The gradient of <dy, y> along random directions of x, against the
    layer's own forward in FP64 with its routing held."""
    cfg = synth.CONFIGS["tiny"]
    layer, C, w = bf16_layer(cfg)
    x, dy = synth.gen_x(cfg), synth.gen_dy(cfg)
    xv, dyv = (bf16_value_from_bits(v).astype(np.float64) for v in (x, dy))
    layer.forward(bf16_dev(x), keep_gu=True)
    bb = layer.backward(bf16_dev(dy), bf16_dev(x))
    idx = host(layer.buffers(cfg.T).topk_idx).astype(np.int64)
    offs, src, inv = permute(idx, cfg.E, cfg.n_shared)
    src, inv = np.asarray(src), np.asarray(inv)[:cfg.T * cfg.k]

    def loss(x):
        s = 1 / (1 + np.exp(-np.take_along_axis(x @ C.astype(np.float64).T, idx, 1)))
        D = OB.products(OB.glu(OB.products(x, w[0], offs, src)[0], OB.SILU), w[1], offs)[0]
        rows, ws = ON.gather(D, inv, s / s.sum(axis=1, keepdims=True), np.ones(cfg.T), cfg.T, cfg.k)
        return (dyv * (rows * ws[:, :, None]).sum(axis=1)).sum()
    rng = np.random.default_rng(1)
    dx, h = bf16_values_host(bb.dx_total).astype(np.float64), 1e-4
    for _ in range(3):
        # (a direction near the gradient, so that the slope is not a small
        # difference of large terms: dx itself is stored in bf16)
        d = dx / np.linalg.norm(dx) + 0.2 * rng.standard_normal(xv.shape) / np.sqrt(xv.size)
        slope = (loss(xv + h * d) - loss(xv - h * d)) / (2 * h)
        assert abs((dx * d).sum() - slope) <= 1e-2 * abs(slope)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("with_add,gated", [(True, False), (False, True)])
def test_block_of_bf16_layer(dtype, post, with_add, gated):
    cfg = synth.CONFIGS["mid"].with_(T=150)
    T, k, H = cfg.T, cfg.k, cfg.H
    layer, C, w = bf16_layer(cfg)
    rng = np.random.default_rng(9)
    x, d_x = stream(rng, (T, H), dtype)
    dy, d_dy = stream(rng, (T, H), dtype, 0.02)
    add = values(rng, (T, H), 0.5) if with_add else None
    weight, post_weight = (1 + 0.1 * rng.standard_normal((2, H))).astype(np.float32)
    sw = rng.random(T).astype(np.float32) if gated else None
    block = M.MoEBlock(layer, dev(weight), EPS, post, dev(post_weight) if post else None, 0.5, 2.0)
    d_add, d_sw = (None if v is None else f(v) for v, f in ((add, up), (sw, dev)))
    log(f"[block] bf16 layer {dtype} post={post} add={with_add} gated={gated}")
    y = block.forward(d_x, d_add, d_sw, keep_gu=True)
    f, b = block.buffers(T, dtype), layer.buffers(T)
    v = x
    if with_add:
        v = get(f.sum).astype(np.float64)
        assert torch.equal(f.sum.cpu(), (d_x.float() + d_add.float()).to(dtype).cpu())
    n, en, r, er = ON.norm(v, weight.astype(np.float64), EPS)
    nv = bf16_values_host(f.n).astype(np.float64)
    check(nv, n, en, "n")
    ref = Reference(cfg, C, w, M.ACT_SILU, nv, b)
    pw = post_weight.astype(np.float64) if post else np.ones(H)
    rows, ws = ref.rows(sw)
    want, _, _ = ON.combine_norm(rows, ws, v, 0.5, post, pw, EPS, 2.0)
    # the layer's bar on the branch; then y is rounded once, by at most half a
    # step of each value (2^-8 of it in bf16), whatever the branch's share of it
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 4 * U
    assert np.linalg.norm(get(y) - want) <= 2e-3 * np.linalg.norm(want - 0.5 * v) + step * np.linalg.norm(want)
    f2, bb = block.backward(d_dy, d_x, d_sw)
    assert f2 is f
    g = ON.combine_norm_backward(dy, rows, ws, post, pw, EPS, 2.0)
    dD = np.zeros(ref.D.shape)
    dD[ref.inv] = g["rows"][0][:, :k].reshape(T * k, H)
    dD[T * k:] = g["rows"][0][:, k]
    dw = g["w"][0]
    assert rel_l2(host(bb.dw), dw[:, :k]) <= 5e-3
    if gated:
        assert rel_l2(host(f.d_shared_w), dw[:, k]) <= 5e-3
    if post:
        assert rel_l2(host(f.d_post_weight), g["weight"][0]) <= 5e-3
    back = ref.backward(bf16_round(dD).astype(np.float64), dw[:, :k], ref.dlogit(layer, b))
    compare(bb, back)
    dx, _, d_weight, _ = ON.norm_backward(back["dx_total"], v, weight.astype(np.float64), r, dy, 0.5)
    assert rel_l2(get(f.dx), dx) <= 5e-3 and rel_l2(host(f.d_weight), d_weight) <= 5e-3


@pytest.mark.parametrize("cls", [M.MoELayer, M.Int8MoELayer])
def test_block_of_quantised_layers(cls):
    """moe_norm's codes are the experts' operand; the experts' rows are those of
    the products called by hand; y and the gradients follow from them."""
    cfg = synth.CONFIGS["mid"]
    T, k, H, R = cfg.T, cfg.k, cfg.H, cfg.T * (cfg.k + 1)
    layer, C, _ = build(cls, cfg, None)
    rng = np.random.default_rng(10)
    x, d_x = stream(rng, (T, H), torch.float32)
    add = values(rng, (T, H), 0.5)
    weight, post_weight = (1 + 0.1 * rng.standard_normal((2, H))).astype(np.float32)
    block = M.MoEBlock(layer, dev(weight), EPS, True, dev(post_weight))
    log(f"[block] {cls.__name__}")
    y = block.forward(d_x, up(add))
    f, b = block.buffers(T, torch.float32), layer.buffers(T)
    v = get(f.sum)
    n, en, r, er = ON.norm(v, weight.astype(np.float64), EPS)
    if cls is M.MoELayer:
        check_e4m3(b.xq, b.xs, n, en, "codes")
        hq, hs = torch.empty_like(b.hq), torch.empty_like(b.hs)
        D = torch.empty_like(b.d)
        M.grouped_fp8_gemm_swiglu(b.xq, b.xs, b.perm_src, layer.w_gu, layer.w_gu_s, b.offsets, cfg.G, R, cfg.I, H, hq, hs)
        M.grouped_fp8_gemm(hq, hs, None, layer.w_dn, layer.w_dn_s, b.offsets, cfg.G, R, H, cfg.I, D)
        assert torch.equal(D.view(torch.int16), b.d.view(torch.int16))
    else:
        s = host(b.xs).astype(np.float64)[:, None]
        assert (np.abs(host(b.xq) * s - n) <= s * (0.5 + 254 * U) + en).all()
    idx, gate = host(b.topk_idx), host(b.topk_w).astype(np.float64)
    inv = np.asarray(permute(idx, cfg.E, 1)[2])[:T * k]
    Dv = bf16_values_host(b.d).astype(np.float64)
    rows, ws = ON.gather(Dv, inv, gate, np.ones(T), T, k)
    pw = post_weight.astype(np.float64)
    want, err, _ = ON.combine_norm(rows, ws, v, 1.0, 1, pw, EPS, 1.0)
    check_as(y, want, err, "y")
    dy, d_dy = stream(rng, (T, H), torch.float32, 0.02)
    if cls is M.Int8MoELayer:
        with pytest.raises(NotImplementedError):
            block.backward(d_dy, d_x)
        return
    f, bb = block.backward(d_dy, d_x)
    g = ON.combine_norm_backward(dy, rows, ws, 1, pw, EPS, 1.0)
    dD, e = np.zeros((R, H)), np.zeros((R, H))
    for out, src in ((dD, g["rows"][0]), (e, g["rows"][1])):
        out[inv], out[T * k:] = src[:, :k].reshape(T * k, H), src[:, k]
    check(bf16_values_host(bb.dD), dD, e, "dD")
    check_e4m3(bb.dDq, bb.dDs, dD, e, "dD codes")
    dt = bf16_values_host(bb.dx_total).astype(np.float64)
    assert np.isfinite(dt).all() and np.abs(dt).max() > 0
    dx, e, dwt, ew = ON.norm_backward(dt, v, weight.astype(np.float64), host(f.rstd).astype(np.float64), dy, 1.0)
    check_as(f.dx, dx, e, "dx")
    assert (np.abs(host(f.d_weight) - dwt) <= ew + U * np.abs(dwt)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_graphs(dtype):
    """Forward and backward as graphs, replayed between eager passes."""
    cfg = synth.CONFIGS["mid"]
    for make in (lambda: bf16_layer(cfg)[0], lambda: build(M.MoELayer, cfg, None)[0]):
        layer = make()
        T, H = cfg.T, cfg.H
        rng = np.random.default_rng(12)
        w = dev((1 + 0.1 * rng.standard_normal((2, H))).astype(np.float32))
        block = M.MoEBlock(layer, w[0].contiguous(), EPS, True, w[1].contiguous())
        xs = [stream(rng, (T, H), dtype)[1] for _ in range(2)]
        adds = [up(values(rng, (T, H))) for _ in range(2)]
        dy = stream(rng, (T, H), dtype, 0.02)[1]
        x_in, add_in = xs[0].clone(), adds[0].clone()
        f, b, bb = block.buffers(T, dtype).gradients(), layer.buffers(T), layer.backward_buffers(T)
        outs = lambda: [host(t.view(torch.uint8)).copy() for t in (f.y, f.sum, b.topk_idx, f.dx, f.d_weight, f.d_post_weight,
                                                                   bb.dC, bb.dw, bb.dW_dn)]
        eager = []
        for v, a in zip(xs, adds):
            x_in.copy_(v), add_in.copy_(a)
            block.forward(x_in, add_in, keep_gu=True)
            block.backward(dy, x_in)
            eager.append(outs())
        fwd = block.capture(x_in, add_in, keep_gu=True)
        bwd = torch.cuda.CUDAGraph()
        with torch.cuda.graph(bwd):
            block.backward(dy, x_in)
        for rep in range(3):
            for i in range(2):
                x_in.copy_(xs[i]), add_in.copy_(adds[i])
                fwd.replay()
                bwd.replay()
                torch.cuda.synchronize()
                for got, want in zip(outs(), eager[i]):
                    assert np.array_equal(got, want), (rep, i)
            block.forward(x_in, add_in, keep_gu=True)
            block.backward(dy, x_in)
            torch.cuda.synchronize()


def test_block_balance_term_and_refusals():
    cfg = synth.CONFIGS["tiny"]
    layer = build(M.MoELayer, cfg, None)[0]
    block = M.MoEBlock(layer)
    x = up(values(np.random.default_rng(1), (cfg.T, cfg.H)))
    block.forward(x, seq_len=16, alpha=0.5)
    f, bb = block.backward(x, x, seq_len=16, alpha=0.5)
    assert np.isfinite(bf16_values_host(f.dx)).all() and np.isfinite(host(layer.buffers(cfg.T).seq_loss)).all()
    with pytest.raises(ValueError, match="differ"):
        block.backward(x.float(), x)
    gated = M.MoEBlock(build(M.MoELayer, cfg, GATES[0])[0])
    with pytest.raises(ValueError, match="Gate"):
        gated.forward(x, seq_len=16)
    odd = dataclasses.replace(cfg, E=12, n_group=4, topk_group=2, k=3)
    blk = M.MoEBlock(bf16_layer(odd, GATES[1])[0])
    blk.forward(x)
    with pytest.raises(ValueError, match="E is 12"):
        blk.backward(x, x)


def test_empty_batches():
    cfg = synth.CONFIGS["tiny"]
    layer = bf16_layer(cfg)[0]
    e = bf16_dev(np.zeros((0, cfg.H), np.uint16))
    assert layer.forward(e).shape == (0, cfg.H)
    bb = layer.backward(e, e)
    assert (host(bb.dW_gu) == 0).all() and (host(bb.dC) == 0).all()
    w = torch.ones(cfg.H, device="cuda")
    block = M.MoEBlock(layer, w, EPS, True, w)
    assert block.forward(e, e).shape == (0, cfg.H)
    f, bb = block.backward(e, e)
    assert (host(f.d_weight) == 0).all() and (host(f.d_post_weight) == 0).all()


def test_new_weights():
    """requantize_from_fp32 rounds new weights in place."""
    cfg = synth.CONFIGS["tiny"]
    layer, _, w = bf16_layer(cfg)
    gu = torch.from_numpy(np.stack([synth.gen_expert_weight(cfg, "gu", e) for e in range(cfg.G)])).cuda()
    dn = torch.from_numpy(np.stack([synth.gen_expert_weight(cfg, "dn", e) for e in range(cfg.G)])).cuda()
    layer.requantize_from_fp32(2 * gu, dn)
    assert np.array_equal(get(layer.w_gu), 2 * w[0]) and np.array_equal(get(layer.w_dn), w[1])
