"""What a forward leaves for the backward, with other forwards between the two:
called, replayed, of another type, of another block on the same layer."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
import synth
from bf16_cases import up, values
from gpu_common import dev, host
from test_gpu_bf16_layer import bf16_layer
from test_gpu_gate_int8_layers import build
from test_gpu_norm import EPS, stream

pytestmark = pytest.mark.gpu

CFG = synth.CONFIGS["mid"]
LAYERS = {"bf16": lambda: bf16_layer(CFG)[0], "fp8": lambda: build(M.MoELayer, CFG, None)[0]}


def weight(seed=1):
    return dev((1 + 0.1 * np.random.default_rng(seed).standard_normal(CFG.H)).astype(np.float32))


def batch(seed, dtype=torch.float32):
    rng = np.random.default_rng(seed)
    shape = (CFG.T, CFG.H)
    return stream(rng, shape, dtype)[1], up(values(rng, shape)), stream(rng, shape, dtype, 0.02)[1]


def gradients(block, dy, x, **kw):
    f, bb = block.backward(dy, x, **kw)
    return [host(t.float()).copy() for t in (f.dx, f.d_weight, bb.dC, bb.dw, bb.dW_gu, bb.dW_dn)]


def same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("kind", LAYERS)
def test_backward_after_another_forward(kind):
    layer = LAYERS[kind]()
    block, other = M.MoEBlock(layer, weight(), EPS), M.MoEBlock(layer, weight(2), EPS)
    x, add, dy = batch(1)
    x2 = batch(2, torch.bfloat16)[0]
    with pytest.raises(ValueError, match="before a forward"):
        block.backward(dy, x)
    block.forward(x, add, keep_gu=True)
    want = gradients(block, dy, x)
    for between in (lambda: block.forward(x2), lambda: other.forward(x), lambda: layer.forward(x2),
                    lambda: layer.forward(x2, keep_gu=True)):
        block.forward(x, add, keep_gu=True)
        between()
        with pytest.raises(ValueError, match="another forward"):
            block.backward(dy, x)
    # (buffers of another number of tokens are others)
    block.forward(x, add, keep_gu=True)
    block.forward(x[:-3].contiguous())
    same(gradients(block, dy, x), want)


@pytest.mark.parametrize("kind", LAYERS)
def test_backward_after_a_replay(kind):
    """The replayed forward's, whatever was called between capture and replay."""
    layer = LAYERS[kind]()
    block, other = M.MoEBlock(layer, weight(), EPS), M.MoEBlock(layer, weight(2), EPS)
    x, add, dy = batch(1)
    x2, add2, _ = batch(2)
    block.forward(x, add, keep_gu=True)
    want = gradients(block, dy, x)
    with_add, without = block.capture(x, add, keep_gu=True), block.capture(x2)
    block.forward(x2, keep_gu=True)
    want2 = gradients(block, dy, x2)
    for between in (lambda: block.forward(x2, keep_gu=False), lambda: other.forward(x2), without.replay,
                    lambda: layer.forward(add2)):
        between()
        with_add.replay()
        same(gradients(block, dy, x), want)
    for between in (lambda: block.forward(x, add, keep_gu=True), with_add.replay):
        between()
        without.replay()   # (gate and up not kept: what lies there is the other's)
        same(gradients(block, dy, x2), want2)


@pytest.mark.parametrize("kind", LAYERS)
def test_layer_backward_after_a_replay(kind):
    """keep_gu is the captured forward's, not that of a call in between."""
    layer = LAYERS[kind]()
    x, x2, dy = (up(values(np.random.default_rng(i), (CFG.T, CFG.H), s)) for i, s in ((1, 1.0), (2, 1.0), (3, 0.02)))

    def grads():
        bb = layer.backward(dy, x)
        return [host(t.float()).copy() for t in (bb.dx_total, bb.dW_gu, bb.dW_dn, bb.dC)]
    layer.forward(x)
    want = grads()
    g = layer.capture(x)
    layer.forward(x2, keep_gu=True)
    g.replay()
    same(grads(), want)


def test_backward_as_its_forward():
    layer = LAYERS["fp8"]()
    block = M.MoEBlock(layer, weight(), EPS)
    x, _, dy = batch(1)
    xb = x.bfloat16()
    sw = dev(np.random.default_rng(1).random(CFG.T).astype(np.float32))
    block.forward(x, None, sw)
    with pytest.raises(ValueError, match="shared_w"):
        block.backward(dy, x)
    block.forward(x)
    with pytest.raises(ValueError, match="shared_w"):
        block.backward(dy, x, sw)
    # the balance statistic of an earlier forward is not this one's
    for f, b in ((lambda **kw: block.forward(x, **kw), lambda **kw: block.backward(dy, x, **kw)),
                 (lambda **kw: layer.forward(xb, **kw), lambda **kw: layer.backward(xb, xb, **kw))):
        f(seq_len=16)
        b(seq_len=16)
        b()
        f()
        with pytest.raises(ValueError, match="seq_len"):
            b(seq_len=16)
        f(seq_len=16)
        with pytest.raises(ValueError, match="seq_len"):
            b(seq_len=8)


def test_refused_before_anything_is_launched():
    """A refused call leaves what the last forward left."""
    for shared in (1, 0):
        cfg = CFG.with_(n_shared=shared)
        layer = bf16_layer(cfg)[0]
        block = M.MoEBlock(layer, weight(), EPS)
        x, add, dy = batch(1)
        x2 = batch(2)[0]
        T, H = cfg.T, cfg.H
        sw = torch.rand(T, device="cuda")
        block.forward(x, add, keep_gu=True)
        want = gradients(block, dy, x)
        f, b = block.buffers(T, x.dtype), layer.buffers(T)
        kept = [t.clone() for t in (f.n, f.sum, f.rstd, f.y, b.d, b.h, b.hgu, b.topk_w, b.inv_perm)]
        wide = torch.zeros((T, 2 * H), device="cuda")
        loose = torch.zeros(T * H + 1, device="cuda")[1:].view(T, H)   # not 16-byte aligned
        bad = [lambda: block.forward(x2, None, sw.double()), lambda: block.forward(x2, None, sw.cpu()),
               lambda: block.forward(x2, None, torch.rand(2 * T, device="cuda")[::2]),
               lambda: block.forward(x2, add.float()), lambda: block.forward(x2, add.t().contiguous().t()),
               lambda: block.forward(x2.half()), lambda: block.forward(wide[:, ::2]), lambda: block.forward(loose),
               lambda: block.backward(dy, loose), lambda: block.backward(loose, x), lambda: block.backward(dy, wide[:, ::2]),
               lambda: block.backward(wide[:, ::2], x)]
        if not shared:
            bad += [lambda: block.forward(x2, None, sw), lambda: block.backward(dy, x, sw)]
        for i, call in enumerate(bad):
            with pytest.raises((ValueError, TypeError, M.MoEError)):
                call()
            torch.cuda.synchronize()
            for t, k in zip((f.n, f.sum, f.rstd, f.y, b.d, b.h, b.hgu, b.topk_w, b.inv_perm), kept):
                assert torch.equal(t.view(torch.uint8), k.view(torch.uint8)), i
        same(gradients(block, dy, x), want)
        H2 = torch.ones(2 * H, device="cuda")
        for w in (H2[:H].double(), H2[:H].cpu(), H2[::2], H2[1:H + 1]):
            for kw in (dict(weight=w), dict(post_norm=True, post_weight=w)):
                with pytest.raises((ValueError, TypeError)):
                    M.MoEBlock(layer, **kw)


def test_intermediates_of_a_bf16_layer():
    """keep_intermediates: dGU and h, whose products are the weights' gradients."""
    layer = LAYERS["bf16"]()
    x, dy = (up(values(np.random.default_rng(i), (CFG.T, CFG.H), s)) for i, s in ((1, 1.0), (2, 0.02)))
    layer.forward(x)
    bb = layer.backward(dy, x, keep_intermediates=True)
    b = layer.buffers(CFG.T)
    offs = host(b.offsets)
    g = int(np.argmax(np.diff(offs)))
    r = slice(int(offs[g]), int(offs[g + 1]))
    h, dD, dgu = (t[r].double() for t in (bb.h, bb.dD, bb.dgu))
    xs = x[b.perm_src[r].long()].double()
    # (fp32 sums over the group's rows: at most so many roundings of 2^-24 in the norm)
    for got, want in ((bb.dW_dn[g], dD.t() @ h), (bb.dW_gu[g], dgu.t() @ xs)):
        assert torch.linalg.norm(got.double() - want) <= len(h) * 2.0 ** -24 * torch.linalg.norm(want)


@pytest.mark.parametrize("what", ["layer", "block"])
def test_replay_with_a_balance_term(what):
    """The statistic of a captured seq_len after a forward of another one."""
    layer = LAYERS["fp8"]()
    b = layer.buffers(CFG.T)
    if what == "block":
        call, (x, _, dy) = M.MoEBlock(layer, weight(), EPS), batch(1)
        dx = lambda bb: bb[0].dx
        bwd = lambda bb: bb[1]
    else:
        call = layer
        x, dy = (up(values(np.random.default_rng(i), (CFG.T, CFG.H), s)) for i, s in ((1, 1.0), (2, 0.02)))
        dx, bwd = lambda bb: bb.dx_total, lambda bb: bb

    def results():
        bb = call.backward(dy, x, seq_len=16, alpha=2.0)
        return [host(t.float()).copy() for t in (dx(bb), bwd(bb).dC, b.seq_loss, b.seq_f, b.scores)]
    call.forward(x, seq_len=16, alpha=2.0)
    want = results()
    g = call.capture(x, seq_len=16, alpha=2.0)
    call.forward(x, seq_len=64, alpha=2.0)
    room = [torch.full((n,), 7.0, device="cuda") for n in (b.scores.numel(), CFG.T, 64, 1024, 4096) for _ in range(8)]
    g.replay()
    same(results(), want)
    assert all((t == 7).all() for t in room)


def test_gradient_in_the_layers_own_buffers():
    """dy comes down the residual path too, after the layer's backward: it
    cannot lie in what that writes.  It can be the block's own dx."""
    layer = LAYERS["bf16"]()
    block = M.MoEBlock(layer, weight(), EPS)
    x, add, dy = batch(1, torch.bfloat16)
    block.forward(x, add)
    want = gradients(block, dy, x)
    f, bb = block.buffers(CFG.T, x.dtype), layer.backward_buffers(CFG.T)
    for t in (bb.dx_total, bb.dx, bb.dD[:CFG.T], bb.dxp[:CFG.T]):
        t.copy_(dy)
        with pytest.raises(ValueError, match="copies"):
            block.backward(t, x)
        with pytest.raises(ValueError, match="copies"):
            block.backward(dy, t)
    f.dx.copy_(dy)
    same(gradients(block, f.dx, x), want)
