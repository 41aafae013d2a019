"""The bf16 products and the norms at their edges: rows of NaN next to the ones
that count, batches larger than a grid, offsets past 32 bits, two streams."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_bias_amd as M
import synth
from bf16_cases import U, check, offsets, up, values
from bf16_plan import plan
from gpu_common import bf16_values_host, dev, host, log
from oracle import bf16 as OB
from oracle import norm as ON
from test_gpu_bf16_layer import bf16_layer
from test_gpu_gate_int8_layers import build
from test_gpu_norm import EPS

pytestmark = pytest.mark.gpu

COUNTS = [0, 130, 1, 0, 256, 64, 65, 0, 17, 300, 5, 129, 63, 2, 97, 0]
NAN = float("nan")


def every_other(v, axis):
    """v with NaN in every other row (axis 0) or column."""
    t = up(v)
    if axis == 0:
        t[1::2] = NAN
    else:
        t[..., 1::2] = NAN
    return t


@pytest.mark.parametrize("want,mode,counts,N,K", [
    ("wide", "gemm", [c * 2 for c in COUNTS], 5128, 72), ("mid", "gemm", COUNTS, 1032, 72),
    ("split64x16", "gemm", [50, 3], 72, 72), ("split16x16", "gemm", [7], 72, 200),
    ("wide", "dgrad", [c * 2 for c in COUNTS], 72, 5128), ("mid", "dgrad", COUNTS, 72, 1032),
    ("wide", "wgrad", COUNTS, 1032, 1032), ("mid", "wgrad", COUNTS, 264, 392)])
def test_nan_rows_and_columns_stay_where_they_are(want, mode, counts, N, K):
    """Every other row of the first operand, and then every other row (column)
    of the second, NaN: the others' results are what they are without."""
    log(f"[edges] nan {want} {mode}")
    rng = np.random.default_rng([N, K])
    offs, G = offsets(counts), len(counts)
    R = int(offs[-1])
    assert plan(mode, G, R, N, K) == want
    if mode == "wgrad":
        dy, a = values(rng, (R, N)), values(rng, (R, K))
        ref, err = OB.wgrad(dy, a, offs)
        for d_dy, d_a, ok in ((every_other(dy, 1), up(a), np.s_[:, ::2]), (up(dy), every_other(a, 1), np.s_[:, :, ::2])):
            dw = torch.empty((G, N, K), device="cuda")
            M.grouped_bf16_wgrad(d_dy, d_a, None, dev(offs), G, R, N, K, dw)
            got = host(dw)
            assert (np.abs(got[ok] - ref[ok]) <= err[ok] + U * np.abs(ref[ok])).all()
            some = np.asarray(counts) > 0
            assert np.isnan(got).any(axis=(1, 2))[some].all() and (got[~some] == 0).all()
        return
    a = values(rng, (R, K if mode == "gemm" else N))
    b = values(rng, (G, N, K), 0.1)
    ref, err = OB.products(a, b, offs) if mode == "gemm" else OB.dgrad(a, b, offs)
    second = up(b)
    if mode == "gemm":
        second[:, 1::2] = NAN
    else:
        second[:, :, 1::2] = NAN
    for da, db, ok in ((every_other(a, 0), up(b), np.s_[::2]), (up(a), second, np.s_[:, ::2])):
        out = torch.empty(ref.shape, dtype=torch.bfloat16, device="cuda")
        if mode == "gemm":
            M.grouped_bf16_gemm(da, None, db, dev(offs), G, R, N, K, out)
        else:
            M.grouped_bf16_gemm_dgrad(da, db, dev(offs), G, R, N, K, out)
        got = bf16_values_host(out)
        check(got[ok], ref[ok], err[ok], want)
        rest = got[1::2] if ok == np.s_[::2] else got[:, 1::2]
        assert np.isnan(rest).all()


def test_more_rows_than_a_grid():
    T, H = (1 << 21) + 5, 16
    rng = np.random.default_rng(1)
    some = np.array([0, 1, (1 << 21) - 1, 1 << 21, T - 1])
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    v = values(rng, (len(some), H))
    x[dev(some)] = up(v)
    n, r = torch.full_like(x, 9), torch.empty(T, device="cuda")
    q, s = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    M.moe_norm(x, None, None, T, H, EPS, None, n, r, M.QUANT_INT8, q, s)
    ref, err, _, _ = ON.norm(v, 1.0, EPS)
    check(bf16_values_host(n[dev(some)]), ref, err, "n")
    assert (n[2:1000].float() == 1).all() and (q[2:1000] == 127).all() and (q[T - 1].abs().max() == 127)
    y = torch.empty_like(x)
    perm = torch.arange(T, dtype=torch.int32, device="cuda")
    M.moe_combine_norm(x, perm, torch.ones(T, device="cuda"), None, None, x, 0.0, 1, None, EPS, 1.0, T, 1, H, y)
    assert torch.equal(y, n)


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31 and 2^32 bytes and elements."""
    T, H = 140000, 16384
    rng = np.random.default_rng(2)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    v = values(rng, (2, H))
    x[T - 2:] = up(v)
    n, r = torch.empty_like(x), torch.empty(T, device="cuda")
    M.moe_norm(x, None, None, T, H, EPS, None, n, r)
    ref, err, rr, _ = ON.norm(v, 1.0, EPS)
    check(bf16_values_host(n[T - 2:]), ref, err, "n")
    assert not n[:T - 2].any()
    # its gradient, in place over the residual's
    dn = x.clone()
    M.moe_norm_backward(dn, x, None, r, n, 0.0, T, H, n, None, None, 0)
    dx, e, _, _ = ON.norm_backward(v, v, 1.0, host(r)[T - 2:].astype(np.float64), np.zeros((2, H)), 1.0)
    check(bf16_values_host(n[T - 2:]), dx, e, "dx")
    # the combine of those rows, last first
    perm = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    w = torch.full((T,), 0.5, device="cuda")
    M.moe_combine_norm(x, perm, w, None, None, x, 0.0, 0, None, EPS, 1.0, T, 1, H, n)
    assert torch.equal(n[:2].float(), x[T - 2:].flip(0).float() * 0.5)
    dD, dw = dn, torch.empty((T, 1), device="cuda")
    M.moe_combine_norm_backward(n, perm, w, x, 0, None, 0, None, EPS, 1.0, T, 1, H, dD, dw, None, None, None, None, None, 0)
    assert torch.equal(dD[T - 2:].float(), x[T - 2:].float() * 0.25) and not dD[:T - 2].any()


def test_two_streams():
    """Gradients with a workspace each and products side by side: the bits of
    calls one after the other."""
    rng = np.random.default_rng(3)
    jobs = []
    for T, H in ((3000, 1024), (700, 4096)):
        x, dn = up(values(rng, (T, H))), up(values(rng, (T, H)))
        r = torch.rand(T, device="cuda") + 0.5
        b = M.moe_norm_backward_workspace_bytes(T, H)
        w = up(values(rng, (1, 512, H)))
        offs = dev(np.array([0, T], np.int32))

        def job(T=T, H=H, x=x, dn=dn, r=r, b=b, w=w, offs=offs, stream=None):
            ws = torch.empty(b, dtype=torch.uint8, device="cuda")
            dx, dw, c = torch.empty_like(x), torch.empty(H, device="cuda"), torch.empty((T, 512), dtype=torch.bfloat16,
                                                                                        device="cuda")
            dW = torch.empty((1, 512, H), device="cuda")
            outs = (dx, dw, c, dW)

            def go():
                M.moe_norm_backward(dn, x, None, r, None, 1.0, T, H, dx, dw, ws, b, stream)
                M.grouped_bf16_gemm(x, None, w, offs, 1, T, 512, H, c, stream)
                M.grouped_bf16_wgrad(c, x, None, offs, 1, T, 512, H, dW, stream)
            return go, outs
        jobs.append(job)
    alone = []
    for job in jobs:
        go, outs = job()
        go()
        torch.cuda.synchronize()
        alone.append([host(t.float()) for t in outs])
    both = [job(stream=torch.cuda.Stream()) for job in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        for go, _ in both:
            go()
    torch.cuda.synchronize()
    for (_, outs), want in zip(both, alone):
        for t, v in zip(outs, want):
            assert np.array_equal(host(t.float()), v)


def test_bindings_refuse_wrong_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    f, i = x.float(), torch.zeros(5, dtype=torch.int32, device="cuda")
    for bad in (lambda: M.grouped_bf16_gemm(f, None, x[None], i, 1, 4, 4, 64, x),
                lambda: M.grouped_bf16_gemm(x, i.long(), x[None], i, 1, 4, 8, 64, x),
                lambda: M.grouped_bf16_wgrad(x, x, None, i, 1, 4, 64, 64, x),
                lambda: M.moe_norm(x.half(), None, None, 4, 64, EPS, None, x),
                lambda: M.moe_norm(f, x, None, 4, 64, EPS, x, x),
                lambda: M.moe_norm(x, None, f[0].bfloat16(), 4, 64, EPS, None, x),
                lambda: M.moe_combine_norm(f, i, f, None, None, x, 1.0, 1, None, EPS, 1.0, 4, 1, 64, x)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        M.moe_norm(x.cpu(), None, None, 4, 64, EPS, None, x)
    with pytest.raises(ValueError):
        M.moe_norm(torch.zeros((64, 4), dtype=torch.bfloat16, device="cuda").t(), None, None, 4, 64, EPS, None, x)


def test_block_on_its_own_output():
    """Forward in place over y; its backward, whose x is gone, is refused."""
    cfg = synth.CONFIGS["tiny"]
    block = M.MoEBlock(bf16_layer(cfg)[0])
    x = up(values(np.random.default_rng(5), (cfg.T, cfg.H)))
    y1 = block.forward(x).clone()
    want = block.forward(y1).clone()
    block.forward(x)
    y = block.forward(block.buffers(cfg.T, x.dtype).y)
    assert torch.equal(y, want)
    with pytest.raises(ValueError, match="written over"):
        block.backward(x, y)
    block.forward(y1)
    block.backward(x, y1)
    blk = M.MoEBlock(build(M.Int8MoELayer, synth.CONFIGS["mid"], None)[0])
    with pytest.raises(ValueError, match="keep_gu"):
        blk.forward(torch.zeros((4, synth.CONFIGS["mid"].H), device="cuda"), keep_gu=True)


def test_block_refuses_wrong_shapes():
    cfg = synth.CONFIGS["tiny"]
    layer = bf16_layer(cfg)[0]
    x, w = (torch.zeros(s, device="cuda") for s in ((cfg.T, cfg.H), (cfg.T,)))
    block = M.MoEBlock(layer)
    for bad in (lambda: M.MoEBlock(layer, x), lambda: M.MoEBlock(layer, None, EPS, True, x[0, 8:]),
                lambda: block.forward(x[:, 8:]), lambda: block.forward(x, x[1:].bfloat16()),
                lambda: block.forward(x, None, w[1:]), lambda: block.backward(x, x, w[1:]), lambda: block.backward(x, x)):
        with pytest.raises(ValueError):
            bad()
