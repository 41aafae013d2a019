"""Host-only checks of the C ABI: the library loads, exports every function
that include/moe_fp8.h declares, and rejects bad arguments with the
documented codes before launching anything (no GPU needed: every call here
fails validation or is a zero-sized no-op, so no HIP API is reached)."""
import ctypes
import os
import re

import pytest

from conftest import ROOT
from fp8_block_scaled_bias_amd import _lib as L

HEADER = os.path.join(ROOT, "include", "moe_fp8.h")
FAKE = ctypes.c_void_p(4096)  # never dereferenced: validation fails first


def header_functions():
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", src, flags=re.M)
    return sorted(set(n for n in names if n not in ("defined",)))


def test_library_exports_every_declared_function():
    lib = L.lib()
    names = header_functions()
    assert "grouped_fp8_gemm" in names and "moe_route" in names and len(names) >= 11
    for n in names:
        assert hasattr(lib, n), n
        assert n in L.SIGNATURES, n
    assert set(L.SIGNATURES) == set(names)
    assert L.version().startswith("moe_fp8")


def rc(name, *args):
    return getattr(L.lib(), name)(*args)


def test_quant_validation():
    assert rc("fp8_quant_1x128", FAKE, 4, 100, 100, 0, FAKE, FAKE, None) == L.MOE_ERR_INVALID
    assert "K=100" in L.last_error()
    assert rc("fp8_quant_1x128", FAKE, 4, 128, 128, 2, FAKE, FAKE, None) == L.MOE_ERR_INVALID
    assert rc("fp8_quant_1x128", FAKE, 4, 128, 128, 1, FAKE, FAKE, None) == L.MOE_ERR_INVALID
    assert "ld_in" in L.last_error()
    assert rc("fp8_quant_1x128", None, 4, 128, 128, 0, FAKE, FAKE, None) == L.MOE_ERR_INVALID
    assert rc("fp8_quant_1x128", ctypes.c_void_p(4100), 4, 128, 128, 0, FAKE, FAKE, None) == L.MOE_ERR_INVALID
    assert "aligned" in L.last_error()
    assert rc("fp8_quant_1x128", None, 0, 128, 128, 0, None, None, None) == L.MOE_OK
    assert rc("fp8_quant_128x128", FAKE, 2, 100, 128, FAKE, FAKE, None) == L.MOE_ERR_INVALID
    assert rc("fp8_quant_128x128", None, 0, 128, 128, None, None, None) == L.MOE_OK


def test_transpose_validation():
    def f(G=2, N=256, K=384, w=FAKE, ws=FAKE, wt=ctypes.c_void_p(8192), wts=ctypes.c_void_p(8192 + 64)):
        return rc("fp8_transpose_128x128", w, ws, G, N, K, wt, wts, None)
    assert f(N=100) == L.MOE_ERR_INVALID and "N=100" in L.last_error()
    assert f(K=0) == L.MOE_ERR_INVALID
    assert f(G=-1) == L.MOE_ERR_INVALID and f(G=70000) == L.MOE_ERR_INVALID
    assert f(w=None) == L.MOE_ERR_INVALID and "null" in L.last_error()
    assert f(w=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert f(wt=FAKE) == L.MOE_ERR_INVALID and "alias" in L.last_error()
    assert f(G=0, w=None, ws=None, wt=None, wts=None) == L.MOE_OK


def test_wgrad_validation():
    cap = 1 + 4                              # M_total = 100, G = 4
    def q(G=4, M=100, C=256, ld_in=256, cap=cap, out=FAKE, idx=None, in_rows=100):
        return rc("fp8_quant_128x1_grouped", FAKE, ld_in, idx, in_rows, FAKE, G, M, C, out, FAKE, cap,
                  None)
    assert q(C=100) == L.MOE_ERR_INVALID and "C=100" in L.last_error()
    assert q(G=0) == L.MOE_ERR_INVALID
    assert q(G=2000) == L.MOE_ERR_UNSUPPORTED
    assert q(ld_in=128) == L.MOE_ERR_INVALID and "ld_in" in L.last_error()
    assert q(cap=cap - 1) == L.MOE_ERR_INVALID and "chunks_cap" in L.last_error()
    assert q(out=None) == L.MOE_ERR_INVALID
    assert q(out=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert q(in_rows=99) == L.MOE_ERR_INVALID and "in_rows" in L.last_error()
    assert q(idx=FAKE, in_rows=0) == L.MOE_ERR_INVALID
    def w(G=4, M=100, N=256, K=384, cap=cap, dW=FAKE):
        return rc("grouped_fp8_wgrad", FAKE, FAKE, FAKE, FAKE, cap, FAKE, G, M, N, K, dW, None)
    assert w(N=200) == L.MOE_ERR_INVALID and "N=200" in L.last_error()
    assert w(G=0) == L.MOE_ERR_INVALID
    assert w(cap=4) == L.MOE_ERR_INVALID and "chunks_cap" in L.last_error()
    assert w(dW=None) == L.MOE_ERR_INVALID
    assert L.wgrad_chunks(100, 4) == cap and L.wgrad_chunks(256, 3) == 5


def test_backward_elementwise_validation():
    def c(T=4, k=2, H=256, ns=1, dD=ctypes.c_void_p(8192)):
        return rc("moe_combine_backward", FAKE, FAKE, FAKE, FAKE, T, k, H, ns, dD, FAKE, None, None,
                  None)
    assert c(k=9) == L.MOE_ERR_INVALID and "k=9" in L.last_error()
    assert c(H=100) == L.MOE_ERR_INVALID
    assert c(ns=2) == L.MOE_ERR_INVALID
    assert c(dD=FAKE) == L.MOE_ERR_INVALID and "alias" in L.last_error()
    assert c(dD=None) == L.MOE_ERR_INVALID
    assert c(T=0, dD=None) == L.MOE_OK
    def g(M=4, I=128, out=FAKE):
        return rc("swiglu_backward", FAKE, FAKE, M, I, out, FAKE, None, None, None)
    assert g(I=100) == L.MOE_ERR_INVALID and "I=100" in L.last_error()
    assert g(out=None) == L.MOE_ERR_INVALID
    assert g(out=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    # the fused 1x128 codes: both or neither, whole 128-column tiles
    assert rc("swiglu_backward", FAKE, FAKE, 4, 128, FAKE, FAKE, FAKE, None, None) == L.MOE_ERR_INVALID
    assert "together" in L.last_error()
    assert rc("swiglu_backward", FAKE, FAKE, 4, 136, FAKE, FAKE, FAKE, FAKE, None) == L.MOE_ERR_INVALID
    assert "I % 128" in L.last_error()
    assert rc("moe_combine_backward", FAKE, FAKE, FAKE, ctypes.c_void_p(8192), 4, 2, 136, 1, FAKE, FAKE,
              FAKE, FAKE, None) == L.MOE_ERR_INVALID and "H % 128" in L.last_error()
    def sg(G=2, M_=300, I=256, cap=100, out=FAKE, codes=FAKE):
        return rc("swiglu_backward_grouped", FAKE, FAKE, FAKE, G, M_, I, out, FAKE, codes, FAKE, cap,
                  FAKE, FAKE, FAKE, FAKE, None)
    assert sg(I=200) == L.MOE_ERR_INVALID and "I=200" in L.last_error()
    assert sg(G=0) == L.MOE_ERR_INVALID
    assert sg(G=2000) == L.MOE_ERR_UNSUPPORTED
    assert sg(cap=3) == L.MOE_ERR_INVALID and "chunks_cap" in L.last_error()
    assert sg(codes=None) == L.MOE_ERR_INVALID and "null" in L.last_error()
    # the bf16 dGU and h are optional, but only together
    assert sg(out=None) == L.MOE_ERR_INVALID and "together" in L.last_error()
    assert sg(out=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert sg(M_=0, out=None) == L.MOE_OK
    assert g(M=0, out=None) == L.MOE_OK
    def r(T=4, H=256, E=16, k=4, dx=FAKE, ts=None):
        return rc("moe_router_backward", FAKE, FAKE, FAKE, FAKE, FAKE, None, T, H, E, k, dx, FAKE, ts,
                  None)
    assert r(k=9) == L.MOE_ERR_INVALID and r(E=2) == L.MOE_ERR_INVALID
    assert r(H=100) == L.MOE_ERR_INVALID and r(dx=None) == L.MOE_ERR_INVALID
    assert r(dx=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert r(ts=ctypes.c_void_p(4098)) == L.MOE_ERR_INVALID and "topk_s" in L.last_error()
    assert r(T=0, dx=None) == L.MOE_OK
    def d(E=16, H=256, out=FAKE):
        return rc("moe_router_dcentroids", FAKE, FAKE, FAKE, FAKE, 4, H, E, out, None)
    assert d(E=0) == L.MOE_ERR_INVALID and d(H=12) == L.MOE_ERR_INVALID and d(out=None) == L.MOE_ERR_INVALID


def test_gemm_validation():
    def f(G, M, N, K, A=FAKE, idx=None, A_rows=None):
        A_rows = M if A_rows is None else A_rows
        return rc("grouped_fp8_gemm", A, FAKE, idx, A_rows, FAKE, FAKE, FAKE, G, M, N, K, FAKE, None)
    assert f(0, 10, 128, 128) == L.MOE_ERR_INVALID
    assert f(5000, 10, 128, 128) == L.MOE_ERR_UNSUPPORTED   # more groups than the LDS tables hold
    assert f(4, 10, 100, 128) == L.MOE_ERR_INVALID and "N=100" in L.last_error()
    assert f(4, 10, 128, 200) == L.MOE_ERR_INVALID and "K=200" in L.last_error()
    assert f(4, -1, 128, 128) == L.MOE_ERR_INVALID
    assert f(4, 10, 128, 128, A=None) == L.MOE_ERR_INVALID
    assert f(4, 0, 128, 128, A=None) == L.MOE_OK          # empty problem is a no-op
    # A_rows: at least M_total rows without a row index, at least one with it
    assert f(4, 10, 128, 128, A_rows=9) == L.MOE_ERR_INVALID and "A_rows" in L.last_error()
    assert f(4, 10, 128, 128, idx=FAKE, A_rows=0) == L.MOE_ERR_INVALID
    assert f(4, 10, 128, 128, idx=FAKE, A_rows=1 << 31) == L.MOE_ERR_INVALID


def test_route_validation():
    def f(T=64, H=256, E=16, ng=4, tg=2, k=4, ws=FAKE, wsb=1 << 30, ts=None):
        return rc("moe_route", FAKE, T, H, FAKE, FAKE, E, ng, tg, k, FAKE, FAKE, FAKE, ws, wsb, ts,
                  None)
    assert f(H=200) == L.MOE_ERR_INVALID
    assert f(E=18, ng=4) == L.MOE_ERR_INVALID and "n_group" in L.last_error()
    assert f(tg=5) == L.MOE_ERR_INVALID
    assert f(k=9) == L.MOE_ERR_INVALID                       # k > topk_group * group size
    assert f(E=512, ng=8, tg=4, k=8) == L.MOE_ERR_UNSUPPORTED
    assert f(E=256, ng=8, tg=4, k=16) == L.MOE_ERR_UNSUPPORTED
    assert f(E=24, ng=4, tg=2, k=4) == L.MOE_ERR_UNSUPPORTED  # group size 6
    assert f(E=16, ng=16, tg=2, k=2) == L.MOE_ERR_INVALID      # group size 1: no top-2 sum
    assert f(wsb=16) == L.MOE_ERR_WORKSPACE
    assert f(ws=None) == L.MOE_ERR_WORKSPACE
    assert f(ts=ctypes.c_void_p(4098)) == L.MOE_ERR_INVALID and "topk_s" in L.last_error()


def test_route_scores_and_seq_balance_validation():
    def r(T=64, sc=FAKE, ss=FAKE, k=4):
        return rc("moe_route_scores", FAKE, T, 256, FAKE, FAKE, 16, 4, 2, k, FAKE, FAKE, FAKE, FAKE,
                  1 << 30, sc, ss, None, None)
    assert r(sc=None) == L.MOE_ERR_INVALID and "scores" in L.last_error()
    assert r(ss=None) == L.MOE_ERR_INVALID
    assert r(sc=ctypes.c_void_p(4100)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert r(k=9) == L.MOE_ERR_INVALID                       # moe_route's own checks still apply
    # workspace: two [B, chunks of 64 tokens, E] planes, 256-byte rounded
    assert L.moe_seq_balance_workspace_bytes(0, 256, 4096) == 0
    assert L.moe_seq_balance_workspace_bytes(16384, 256, 4096) == 2 * 4 * 64 * 256 * 4
    assert L.moe_seq_balance_workspace_bytes(100, 16, 64) == 2 * 256 * ((2 * 1 * 16 * 4 + 255) // 256)
    def b(T=100, E=16, k=4, L_=64, ws=FAKE, wsb=1 << 20, out=FAKE):
        return rc("moe_seq_balance", FAKE, FAKE, FAKE, T, E, k, L_, 1e-4, out, FAKE, FAKE, ws, wsb,
                  None)
    assert b(E=0) == L.MOE_ERR_INVALID and b(E=257) == L.MOE_ERR_INVALID
    assert b(k=17) == L.MOE_ERR_INVALID and b(k=0) == L.MOE_ERR_INVALID
    assert b(L_=0) == L.MOE_ERR_INVALID and b(L_=65537) == L.MOE_ERR_INVALID
    assert b(out=None) == L.MOE_ERR_INVALID
    assert b(wsb=64) == L.MOE_ERR_WORKSPACE and b(ws=None) == L.MOE_ERR_WORKSPACE
    assert b(T=0, out=None, ws=None) == L.MOE_OK


def test_router_backward_dense_validation():
    def d(T=64, H=256, E=16, k=4, L_=32, dxo=FAKE, dC=FAKE, ws=FAKE, wsb=1 << 30, dxi=None):
        return rc("moe_router_backward_dense", FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, T, H, E, k,
                  L_, 1e-4, dxi, dxo, dC, FAKE, ws, wsb, None)
    assert d(E=24) == L.MOE_ERR_INVALID and d(E=272) == L.MOE_ERR_INVALID
    assert d(k=9) == L.MOE_ERR_INVALID and d(H=192) == L.MOE_ERR_INVALID
    assert d(L_=0) == L.MOE_ERR_INVALID and d(dC=None) == L.MOE_ERR_INVALID
    assert d(dxo=None) == L.MOE_ERR_INVALID
    assert d(dxi=FAKE) == L.MOE_ERR_INVALID and "alias" in L.last_error()
    assert d(dxo=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    # slices of ~1024 tokens, at most 16; one slice needs no workspace
    assert L.moe_router_backward_dense_workspace_bytes(1000, 256, 16) == 0
    assert L.moe_router_backward_dense_workspace_bytes(16384, 7168, 256) == 16 * 256 * 7168 * 4
    assert L.moe_router_backward_dense_workspace_bytes(2000, 256, 16) == 2 * 16 * 256 * 4
    assert d(T=2000, wsb=16) == L.MOE_ERR_WORKSPACE


def test_swiglu_keep_validation():
    def k(I=256, GU=FAKE, M=100):
        return rc("grouped_fp8_gemm_swiglu_keep", FAKE, FAKE, None, M, FAKE, FAKE, FAKE, 4, M, I,
                  1024, FAKE, FAKE, GU, None)
    assert k(I=200) == L.MOE_ERR_INVALID
    assert k(GU=None) == L.MOE_ERR_INVALID and "GU" in L.last_error()
    assert k(GU=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID
    assert k(M=0, GU=None) == L.MOE_OK


def test_route_group_size_two_is_valid_shape():
    # E=16 in 8 groups has group size 2: valid, but 2 is not 4 * 2^n
    assert rc("moe_route", FAKE, 8, 256, FAKE, FAKE, 16, 8, 2, 4, FAKE, FAKE, FAKE, FAKE, 1 << 30,
              None, None) == L.MOE_ERR_UNSUPPORTED


def test_permute_and_combine_and_bias_validation():
    p = lambda T=10, k=8, E=256, ns=1, ws=FAKE, wsb=1 << 20: rc(
        "moe_permute", FAKE, FAKE, T, k, E, ns, FAKE, FAKE, FAKE, None, None, 7168, None, None,
        ws, wsb, None)
    assert p(k=9) == L.MOE_ERR_INVALID
    assert p(ns=2) == L.MOE_ERR_INVALID
    assert p(E=5000) == L.MOE_ERR_INVALID
    assert p(wsb=8) == L.MOE_ERR_WORKSPACE
    c = lambda T=4, k=8, H=7168: rc("moe_combine", FAKE, FAKE, FAKE, None, T, k, H, FAKE, None)
    assert c(H=7) == L.MOE_ERR_INVALID
    assert c(k=0) == L.MOE_ERR_INVALID
    assert c(T=0) == L.MOE_OK
    assert rc("moe_bias_update", FAKE, FAKE, 0, ctypes.c_float(0.001), None) == L.MOE_ERR_INVALID
    assert rc("moe_bias_update", None, FAKE, 256, ctypes.c_float(0.001), None) == L.MOE_ERR_INVALID


def test_workspace_sizes():
    assert L.moe_permute_workspace_bytes(16384, 8, 256) == 256 * 256 * 4
    assert L.moe_permute_workspace_bytes(0, 8, 256) == 0
    # router: partial logits [splits, T, E] fp32 (256-byte aligned); large
    # batches (4 splits here) also hold the three bf16 planes of the centroids
    assert L.moe_route_workspace_bytes(16384, 7168, 256) == 4 * 16384 * 256 * 4 + 3 * 256 * 7168 * 2
    b = L.moe_route_workspace_bytes(128, 7168, 256)
    assert b % (128 * 256 * 4) == 0 and b >= 128 * 256 * 4


def test_gate_validation():
    def g(lt=0, T=4, E=64, score=0, ng=4, tg=2, gt=2, k=4, rn=1, scale=1.0, logits=FAKE, idx=FAKE,
          counts=FAKE, scores=None, bias=None):
        return rc("moe_gate", logits, lt, T, E, bias, score, ng, tg, gt, k, rn, scale, idx, FAKE, counts,
                  scores, None)
    assert g(T=-1) == L.MOE_ERR_INVALID and "T=-1" in L.last_error()
    assert g(E=0) == L.MOE_ERR_INVALID and g(E=66) == L.MOE_ERR_INVALID and "n_group" in L.last_error()
    assert g(E=1028, k=1) == L.MOE_ERR_UNSUPPORTED and "1024" in L.last_error()
    assert g(lt=2) == L.MOE_ERR_INVALID and g(score=2) == L.MOE_ERR_INVALID and g(rn=2) == L.MOE_ERR_INVALID
    assert g(tg=5) == L.MOE_ERR_INVALID and g(tg=0) == L.MOE_ERR_INVALID
    assert g(gt=3) == L.MOE_ERR_INVALID and "group_top=3" in L.last_error()
    assert g(k=0) == L.MOE_ERR_INVALID and g(k=9) == L.MOE_ERR_UNSUPPORTED
    assert g(E=8, k=5) == L.MOE_ERR_INVALID        # two groups of two are kept
    assert g(E=66, ng=33, tg=33) == L.MOE_ERR_UNSUPPORTED and "n_group=33" in L.last_error()
    assert g(scale=float("inf")) == L.MOE_ERR_INVALID and g(scale=float("nan")) == L.MOE_ERR_INVALID
    assert g(logits=None) == L.MOE_ERR_INVALID and g(idx=None) == L.MOE_ERR_INVALID
    assert g(counts=None) == L.MOE_ERR_INVALID and "expert_counts" in L.last_error()
    assert g(logits=ctypes.c_void_p(4098)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert g(scores=ctypes.c_void_p(4098)) == L.MOE_ERR_INVALID
    assert g(bias=ctypes.c_void_p(4097)) == L.MOE_ERR_INVALID
    assert g(scores=FAKE) == L.MOE_ERR_INVALID and "alias" in L.last_error()

    def b(lt=0, T=4, E=64, score=0, k=4, rn=1, scale=1.0, idx=FAKE, dl=ctypes.c_void_p(8192), ds=None):
        return rc("moe_gate_backward", FAKE, lt, T, E, score, k, rn, scale, idx, FAKE, ds, dl, None)
    assert b(k=9) == L.MOE_ERR_UNSUPPORTED and b(E=3) == L.MOE_ERR_INVALID and b(E=2000) == L.MOE_ERR_UNSUPPORTED
    assert b(idx=None) == L.MOE_ERR_INVALID and b(dl=None) == L.MOE_ERR_INVALID
    assert b(dl=FAKE) == L.MOE_ERR_INVALID and "alias" in L.last_error()
    assert b(ds=ctypes.c_void_p(4098)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert b(rn=-1) == L.MOE_ERR_INVALID and b(scale=float("nan")) == L.MOE_ERR_INVALID
    assert b(T=0, idx=None, dl=None) == L.MOE_OK


def test_router_logits_validation():
    def f(T=4, H=256, E=16, x=FAKE, out=FAKE, ws=FAKE, n=1 << 20):
        return rc("moe_router_logits", x, T, H, FAKE, E, out, ws, n, None)
    assert f(H=100) == L.MOE_ERR_INVALID and f(E=0) == L.MOE_ERR_INVALID and f(T=-1) == L.MOE_ERR_INVALID
    assert f(E=1025) == L.MOE_ERR_UNSUPPORTED
    assert f(x=None) == L.MOE_ERR_INVALID and f(x=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID
    assert f(n=4) == L.MOE_ERR_WORKSPACE and f(ws=None) == L.MOE_ERR_WORKSPACE
    assert f(T=0, x=None, out=None) == L.MOE_OK

    def b(T=4, H=256, E=16, dx=ctypes.c_void_p(8192), dxin=None, dC=FAKE, ws=FAKE, n=1 << 30):
        return rc("moe_router_logits_backward", FAKE, FAKE, FAKE, T, H, E, dxin, dx, dC, ws, n, None)
    assert b(E=24) == L.MOE_ERR_INVALID and b(E=1040) == L.MOE_ERR_INVALID and b(H=64) == L.MOE_ERR_INVALID
    assert b(dC=None) == L.MOE_ERR_INVALID and b(dx=None) == L.MOE_ERR_INVALID
    assert b(dx=FAKE, dxin=FAKE) == L.MOE_ERR_INVALID and "alias" in L.last_error()
    assert b(T=5000, n=16) == L.MOE_ERR_WORKSPACE


def test_int8_validation():
    def q(M=4, K=128, ld=128, x=FAKE, out=FAKE):
        return rc("int8_quant_rows", x, M, K, ld, out, FAKE, None)
    assert q(K=100) == L.MOE_ERR_INVALID and "K=100" in L.last_error()
    assert q(ld=120) == L.MOE_ERR_INVALID and q(ld=132) == L.MOE_ERR_INVALID and q(M=-1) == L.MOE_ERR_INVALID
    assert q(x=None) == L.MOE_ERR_INVALID and q(x=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID
    assert q(out=ctypes.c_void_p(4100)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert q(K=1 << 25, ld=1 << 25) == L.MOE_ERR_UNSUPPORTED
    assert q(M=0, x=None, out=None) == L.MOE_OK

    def c(G=2, N=4, K=128, w=FAKE):
        return rc("int8_quant_channels", w, G, N, K, FAKE, FAKE, None)
    assert c(K=12) == L.MOE_ERR_INVALID and c(N=0) == L.MOE_ERR_INVALID and c(G=-1) == L.MOE_ERR_INVALID
    assert c(G=1 << 20, N=1 << 12) == L.MOE_ERR_UNSUPPORTED and c(w=None) == L.MOE_ERR_INVALID
    assert c(G=0, w=None) == L.MOE_OK

    for name in ("grouped_int8_gemm", "grouped_int8_gemm_swiglu"):
        def g(G=4, M=100, N=128, K=256, rows=100, idx=None, a=FAKE, out=FAKE):
            return rc(name, a, FAKE, idx, rows, FAKE, FAKE, FAKE, G, M, N, K, out, None)
        assert g(N=100) == L.MOE_ERR_INVALID and "=100" in L.last_error() and name in L.last_error()
        assert g(K=24) == L.MOE_ERR_INVALID and g(K=0) == L.MOE_ERR_INVALID and g(N=0) == L.MOE_ERR_INVALID
        assert g(K=131072) == L.MOE_ERR_UNSUPPORTED and g(G=1025) == L.MOE_ERR_UNSUPPORTED
        assert g(G=0) == L.MOE_ERR_INVALID and g(M=-1) == L.MOE_ERR_INVALID
        assert g(rows=99) == L.MOE_ERR_INVALID and "A_rows" in L.last_error()
        assert g(rows=0, idx=FAKE) == L.MOE_ERR_INVALID
        assert g(a=None) == L.MOE_ERR_INVALID and g(out=None) == L.MOE_ERR_INVALID
        assert g(a=ctypes.c_void_p(4104)) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
        assert g(M=0, a=None, out=None) == L.MOE_OK


def test_bf16_products_validation():
    odd, B, OUT = ctypes.c_void_p(4104), ctypes.c_void_p(16384), ctypes.c_void_p(12288)
    calls = {
        "grouped_bf16_gemm": lambda G=2, M=8, N=64, K=64, rows=8, idx=None, a=FAKE, b=B, o=OUT, act=0:
            rc("grouped_bf16_gemm", a, idx, rows, b, FAKE, G, M, N, K, o, None),
        "grouped_bf16_gemm_glu": lambda G=2, M=8, N=64, K=64, rows=8, idx=None, a=FAKE, b=B, o=OUT, act=0:
            rc("grouped_bf16_gemm_glu", a, idx, rows, b, FAKE, G, M, N, K, act, o, None, None),
        "grouped_bf16_gemm_dgrad": lambda G=2, M=8, N=64, K=64, rows=8, idx=None, a=FAKE, b=B, o=OUT, act=0:
            rc("grouped_bf16_gemm_dgrad", a, b, FAKE, G, M, N, K, o, None),
        "grouped_bf16_gemm_dgrad_glu": lambda G=2, M=8, N=64, K=64, rows=8, idx=None, a=FAKE, b=B, o=OUT, act=0:
            rc("grouped_bf16_gemm_dgrad_glu", a, b, ctypes.c_void_p(8192), FAKE, G, M, N, K, act, o, None),
        "grouped_bf16_wgrad": lambda G=2, M=8, N=64, K=64, rows=8, idx=None, a=FAKE, b=B, o=OUT, act=0:
            rc("grouped_bf16_wgrad", a, b, idx, rows, FAKE, G, M, N, K, o, None),
    }
    for name, f in calls.items():
        for bad in (dict(G=0), dict(M=-1), dict(N=60), dict(N=0), dict(K=4), dict(K=-8)):
            assert f(**bad) == L.MOE_ERR_INVALID and name in L.last_error(), (name, bad)
        for bad in (dict(G=1025), dict(N=(1 << 21) + 8), dict(K=(1 << 21) + 8)):
            assert f(**bad) == L.MOE_ERR_UNSUPPORTED, (name, bad)
        for p in "abo":
            assert f(**{p: None}) == L.MOE_ERR_INVALID and "null" in L.last_error(), (name, p)
            assert f(**{p: odd}) == L.MOE_ERR_INVALID and "aligned" in L.last_error(), (name, p)
        assert f(o=FAKE) == L.MOE_ERR_INVALID and f(o=B) == L.MOE_ERR_INVALID and "alias" in L.last_error()
        if name != "grouped_bf16_wgrad":
            assert f(M=0, a=None, b=None, o=None, rows=0) == L.MOE_OK
        if "glu" in name:
            assert f(act=2) == L.MOE_ERR_INVALID and "act=2" in L.last_error()
    for name in ("grouped_bf16_gemm", "grouped_bf16_gemm_glu", "grouped_bf16_wgrad"):
        assert calls[name](rows=7) == L.MOE_ERR_INVALID and "A_rows" in L.last_error()
        assert calls[name](rows=0, idx=FAKE) == L.MOE_ERR_INVALID
        assert calls[name](rows=4, idx=ctypes.c_void_p(4098)) == L.MOE_ERR_INVALID
    assert rc("grouped_bf16_gemm_dgrad_glu", FAKE, FAKE, FAKE, FAKE, 2, 8, 64, 64, 0, FAKE, None) == \
        L.MOE_ERR_INVALID and "alias" in L.last_error()


def test_norm_validation():
    odd = ctypes.c_void_p(4104)
    P = [ctypes.c_void_p(16384 * i) for i in range(1, 12)]

    def n(x=P[0], t=1, add=None, w=None, T=4, H=128, eps=1e-6, s=None, o=P[1], r=None, q=0, c=None, sc=None):
        return rc("moe_norm", x, t, add, w, T, H, eps, s, o, r, q, c, sc, None)

    def nb(dn=P[0], x=P[1], t=1, w=None, r=P[2], res=None, T=4, H=128, dx=P[3], dw=None, ws=None, b=0):
        return rc("moe_norm_backward", dn, x, t, w, r, res, 1.0, T, H, dx, dw, ws, b, None)

    def c(D=P[0], i=P[1], w=P[2], S=None, sw=None, x=P[3], t=1, norm=1, wt=None, eps=1e-6, T=4, k=2, H=128, y=P[4]):
        return rc("moe_combine_norm", D, i, w, S, sw, x, t, 1.0, norm, wt, eps, 1.0, T, k, H, y, None, None)

    def cb(dy=P[0], t=1, i=P[1], w=P[2], D=P[3], ns=0, sw=None, norm=1, wt=None, eps=1e-6, T=4, k=2, H=128, dD=P[4],
           dw=P[5], dsw=None, q=None, qs=None, dwt=None, ws=None, b=0):
        return rc("moe_combine_norm_backward", dy, t, i, w, D, ns, sw, norm, wt, eps, 1.0, T, k, H, dD, dw, dsw, q, qs,
                  dwt, ws, b, None)
    for name, f in (("moe_norm", n), ("moe_norm_backward", nb), ("moe_combine_norm", c), ("moe_combine_norm_backward", cb)):
        for bad in (dict(T=-1), dict(T=1 << 28), dict(H=0), dict(H=100), dict(t=2)):
            assert f(**bad) == L.MOE_ERR_INVALID and name in L.last_error(), (name, bad)
        assert f(H=16392) == L.MOE_ERR_UNSUPPORTED
    nan = float("nan")
    for f in (n, c, cb):
        for eps in (-1.0, 2.0, nan):
            assert f(eps=eps) == L.MOE_ERR_INVALID and "eps" in L.last_error()
    assert n(q=3) == L.MOE_ERR_INVALID and n(q=-1) == L.MOE_ERR_INVALID
    assert n(q=1, H=136, c=P[2], sc=P[3]) == L.MOE_ERR_INVALID and "128" in L.last_error()
    assert n(add=P[2]) == L.MOE_ERR_INVALID and n(s=P[2]) == L.MOE_ERR_INVALID and "together" in L.last_error()
    assert n(q=1) == L.MOE_ERR_INVALID and "null" in L.last_error()
    assert n(q=2, c=P[2], sc=None) == L.MOE_ERR_INVALID and n(x=None) == L.MOE_ERR_INVALID
    assert n(x=odd) == L.MOE_ERR_INVALID and n(w=odd) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert n(o=P[0]) == L.MOE_ERR_INVALID and "alias" in L.last_error()
    assert n(T=0, x=None, o=None) == L.MOE_OK
    for p in ("dn", "x", "r", "dx"):
        assert nb(**{p: None}) == L.MOE_ERR_INVALID and "null" in L.last_error()
    assert nb(dn=odd) == L.MOE_ERR_INVALID and "aligned" in L.last_error()
    assert nb(dx=P[0]) == L.MOE_ERR_INVALID and nb(dx=P[1]) == L.MOE_ERR_INVALID and "alias" in L.last_error()
    need = rc("moe_norm_backward_workspace_bytes", 4, 128)
    assert need == 4 * 128 * 4 and rc("moe_norm_backward_workspace_bytes", 1 << 20, 128) == 2048 * 128 * 4
    assert rc("moe_norm_backward_workspace_bytes", 1 << 20, 7168) == 512 * 7168 * 4
    assert rc("moe_combine_norm_backward_workspace_bytes", 4, 128) == need
    assert nb(dw=P[4], ws=P[5], b=need - 1) == L.MOE_ERR_WORKSPACE and str(need) in L.last_error()
    assert nb(dw=P[4]) == L.MOE_ERR_WORKSPACE
    assert nb(T=0, dn=None, x=None, r=None, dx=None) == L.MOE_OK
    for f in (c, cb):
        for bad in (dict(k=0), dict(k=9), dict(norm=2), dict(D=None), dict(i=None), dict(w=None), dict(D=odd)):
            assert f(**bad) == L.MOE_ERR_INVALID, bad
    assert c(sw=P[5]) == L.MOE_ERR_INVALID and "shared" in L.last_error()
    assert c(x=None) == L.MOE_ERR_INVALID and c(y=None) == L.MOE_ERR_INVALID
    assert c(y=P[0]) == L.MOE_ERR_INVALID and "alias" in L.last_error()
    assert c(T=0, D=None, i=None, w=None, x=None, y=None) == L.MOE_OK
    assert cb(ns=2) == L.MOE_ERR_INVALID
    assert cb(sw=P[6]) == L.MOE_ERR_INVALID and cb(dsw=P[6]) == L.MOE_ERR_INVALID and "shared" in L.last_error()
    assert cb(q=P[6]) == L.MOE_ERR_INVALID and "together" in L.last_error()
    assert cb(q=P[6], qs=P[7], H=136) == L.MOE_ERR_INVALID and "128" in L.last_error()
    assert cb(dD=P[3]) == L.MOE_ERR_INVALID and "alias" in L.last_error()
    assert cb(dwt=P[6], ws=P[7], b=need - 1) == L.MOE_ERR_WORKSPACE
    assert cb(T=0, dy=None, i=None, w=None, D=None, dD=None, dw=None) == L.MOE_OK
