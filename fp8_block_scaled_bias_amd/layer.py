"""DeepSeekMoE layer forward composed from the C-ABI calls.

The steps, in the order the method applies them (aliyun study note
developer.aliyun.com/article/1776647 section 2.2; news.qq.com/rain/a/
20241229A05OQF00 sections DeepSeekMoE 架构, 无额外损耗的负载均衡 and
FP8 低精度训练):

  1. moe_route         sigmoid scores + selection bias, 4-of-8-group top-8
     (moe_route_scores + moe_seq_balance with seq_len: also the
     sequence-wise balance statistic, factor alpha = 0.0001)
  2. fp8_quant_1x128   x -> E4M3 with 1x128 scales
  3. moe_permute       expert-major dispatch order (no copy: GEMM 1 gathers)
  4. grouped_fp8_gemm_swiglu
                       gate+up of the 256 routed experts and the shared one,
                       SwiGLU and 1x128 requantisation in the epilogue
  5. grouped_fp8_gemm  down projection
  6. moe_combine       gate-weighted sum of routed outputs + shared output
  7. moe_bias_update   (optional) aux-loss-free bias step for the next batch

MoELayer.backward runs the backward of the expert path in FP8 (the pages'
backward-for-input and backward-for-weights chunks, section 工程 › DualPipe
流水线并行, with the FP8 formats of section FP8 低精度训练):

  1. moe_combine_backward   dD = w * dy per routed row, dy for the shared rows
                            (bf16, and its 1x128 E4M3 codes in the same pass);
                            dw = <dy, D> (the gate weights' gradient)
  2. grouped_fp8_gemm_dgrad on W_dn                   dh = dD W_dn
  3. grouped_fp8_gemm       the gate+up outputs again (bf16; the fused
                            forward keeps none)
  4. swiglu_backward_grouped  dGU = [dg | du] and h (bf16), dGU's 1x128
                            codes, the 128x1 chunk codes of dGU and h
  5. grouped_fp8_gemm_dgrad on W_gu                   dX = dGU W_gu
  6. moe_combine            dx = the sum of a token's rows of dX (unit weights)
  7. fp8_quant_128x1_grouped (dD, gathered x) + grouped_fp8_wgrad
                            dW_dn = dD^T h,
                            dW_gu = dGU^T x (x gathered through the permutation)
  8. moe_router_backward    dw -> the gate logits' gradient, dx += its part
     moe_router_dcentroids  the centroids' gradient (the bias has none)
     (with seq_len: moe_router_backward_dense - the balance term's gradient
     on every expert's logit joins the gate's, dx and dC as fp32 GEMMs)

The input gradients read the weights in their forward layout (LDS transpose
reads inside the GEMM), so the backward keeps nothing derived from the
weights: after a weight update (requantize_from_fp32, or any write to w_gu /
w_dn) the next forward and backward use the new weights as they are.

With a Gate, the router is moe_router_logits + moe_gate instead of moe_route
(softmax scores, weights that are not renormalised, a scale, no bias, other
groups), and its backward moe_gate_backward + moe_router_logits_backward.

Int8MoELayer is the layer's forward with the experts in 8-bit integers (a scale
for each token and each output channel):

  1. the router, as above
  2. int8_quant_rows        x (on the side stream)
  3. moe_permute
  4. grouped_int8_gemm_swiglu   h = silu(gate) up, bf16
  5. int8_quant_rows        h
  6. grouped_int8_gemm      down projection
  7. moe_combine

Bf16MoELayer is the layer, forward and backward, on unquantised experts:

  1. the router and moe_permute, as above
  2. grouped_bf16_gemm_glu  h = act(gate) up, gathered x (its gate and up
                            outputs kept on demand)
  3. grouped_bf16_gemm      down projection
  4. moe_combine
  and backward moe_combine_backward, grouped_bf16_gemm_dgrad_glu (down, with the
  activation's backward), grouped_bf16_gemm_dgrad (gate and up), moe_combine,
  grouped_bf16_wgrad twice, the router's as above.

MoEBlock is one of these layers between its norms, on the residual stream:
moe_norm in front (in place of the operand's quantisation), moe_combine_norm at
the end (in place of moe_combine), and their backward.

torch is only used to hold device memory, to name the stream and to round new
bf16 weights; every step runs in the library's HIP kernels.
"""
from __future__ import annotations

import dataclasses
import functools
import inspect

import torch

from . import _lib as L


def _on_stream(call):
    """call with its `stream`, if one is given, as the current one: what it
    allocates and fills the first time comes before its launches there, and not
    in the order of whatever other stream was current."""
    where = list(inspect.signature(call).parameters).index("stream")

    @functools.wraps(call)
    def on_stream(*args, **kw):
        st = args[where] if len(args) > where else kw.get("stream")
        if not isinstance(st, torch.cuda.Stream) or st == torch.cuda.current_stream():
            return call(*args, **kw)
        with torch.cuda.stream(st):
            return call(*args, **kw)
    return on_stream


@dataclasses.dataclass(frozen=True)
class LayerShape:
    H: int
    E: int
    n_group: int
    topk_group: int
    k: int
    I: int
    n_shared: int = 1

    @property
    def G(self):
        return self.E + self.n_shared


@dataclasses.dataclass(frozen=True)
class Gate:
    """A router in one of moe_gate's forms: score SCORE_SOFTMAX or
    SCORE_SIGMOID; use_bias: the layer's bias moves the choice; groups (of the
    shape) by their group_top largest; renormalize: a token's weights sum to
    scale, else they are scale times the scores.  The layer's backward needs a
    number of experts that is a multiple of 16; its sequence-wise balance term
    (seq_len) goes with moe_route only."""
    score: int = L.SCORE_SOFTMAX
    use_bias: bool = True
    group_top: int = 2
    renormalize: bool = True
    scale: float = 1.0


@dataclasses.dataclass(frozen=True)
class Held:
    """Which forward a layer's buffers hold, as far as its backward has to know:
    whether the gate and up outputs were kept, the balance statistic's seq_len;
    of a MoEBlock its own buffers, whether it had an add and a shared_w."""
    gu: bool
    seq_len: int | None = None
    block: object = None
    added: bool = False
    gated: bool = False


class CapturedForward(torch.cuda.CUDAGraph):
    """The graph of one forward.  A replay leaves its buffers as that forward
    does, whichever was called in between, and they are noted as such."""
    bufs = held = None

    def replay(self):
        super().replay()
        self.bufs.held = self.held
        if self.held.seq_len is not None:
            self.bufs.balance(self.held.seq_len)


class Buffers:
    """Device buffers of one forward at T tokens (reused across calls).  held:
    the forward that they hold, None before the first."""

    def __init__(self, shape: LayerShape, T: int, device="cuda"):
        s = shape
        R = T * s.k + s.n_shared * T
        dev = torch.device(device)
        u8, i32, f32, bf = torch.uint8, torch.int32, torch.float32, torch.bfloat16
        self.T, self.R = T, R
        self.held = None
        self.topk_idx = torch.empty((T, s.k), dtype=i32, device=dev)
        self.topk_w = torch.empty((T, s.k), dtype=f32, device=dev)
        self.topk_s = torch.empty((T, s.k), dtype=f32, device=dev)   # the chosen experts' scores
        self.counts = torch.empty((s.E,), dtype=i32, device=dev)
        self.route_ws_bytes = max(16, L.moe_route_workspace_bytes(T, s.H, s.E))
        self.route_ws = torch.empty((self.route_ws_bytes,), dtype=u8, device=dev)
        self.offsets = torch.empty((s.G + 1,), dtype=i32, device=dev)
        self.perm_src = torch.empty((max(R, 1),), dtype=i32, device=dev)
        self.inv_perm = torch.empty((max(T * s.k, 1),), dtype=i32, device=dev)
        self.perm_ws_bytes = max(16, L.moe_permute_workspace_bytes(T, s.k, s.E))
        self.perm_ws = torch.empty((self.perm_ws_bytes,), dtype=u8, device=dev)
        self._hgu = None
        self._logits = None
        self._balance = {}
        self._dev = dev
        self._shape = s
        self.d = torch.empty((R, s.H), dtype=bf, device=dev)
        self.y = torch.empty((T, s.H), dtype=bf, device=dev)
        self._operands()

    def _operands(self):
        """The expert products' operands: x and h in E4M3 with 1x128 scales."""
        s, T, R, dev = self._shape, self.T, self.R, self._dev
        u8, f32 = torch.uint8, torch.float32
        self.xq = torch.empty((T, s.H), dtype=u8, device=dev)
        self.xs = torch.empty((T, s.H // 128), dtype=f32, device=dev)
        self.hq = torch.empty((R, s.I), dtype=u8, device=dev)
        self.hs = torch.empty((R, s.I // 128), dtype=f32, device=dev)

    def balance(self, seq_len: int):
        """Buffers of the sequence-wise balance statistic (allocated on first use
        and kept for each seq_len, which a captured graph may write): scores
        [T, E], score_sums [T], seq_f, seq_p [B, E], seq_loss [B], B = ceil(T /
        seq_len).  The names hold the last seq_len's."""
        s, T = self._shape, self.T
        if seq_len not in self._balance:
            dev, f32 = self._dev, torch.float32
            B = -(-T // seq_len)
            ws_bytes = max(16, L.moe_seq_balance_workspace_bytes(T, s.E, seq_len))
            self._balance[seq_len] = dict(
                scores=torch.empty((max(T, 1), s.E), dtype=f32, device=dev),
                score_sums=torch.empty((max(T, 1),), dtype=f32, device=dev),
                seq_f=torch.empty((max(B, 1), s.E), dtype=f32, device=dev),
                seq_p=torch.empty((max(B, 1), s.E), dtype=f32, device=dev),
                seq_loss=torch.empty((max(B, 1),), dtype=f32, device=dev),
                seq_ws_bytes=ws_bytes,
                seq_ws=torch.empty((ws_bytes,), dtype=torch.uint8, device=dev))
        vars(self).update(self._balance[seq_len])
        return self

    @property
    def logits(self):
        """fp32 router logits [T, E] of a layer with a Gate, which its backward
        reads (allocated on first use)."""
        if self._logits is None:
            self._logits = torch.empty((self.T, self._shape.E), dtype=torch.float32,
                                       device=self._dev)
        return self._logits

    @property
    def hgu(self):
        """bf16 gate+up outputs kept by forward(keep_gu=True) for the backward
        (allocated on first use)."""
        if self._hgu is None:
            self._hgu = torch.empty((self.R, 2 * self._shape.I), dtype=torch.bfloat16,
                                    device=self._dev)
        return self._hgu


class BackwardBuffers:
    """Device buffers of one layer backward at T tokens (reused across calls)."""

    def dense(self):
        """Buffers of the dense router backward (allocated on first use):
        dlogit [T, E] fp32 and its workspace."""
        if self.dlogit is None:
            s, T = self._shape, self.T
            self.dlogit = torch.empty((max(T, 1), s.E), dtype=torch.float32, device=self._dev)
            self.dense_ws_bytes = max(16, L.moe_router_backward_dense_workspace_bytes(T, s.H, s.E))
            self.dense_ws = torch.empty((self.dense_ws_bytes,), dtype=torch.uint8, device=self._dev)
        return self

    def intermediates(self):
        """Allocate the bf16 dGU [R, 2I] and h [R, I] that a backward with
        keep_intermediates writes (the GEMMs read only their FP8 codes)."""
        if self.dgu is None:
            I = self._shape.I
            self.dgu = torch.empty((self.R, 2 * I), dtype=torch.bfloat16, device=self._dev)
            self.h = torch.empty((self.R, I), dtype=torch.bfloat16, device=self._dev)
        return self

    def __init__(self, shape: LayerShape, T: int, device="cuda"):
        s = shape
        R = T * s.k + s.n_shared * T
        dev = torch.device(device)
        f32, bf = torch.float32, torch.bfloat16
        H, I = s.H, s.I
        self.T, self.R = T, R
        self.dD = torch.empty((R, H), dtype=bf, device=dev)
        self.dw = torch.empty((T, s.k), dtype=f32, device=dev)
        self.dxp = torch.empty((R, H), dtype=bf, device=dev)
        self.dx = torch.empty((T, H), dtype=bf, device=dev)
        self.ones = torch.ones((T, s.k), dtype=f32, device=dev)
        self.dW_gu = torch.empty((s.G, 2 * I, H), dtype=f32, device=dev)
        self.dW_dn = torch.empty((s.G, H, I), dtype=f32, device=dev)
        self.dx_total = torch.empty((T, H), dtype=bf, device=dev)
        self._shape, self._dev, self.dlogit = s, dev, None
        self.dlogit_rows = torch.empty((max(T * s.k, 1),), dtype=f32, device=dev)
        self.dC = torch.empty((s.E, H), dtype=f32, device=dev)
        self._operands()

    def _operands(self):
        """What only the products in E4M3 read and write."""
        s, R, dev = self._shape, self.R, self._dev
        u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
        H, I = s.H, s.I
        self.dDq = torch.empty((R, H), dtype=u8, device=dev)
        self.dDs = torch.empty((R, H // 128), dtype=f32, device=dev)
        self.dh = torch.empty((R, I), dtype=bf, device=dev)
        self.gu = torch.empty((R, 2 * I), dtype=bf, device=dev)
        self.dgu = self.h = None   # bf16 dGU and h: only with keep_intermediates
        self.dguq = torch.empty((R, 2 * I), dtype=u8, device=dev)
        self.dgus = torch.empty((R, 2 * I // 128), dtype=f32, device=dev)
        c = self.cap = L.wgrad_chunks(R, s.G)
        self.c_dD = torch.empty((c, H, 128), dtype=u8, device=dev)
        self.s_dD = torch.empty((c, H), dtype=f32, device=dev)
        self.c_h = torch.empty((c, I, 128), dtype=u8, device=dev)
        self.s_h = torch.empty((c, I), dtype=f32, device=dev)
        self.c_dgu = torch.empty((c, 2 * I, 128), dtype=u8, device=dev)
        self.s_dgu = torch.empty((c, 2 * I), dtype=f32, device=dev)
        self.c_x = torch.empty((c, H, 128), dtype=u8, device=dev)
        self.s_x = torch.empty((c, H), dtype=f32, device=dev)


def _check_weights(w, out):
    """New weights are fp32 of the shape that they replace: the kernels take
    their sizes from it, and a copy would repeat one expert's for all."""
    if w.dtype != torch.float32:
        raise TypeError(f"weights must be float32, not {w.dtype}")
    if w.shape != out.shape:
        raise ValueError(f"weights {list(w.shape)} in the place of {list(out.shape)}")


def _run(name, *args):
    """A step that is not timed."""
    args[-1]()


class MoELayer:
    """One MoE layer on one GPU: router state and FP8 expert weights.

    Weights are E4M3 with 128x128 scales:
      w_gu [G, 2I, H] (rows [0, I) gate, [I, 2I) up), w_gu_s [G, 2I/128, H/128]
      w_dn [G, H, I],                                  w_dn_s [G, H/128, I/128]
    Group E (the last) is the shared expert.
    """
    CODES = L.QUANT_E4M3   # the experts' operand, as moe_norm writes it

    def __init__(self, shape: LayerShape, centroids, bias, w_gu, w_gu_s, w_dn, w_dn_s,
                 gate: Gate | None = None):
        self.shape = shape
        self.gate = gate
        self.centroids = centroids
        self.bias = bias
        self.w_gu, self.w_gu_s, self.w_dn, self.w_dn_s = w_gu, w_gu_s, w_dn, w_dn_s
        self._bwd = {}
        self._bufs = {}
        self._side = None   # stream for x's quantisation beside the router (lazily made)

    @staticmethod
    def empty_weights(shape: LayerShape, device="cuda"):
        s = shape
        dev = torch.device(device)
        return (torch.empty((s.G, 2 * s.I, s.H), dtype=torch.uint8, device=dev),
                torch.empty((s.G, 2 * s.I // 128, s.H // 128), dtype=torch.float32, device=dev),
                torch.empty((s.G, s.H, s.I), dtype=torch.uint8, device=dev),
                torch.empty((s.G, s.H // 128, s.I // 128), dtype=torch.float32, device=dev))

    @staticmethod
    def quantize_into(w_f32, out_q, out_s, stream=None):
        """128x128 block quantisation of fp32 weights [G', N, K] into E4M3 + scales."""
        _check_weights(w_f32, out_q)
        G, N, K = w_f32.shape
        L.fp8_quant_128x128(w_f32, G, N, K, out_q, out_s, stream)

    @classmethod
    def from_fp32_experts(cls, shape: LayerShape, centroids, bias, gu_fp32, dn_fp32,
                          device="cuda", gate: Gate | None = None, **kw):
        """Build a layer from per-expert fp32 weights, quantised on the GPU.

        gu_fp32 / dn_fp32: iterables of (expert, array [2I, H] / [H, I]) covering
        every group 0..G-1 (G-1 is the shared expert).  Each array is copied
        to the GPU and quantised there (quantize_into).  kw: the class's own.
        """
        w_gu, w_gu_s, w_dn, w_dn_s = cls.empty_weights(shape, device)
        stream = torch.cuda.current_stream()
        for src, q, s in ((gu_fp32, w_gu, w_gu_s), (dn_fp32, w_dn, w_dn_s)):
            for e, arr in src:
                t = torch.from_numpy(arr).to(device)
                cls.quantize_into(t[None], q[e:e + 1], None if s is None else s[e:e + 1], stream)
                stream.synchronize()
        return cls(shape, centroids, bias, w_gu, w_gu_s, w_dn, w_dn_s, gate, **kw)

    def buffers(self, T: int) -> Buffers:
        b = self._bufs.get(T)
        if b is None:
            b = self._bufs[T] = Buffers(self.shape, T, self.centroids.device)
        return b

    @_on_stream
    def forward(self, x_bf16: torch.Tensor, bufs: Buffers | None = None, stream=None,
                update_bias: bool = False, gamma: float = 0.001,
                events: dict | None = None,
                seq_len: int | None = None, alpha: float = 0.0001,
                keep_gu: bool = False) -> torch.Tensor:
        """One layer forward.  With seq_len, also the sequence-wise balance
        statistic of the routing (factor alpha) over consecutive runs of
        seq_len tokens, into bufs.seq_f, seq_p and seq_loss.  keep_gu (for
        training): the fused gate+up kernel also writes its bf16 gate/up
        outputs into bufs.hgu (1.2 GB at T=16384), which the backward then
        reads instead of running the gate+up GEMM again; the layer's output
        is unchanged.  `events`, if
        given, maps a step name ("route", "seq_balance", "quant", "permute",
        "gate_up", "down", "combine", "bias") to a list that receives a
        (start, end) pair of torch.cuda.Event recorded on the launch stream
        around that step (quant: on the side stream it runs on); a dict that
        already holds keys times only those steps (each event pair adds a few
        microseconds to the step).

        x's 1x128 quantisation does not depend on the routing: it runs on a
        side stream (default priority) that forks from the launch stream
        before the router and joins it before the first expert GEMM, so the
        two overlap."""
        self._check_gate(seq_len)
        s = self.shape
        T = x_bf16.shape[0]
        b = bufs or self.buffers(T)
        self._check_rows(b, x_bf16)
        st = stream if stream is not None else torch.cuda.current_stream()
        if self._side is None:
            self._side = torch.cuda.Stream(device=st.device)
        side = self._side
        only = set(events) if events else None

        def step(name, on, fn):
            if events is None or (only is not None and name not in only):
                fn()
                return
            e0 = torch.cuda.Event(enable_timing=True)
            e1 = torch.cuda.Event(enable_timing=True)
            e0.record(on)
            fn()
            e1.record(on)
            events.setdefault(name, []).append((e0, e1))

        b.held = None
        side.wait_stream(st)
        step("quant", side, lambda: self._quantise(x_bf16, b, side))
        step("route", st, lambda: self._route(x_bf16, b, seq_len, st))
        if seq_len is not None:
            step("seq_balance", st, lambda: self._seq_balance(b, seq_len, alpha, st))
        step("permute", st, lambda: self._permute(b, st))
        st.wait_stream(side)
        self._experts(x_bf16, b, keep_gu, st, step)
        shared = b.d[T * s.k:T * s.k + T] if s.n_shared else None
        step("combine", st, lambda: L.moe_combine(b.d, b.inv_perm, b.topk_w, shared, T, s.k,
                                                  s.H, b.y, st))
        if update_bias:
            step("bias", st, lambda: L.moe_bias_update(b.counts, self.bias, s.E, gamma, st))
        b.held = Held(keep_gu, seq_len)
        return b.y

    def _quantise(self, x_bf16, b, stream):
        """The experts' operand of x."""
        H = self.shape.H
        L.fp8_quant_1x128(x_bf16, x_bf16.shape[0], H, H, 0, b.xq, b.xs, stream)

    def _permute(self, b, st):
        s = self.shape
        L.moe_permute(b.topk_idx, b.counts, b.T, s.k, s.E, s.n_shared, b.offsets, b.perm_src, b.inv_perm,
                      None, None, s.H, None, None, b.perm_ws, b.perm_ws_bytes, st)

    def _experts(self, x_bf16, b, keep_gu, st, step):
        """The experts' rows b.d of the operand and the permutation in b."""
        s, R = self.shape, b.R
        if keep_gu:
            step("gate_up", st, lambda: L.grouped_fp8_gemm_swiglu_keep(
                b.xq, b.xs, b.perm_src, self.w_gu, self.w_gu_s, b.offsets, s.G, R, s.I, s.H,
                b.hq, b.hs, b.hgu, st))
        else:
            step("gate_up", st, lambda: L.grouped_fp8_gemm_swiglu(
                b.xq, b.xs, b.perm_src, self.w_gu, self.w_gu_s, b.offsets, s.G, R, s.I, s.H,
                b.hq, b.hs, st))
        step("down", st, lambda: L.grouped_fp8_gemm(
            b.hq, b.hs, None, self.w_dn, self.w_dn_s, b.offsets, s.G, R, s.H, s.I, b.d, st))

    def requantize_from_fp32(self, gu_fp32, dn_fp32, stream=None):
        """Requantise both weight sets in place from fp32 master weights
        ([G, 2I, H] and [G, H, I] device tensors), as quantize_into does (the
        per-update cast after an optimizer step)."""
        _check_weights(dn_fp32, self.w_dn)   # (before the other is written)
        self.quantize_into(gu_fp32, self.w_gu, self.w_gu_s, stream)
        self.quantize_into(dn_fp32, self.w_dn, self.w_dn_s, stream)

    def capture(self, x_bf16: torch.Tensor, bufs: Buffers | None = None, **forward_kw):
        """One forward captured as a HIP graph (torch.cuda.CUDAGraph); its
        replay() reruns the whole layer on the same buffers - write the next
        batch into x_bf16 first - with one launch.  The library only launches
        kernels (no allocation, no memset, no host synchronisation), so every
        step is capturable.  forward_kw as in forward (not events).  A backward
        that is called after a replay is that of the captured forward."""
        T = x_bf16.shape[0]
        b = bufs or self.buffers(T)
        side = torch.cuda.Stream()   # default priority
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.forward(x_bf16, b, stream=side, **forward_kw)   # warm-up outside the capture
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = CapturedForward()
        with torch.cuda.graph(graph):
            self.forward(x_bf16, b, stream=torch.cuda.current_stream(), **forward_kw)
        graph.bufs, graph.held = b, b.held
        return graph

    def backward_buffers(self, T: int) -> BackwardBuffers:
        bb = self._bwd.get(T)
        if bb is None:
            bb = self._bwd[T] = BackwardBuffers(self.shape, T, self.centroids.device)
        return bb

    @_on_stream
    def backward(self, dy_bf16: torch.Tensor, x_bf16: torch.Tensor, bufs: Buffers | None = None,
                 bwd: BackwardBuffers | None = None, stream=None, events: dict | None = None,
                 seq_len: int | None = None, alpha: float = 0.0001,
                 keep_intermediates: bool = False):
        """Backward of the layer for the output gradient dy, after a forward of
        x on `bufs` (its routing, permutation, quantised x and D).  With
        seq_len (the forward's, which left the scores and f in `bufs`), the
        loss also holds the sequence-wise balance term alpha * sum_b L_bal,b
        and the router's backward is the dense one (bwd.dlogit [T, E]).
        After a forward with keep_gu the gate+up outputs are read from
        bufs.hgu; otherwise the gate+up GEMM runs again (into bwd.gu).
        Returns the BackwardBuffers: dx_total (the input gradient), dx (its
        expert-path part), dw (gate weights), dC (centroids), dW_gu, dW_dn.
        keep_intermediates: also write the bf16 dGU and h (bwd.dgu, bwd.h),
        which the step itself does not need (its GEMMs read their codes).
        `events` as in forward, keys "combine_bwd", "dgrad_down",
        "recompute_gate_up", "swiglu_bwd", "dgrad_gate_up", "unpermute",
        "wgrad_down", "wgrad_gate_up", "router_bwd"."""
        self._check_backward(seq_len)
        s = self.shape
        T = dy_bf16.shape[0]
        b = bufs or self.buffers(T)
        self._check_rows(b, dy_bf16, x_bf16)
        self._check_seq_len(b, seq_len)
        bb = bwd or self.backward_buffers(T)
        if bb.T != T:
            raise ValueError(f"backward buffers of {bb.T} tokens for {T}")
        if keep_intermediates:
            bb.intermediates()
        st = stream if stream is not None else torch.cuda.current_stream()

        def step(name, fn):
            if events is None:
                fn()
                return
            e0 = torch.cuda.Event(enable_timing=True)
            e1 = torch.cuda.Event(enable_timing=True)
            e0.record(st)
            fn()
            e1.record(st)
            events.setdefault(name, []).append((e0, e1))

        # the combine and SwiGLU backward also write the 1x128 quantisation of
        # their bf16 gradients (the input-gradient GEMMs' operands)
        step("combine_bwd", lambda: L.moe_combine_backward(
            dy_bf16, b.inv_perm, b.topk_w, b.d, T, s.k, s.H, s.n_shared, bb.dD, bb.dw, st,
            d_expert_out_e4m3=bb.dDq, d_expert_out_scale=bb.dDs))
        self._experts_backward(x_bf16, b, bb, keep_intermediates, st, step)
        self._router_backward(x_bf16, b, bb, seq_len, alpha, st, step)
        return bb

    def _experts_backward(self, x_bf16, b, bb, keep_intermediates, st, step):
        """From the gradient of the experts' rows in bb to their input's (bb.dx)
        and the weights'."""
        s, T = self.shape, b.T
        R, G, H, I, k, cap = b.R, s.G, s.H, s.I, s.k, bb.cap
        step("dgrad_down", lambda: L.grouped_fp8_gemm_dgrad(
            bb.dDq, bb.dDs, self.w_dn, self.w_dn_s, b.offsets, G, R, H, I, bb.dh, st))
        if b.held is not None and b.held.gu:
            gu = b.hgu   # kept by the forward (keep_gu): the same bf16 GEMM output
        else:
            gu = bb.gu
            step("recompute_gate_up", lambda: L.grouped_fp8_gemm(
                b.xq, b.xs, b.perm_src, self.w_gu, self.w_gu_s, b.offsets, G, R, 2 * I, H, gu,
                st))
        # the SwiGLU backward also writes dGU's 1x128 codes and the 128x1 chunk
        # codes of dGU and h that the input and weight gradients read
        step("swiglu_bwd", lambda: L.swiglu_backward_grouped(
            gu, bb.dh, b.offsets, G, R, I, bb.dgu if keep_intermediates else None,
            bb.h if keep_intermediates else None, bb.dguq, bb.dgus, cap, bb.c_dgu,
            bb.s_dgu, bb.c_h, bb.s_h, st))
        step("dgrad_gate_up", lambda: L.grouped_fp8_gemm_dgrad(
            bb.dguq, bb.dgus, self.w_gu, self.w_gu_s, b.offsets, G, R, 2 * I, H, bb.dxp, st))
        step("unpermute", lambda: self._unpermute(b, bb, st))
        step("wgrad_down", lambda: (
            L.fp8_quant_128x1_grouped(bb.dD, H, None, b.offsets, G, R, H, bb.c_dD, bb.s_dD, cap, st),
            L.grouped_fp8_wgrad(bb.c_dD, bb.s_dD, bb.c_h, bb.s_h, cap, b.offsets, G, R, H, I,
                                bb.dW_dn, st)))
        step("wgrad_gate_up", lambda: (
            L.fp8_quant_128x1_grouped(x_bf16, H, b.perm_src, b.offsets, G, R, H, bb.c_x, bb.s_x,
                                      cap, st),
            L.grouped_fp8_wgrad(bb.c_dgu, bb.s_dgu, bb.c_x, bb.s_x, cap, b.offsets, G, R, 2 * I, H,
                                bb.dW_gu, st)))

    def _unpermute(self, b, bb, st):
        s, T = self.shape, b.T
        shared = bb.dxp[T * s.k:T * s.k + T] if s.n_shared else None
        L.moe_combine(bb.dxp, b.inv_perm, bb.ones, shared, T, s.k, s.H, bb.dx, st)

    def _router_backward(self, x_bf16, b, bb, seq_len, alpha, st, step):
        """The router's part on top of bb.dx: bb.dx_total and bb.dC."""
        s, T = self.shape, b.T
        H, k = s.H, s.k
        if self.gate is not None:
            g = self.gate
            bb.dense()
            step("router_bwd", lambda: (
                L.moe_gate_backward(b.logits, T, s.E, g.score, k, g.renormalize, g.scale, b.topk_idx,
                                    bb.dw, bb.dlogit[:T], st),
                L.moe_router_logits_backward(x_bf16, self.centroids, bb.dlogit[:T], T, H, s.E, bb.dx,
                                             bb.dx_total, bb.dC, bb.dense_ws, bb.dense_ws_bytes,
                                             st)))
        elif seq_len is None:
            step("router_bwd", lambda: (
                L.moe_router_backward(x_bf16, self.centroids, b.topk_idx, bb.dw, b.inv_perm, bb.dx,
                                      T, H, s.E, k, bb.dx_total, bb.dlogit_rows, st,
                                      topk_s=b.topk_s),
                L.moe_router_dcentroids(x_bf16, b.perm_src, b.offsets, bb.dlogit_rows, T, H, s.E,
                                        bb.dC, st)))
        else:
            b.balance(seq_len)   # (the names may hold another's)
            bb.dense()
            step("router_bwd", lambda: L.moe_router_backward_dense(
                x_bf16, self.centroids, b.topk_idx, bb.dw, b.scores, b.score_sums, b.seq_f, T, H,
                s.E, k, seq_len, alpha, bb.dx, bb.dx_total, bb.dC, bb.dlogit, bb.dense_ws,
                bb.dense_ws_bytes, st))

    def _check_backward(self, seq_len):
        self._check_gate(seq_len)
        if self.gate is not None and self.shape.E % 16:
            raise ValueError(f"the backward of a layer with a Gate needs E % 16 == 0, E is {self.shape.E}")

    def _check_rows(self, b, *tensors):
        """The layer's inputs, before anything is launched: the kernels take
        their sizes from the shape."""
        for t in tensors:
            if t.dim() != 2 or t.shape != (b.T, self.shape.H):
                raise ValueError(f"{list(t.shape)} in buffers of [T, H] = [{b.T}, {self.shape.H}]")
        dev = L._device()
        for t in tensors:
            L._ptr(t, torch.bfloat16, dev)

    @staticmethod
    def _check_seq_len(b, seq_len):
        if seq_len is not None and (b.held is None or b.held.seq_len != seq_len):
            raise ValueError("backward with seq_len needs the forward run with the same seq_len")

    def _check_gate(self, seq_len):
        """What a layer with a Gate does not do, before anything is launched."""
        if self.gate is not None and seq_len is not None:
            raise ValueError("the sequence-wise balance term needs moe_route's scores: no Gate")

    def _route(self, x_bf16, b, seq_len, stream):
        s = self.shape
        T = x_bf16.shape[0]
        if self.gate is not None:
            g = self.gate
            L.moe_router_logits(x_bf16, T, s.H, self.centroids, s.E, b.logits, b.route_ws,
                                b.route_ws_bytes, stream)
            L.moe_gate(b.logits, T, s.E, self.bias if g.use_bias else None, g.score, s.n_group,
                       s.topk_group, g.group_top, s.k, g.renormalize, g.scale, b.topk_idx, b.topk_w,
                       b.counts, stream)
        elif seq_len is None:
            L.moe_route(x_bf16, T, s.H, self.centroids, self.bias, s.E, s.n_group, s.topk_group,
                        s.k, b.topk_idx, b.topk_w, b.counts, b.route_ws, b.route_ws_bytes, stream,
                        topk_s=b.topk_s)
        else:
            b.balance(seq_len)
            L.moe_route_scores(x_bf16, T, s.H, self.centroids, self.bias, s.E, s.n_group,
                               s.topk_group, s.k, b.topk_idx, b.topk_w, b.counts, b.route_ws,
                               b.route_ws_bytes, b.scores, b.score_sums, stream, topk_s=b.topk_s)

    def _seq_balance(self, b, seq_len, alpha, stream):
        s = self.shape
        L.moe_seq_balance(b.scores, b.score_sums, b.topk_idx, b.T, s.E, s.k, seq_len, alpha,
                          b.seq_f, b.seq_p, b.seq_loss, b.seq_ws, b.seq_ws_bytes, stream)


class Int8Buffers(Buffers):
    """Device buffers of one int8 forward at T tokens (reused across calls)."""

    def _operands(self):
        """x in 8-bit integers with a scale for each token; h in bf16, then as x."""
        s, T, R, dev = self._shape, self.T, self.R, self._dev
        i8, f32 = torch.int8, torch.float32
        self.xq = torch.empty((T, s.H), dtype=i8, device=dev)
        self.xs = torch.empty((T,), dtype=f32, device=dev)
        self.h = torch.empty((R, s.I), dtype=torch.bfloat16, device=dev)
        self.hq = torch.empty((R, s.I), dtype=i8, device=dev)
        self.hs = torch.empty((R,), dtype=f32, device=dev)


class Int8MoELayer(MoELayer):
    """The layer's forward with expert weights and activations in 8-bit integers.

      w_gu [G, 2I, H] int8 (rows [0, I) gate, [I, 2I) up), w_gu_s [G, 2I] fp32
      w_dn [G, H, I],                                       w_dn_s [G, H]
    Built by from_fp32_experts like MoELayer; inference only.
    """
    CODES = L.QUANT_INT8

    @staticmethod
    def empty_weights(shape: LayerShape, device="cuda"):
        s, dev = shape, torch.device(device)
        return (torch.empty((s.G, 2 * s.I, s.H), dtype=torch.int8, device=dev),
                torch.empty((s.G, 2 * s.I), dtype=torch.float32, device=dev),
                torch.empty((s.G, s.H, s.I), dtype=torch.int8, device=dev),
                torch.empty((s.G, s.H), dtype=torch.float32, device=dev))

    @staticmethod
    def quantize_into(w_f32, out_q, out_s, stream=None):
        """Quantisation of fp32 weights [G', N, K], one scale an output channel."""
        _check_weights(w_f32, out_q)
        G, N, K = w_f32.shape
        L.int8_quant_channels(w_f32, G, N, K, out_q, out_s, stream)

    def buffers(self, T: int) -> Int8Buffers:
        b = self._bufs.get(T)
        if b is None:
            b = self._bufs[T] = Int8Buffers(self.shape, T, self.centroids.device)
        return b

    @_on_stream
    def forward(self, x_bf16: torch.Tensor, bufs: Int8Buffers | None = None, stream=None,
                update_bias: bool = False, gamma: float = 0.001) -> torch.Tensor:
        """One layer forward (x's quantisation beside the router, as in
        MoELayer.forward)."""
        s = self.shape
        T = x_bf16.shape[0]
        b = bufs or self.buffers(T)
        self._check_rows(b, x_bf16)
        st = stream if stream is not None else torch.cuda.current_stream()
        if self._side is None:
            self._side = torch.cuda.Stream(device=st.device)
        side = self._side
        b.held = None
        side.wait_stream(st)
        self._quantise(x_bf16, b, side)
        self._route(x_bf16, b, None, st)
        self._permute(b, st)
        st.wait_stream(side)
        self._experts(x_bf16, b, False, st, _run)
        shared = b.d[T * s.k:T * s.k + T] if s.n_shared else None
        L.moe_combine(b.d, b.inv_perm, b.topk_w, shared, T, s.k, s.H, b.y, st)
        if update_bias:
            L.moe_bias_update(b.counts, self.bias, s.E, gamma, st)
        b.held = Held(False)
        return b.y

    def _quantise(self, x_bf16, b, stream):
        H = self.shape.H
        L.int8_quant_rows(x_bf16, x_bf16.shape[0], H, H, b.xq, b.xs, stream)

    def _experts(self, x_bf16, b, keep_gu, st, step):
        s, R = self.shape, b.R
        L.grouped_int8_gemm_swiglu(b.xq, b.xs, b.perm_src, self.w_gu, self.w_gu_s, b.offsets, s.G,
                                   R, s.I, s.H, b.h, st)
        L.int8_quant_rows(b.h, R, s.I, s.I, b.hq, b.hs, st)
        L.grouped_int8_gemm(b.hq, b.hs, None, self.w_dn, self.w_dn_s, b.offsets, s.G, R, s.H, s.I,
                            b.d, st)

    def backward(self, *args, **kw):
        raise NotImplementedError("Int8MoELayer is a forward only: train with MoELayer")


class Bf16Buffers(Buffers):
    """Device buffers of one bf16 forward at T tokens (reused across calls)."""

    def _operands(self):
        """h in bf16 (x is read as it is)."""
        self.h = torch.empty((self.R, self._shape.I), dtype=torch.bfloat16, device=self._dev)


class Bf16BackwardBuffers(BackwardBuffers):
    """Device buffers of one bf16 layer backward at T tokens (reused across calls)."""

    def _operands(self):
        self.dgu = torch.empty((self.R, 2 * self._shape.I), dtype=torch.bfloat16, device=self._dev)
        self.dDq = self.dDs = self._gu = self.h = None

    @property
    def gu(self):
        """Gate and up outputs formed again, after a forward that kept none
        (allocated on first use)."""
        if self._gu is None:
            self._gu = torch.empty_like(self.dgu)
        return self._gu


class Bf16MoELayer(MoELayer):
    """The layer with its expert weights and activations in bf16, forward and
    backward: for training or checking without quantisation.

      w_gu [G, 2I, H] bf16 (rows [0, I) gate, [I, 2I) up), w_dn [G, H, I]
    act: the gate's activation, ACT_SILU or ACT_GELU.  Built by
    from_fp32_experts like MoELayer (the fp32 weights are rounded to bf16).
    """
    CODES = L.QUANT_NONE

    def __init__(self, shape: LayerShape, centroids, bias, w_gu, w_gu_s, w_dn, w_dn_s,
                 gate: Gate | None = None, act: int = L.ACT_SILU):
        super().__init__(shape, centroids, bias, w_gu, w_gu_s, w_dn, w_dn_s, gate)
        self.act = act

    @staticmethod
    def empty_weights(shape: LayerShape, device="cuda"):
        """w_gu, None, w_dn, None: bf16 weights have no scales."""
        s, dev = shape, torch.device(device)
        return (torch.empty((s.G, 2 * s.I, s.H), dtype=torch.bfloat16, device=dev), None,
                torch.empty((s.G, s.H, s.I), dtype=torch.bfloat16, device=dev), None)

    @staticmethod
    def quantize_into(w_f32, out_q, out_s=None, stream=None):
        """fp32 weights rounded to bf16."""
        _check_weights(w_f32, out_q)
        st = stream if stream is not None else torch.cuda.current_stream()
        with torch.cuda.stream(st):
            out_q.copy_(w_f32)

    def buffers(self, T: int) -> Bf16Buffers:
        b = self._bufs.get(T)
        if b is None:
            b = self._bufs[T] = Bf16Buffers(self.shape, T, self.centroids.device)
        return b

    def backward_buffers(self, T: int) -> Bf16BackwardBuffers:
        bb = self._bwd.get(T)
        if bb is None:
            bb = self._bwd[T] = Bf16BackwardBuffers(self.shape, T, self.centroids.device)
        return bb

    def _quantise(self, x_bf16, b, stream):
        pass

    def _experts(self, x_bf16, b, keep_gu, st, step):
        s, R = self.shape, b.R
        step("gate_up", st, lambda: L.grouped_bf16_gemm_glu(
            x_bf16, b.perm_src, self.w_gu, b.offsets, s.G, R, s.I, s.H, self.act, b.h,
            b.hgu if keep_gu else None, st))
        step("down", st, lambda: L.grouped_bf16_gemm(b.h, None, self.w_dn, b.offsets, s.G, R, s.H, s.I, b.d,
                                                     st))

    def _experts_backward(self, x_bf16, b, bb, keep_intermediates, st, step):
        s = self.shape
        R, G, H, I = b.R, s.G, s.H, s.I
        if keep_intermediates:   # (dGU and h are the products' own operands)
            bb.h = b.h
        if b.held is not None and b.held.gu:
            gu = b.hgu
        else:
            gu = bb.gu
            step("recompute_gate_up", lambda: L.grouped_bf16_gemm(
                x_bf16, b.perm_src, self.w_gu, b.offsets, G, R, 2 * I, H, gu, st))
        # the down projection's input gradient and the activation's backward
        step("dgrad_down", lambda: L.grouped_bf16_gemm_dgrad_glu(
            bb.dD, self.w_dn, gu, b.offsets, G, R, H, I, self.act, bb.dgu, st))
        step("dgrad_gate_up", lambda: L.grouped_bf16_gemm_dgrad(
            bb.dgu, self.w_gu, b.offsets, G, R, 2 * I, H, bb.dxp, st))
        step("unpermute", lambda: self._unpermute(b, bb, st))
        step("wgrad_down", lambda: L.grouped_bf16_wgrad(
            bb.dD, b.h, None, b.offsets, G, R, H, I, bb.dW_dn, st))
        step("wgrad_gate_up", lambda: L.grouped_bf16_wgrad(
            bb.dgu, x_bf16, b.perm_src, b.offsets, G, R, 2 * I, H, bb.dW_gu, st))


class BlockBuffers:
    """Device buffers of a MoEBlock at T tokens of the residual stream's type
    (reused across calls)."""

    def __init__(self, shape: LayerShape, T: int, dtype, device="cuda"):
        dev, f32 = torch.device(device), torch.float32
        self.T, self.H, self.dtype, self._dev = T, shape.H, dtype, dev
        self.n = torch.empty((T, shape.H), dtype=torch.bfloat16, device=dev)
        self.rstd = torch.empty((T,), dtype=f32, device=dev)
        self.y = torch.empty((T, shape.H), dtype=dtype, device=dev)
        self._sum = self.dx = None

    @property
    def sum(self):
        """The residual stream after a forward's add (allocated on first use)."""
        if self._sum is None:
            self._sum = torch.empty_like(self.y)
        return self._sum

    def gradients(self):
        """Buffers of the backward (allocated on first use): dx [T, H],
        d_weight, d_post_weight [H], d_shared_w [T] and the workspace."""
        if self.dx is None:
            dev, f32 = self._dev, torch.float32
            self.dx = torch.empty_like(self.y)
            self.d_weight = torch.empty((self.H,), dtype=f32, device=dev)
            self.d_post_weight = torch.empty((self.H,), dtype=f32, device=dev)
            self.d_shared_w = torch.empty((self.T,), dtype=f32, device=dev)
            self.ws_bytes = max(L.moe_norm_backward_workspace_bytes(self.T, self.H),
                                L.moe_combine_norm_backward_workspace_bytes(self.T, self.H))
            self.ws = torch.empty((max(16, self.ws_bytes),), dtype=torch.uint8, device=dev)
        return self


class MoEBlock:
    """A layer between its norms, on the residual stream (bf16 or fp32):

      v = x + add (or x);  n = norm(v) * weight
      y = residual_scale * v + scale * [norm](layer(n)) * post_weight

    moe_norm writes the experts' operand beside n, and moe_combine_norm takes
    the layer's combine with the norm after it and the residual sum, so neither
    is a pass of its own.  layer: a MoELayer, Bf16MoELayer or Int8MoELayer.
    post_norm: norm the layer's output; without it post_weight (optional)
    scales its channels.  Weights are fp32 [H]."""

    def __init__(self, layer: MoELayer, weight=None, eps: float = 1e-6, post_norm: bool = False,
                 post_weight=None, residual_scale: float = 1.0, scale: float = 1.0):
        for w in (weight, post_weight):
            if w is None:
                continue
            if w.shape != (layer.shape.H,):
                raise ValueError(f"a norm's weight has the shape [H] = [{layer.shape.H}], not {list(w.shape)}")
            if L._ptr(w, torch.float32, layer.centroids.get_device()) % 16:
                raise ValueError("a norm's weight must be 16-byte aligned")
        self.layer, self.weight, self.eps = layer, weight, eps
        self.post_norm, self.post_weight = post_norm, post_weight
        self.residual_scale, self.scale = residual_scale, scale
        self._bufs = {}

    def buffers(self, T: int, dtype) -> BlockBuffers:
        key = (T, dtype)
        if key not in self._bufs:
            self._bufs[key] = BlockBuffers(self.layer.shape, T, dtype, self.layer.centroids.device)
        return self._bufs[key]

    def _check(self, x, add, shared_w):
        """All that a call refuses of its tensors, before anything is launched."""
        H, dev = self.layer.shape.H, L._device()
        if x.dim() != 2 or x.shape[1] != H or (add is not None and add.shape != x.shape):
            raise ValueError(f"x {list(x.shape)}{'' if add is None else f' and add {list(add.shape)}'}: not [T, {H}]")
        if shared_w is not None and shared_w.shape != (x.shape[0],):
            raise ValueError(f"shared_w {list(shared_w.shape)}: not [{x.shape[0]}]")
        if shared_w is not None and not self.layer.shape.n_shared:
            raise ValueError("shared_w of a layer without a shared expert")
        L._logits_type(x, "x")
        L._ptr(x, None, dev), L._ptr(add, torch.bfloat16, dev), L._ptr(shared_w, torch.float32, dev)

    @_on_stream
    def forward(self, x, add=None, shared_w=None, stream=None, update_bias: bool = False,
                gamma: float = 0.001, seq_len: int | None = None, alpha: float = 0.0001,
                keep_gu: bool = False) -> torch.Tensor:
        """One block forward of x [T, H] (fp32 or bf16), with add [T, H] bf16
        added to the stream first.  shared_w [T] fp32: the shared expert's own
        gate.  The rest as in the layer's forward.  Returns y in the buffers of
        this T and type (buffers(T, x.dtype).sum holds v after an add)."""
        layer, s = self.layer, self.layer.shape
        layer._check_gate(seq_len)
        self._check(x, add, shared_w)
        if keep_gu and isinstance(layer, Int8MoELayer):
            raise ValueError("keep_gu is for the backward, which an Int8MoELayer does not have")
        T = x.shape[0]
        f, b = self.buffers(T, x.dtype), layer.buffers(T)
        st = stream if stream is not None else torch.cuda.current_stream()
        v = f.sum if add is not None else x
        codes, scales = (None, None) if layer.CODES == L.QUANT_NONE else (b.xq, b.xs)
        L.moe_norm(x, add, self.weight, T, s.H, self.eps, None if add is None else v, f.n, f.rstd, layer.CODES,
                   codes, scales, st)
        b.held = None
        layer._route(f.n, b, seq_len, st)
        if seq_len is not None:
            layer._seq_balance(b, seq_len, alpha, st)
        layer._permute(b, st)
        layer._experts(f.n, b, keep_gu, st, _run)
        shared = b.d[T * s.k:T * s.k + T] if s.n_shared else None
        L.moe_combine_norm(b.d, b.inv_perm, b.topk_w, shared, shared_w, v, self.residual_scale, self.post_norm,
                           self.post_weight, self.eps, self.scale, T, s.k, s.H, f.y, None, st)
        if update_bias:
            L.moe_bias_update(b.counts, layer.bias, s.E, gamma, st)
        b.held = Held(keep_gu, seq_len, f, add is not None, shared_w is not None)
        return f.y

    @_on_stream
    def backward(self, dy, x, shared_w=None, stream=None, seq_len: int | None = None,
                 alpha: float = 0.0001):
        """Backward for the output gradient dy (x's type) of the last forward of
        the layer at this T, which has to be this block's of x (with the same
        shared_w and seq_len): what a forward leaves for it lies in the layer's
        buffers, so that batches in flight together, or another type's of the
        same T, need a layer each.  Returns (the block's buffers, the
        layer's backward buffers): dx - the gradient of x and of add alike -,
        d_weight (with a weight), d_post_weight (with a post_weight) and
        d_shared_w (with shared_w); dC, dW_gu, dW_dn, dw of the layer."""
        layer, s = self.layer, self.layer.shape
        if isinstance(layer, Int8MoELayer):
            layer.backward()
        layer._check_backward(seq_len)
        if dy.dtype != x.dtype or dy.shape != x.shape:
            raise ValueError(f"dy {tuple(dy.shape)} {dy.dtype} and x {tuple(x.shape)} {x.dtype} differ")
        self._check(x, None, shared_w)
        L._ptr(dy, None, L._device())
        if dy.data_ptr() % 16 or x.data_ptr() % 16:
            raise ValueError("dy and x must be 16-byte aligned")
        T = dy.shape[0]
        f, b = self.buffers(T, dy.dtype), layer.buffers(T)
        held = b.held
        if held is None or held.block is not f:
            raise ValueError(f"backward of {T} tokens in {dy.dtype} before a forward of them, or after another forward "
                             "on the layer's buffers")
        if held.gated != (shared_w is not None):
            raise ValueError(f"backward {'without' if held.gated else 'with'} shared_w of a forward "
                             f"{'with' if held.gated else 'without'} it")
        layer._check_seq_len(b, seq_len)
        if T and not held.added and x.data_ptr() == f.y.data_ptr():
            raise ValueError("x is the block's own y, which the forward has written over: pass a copy of it to both")
        f, bb = f.gradients(), layer.backward_buffers(T)
        written = (bb.dx.data_ptr(), bb.dx_total.data_ptr(), bb.dD.data_ptr(), bb.dxp.data_ptr())
        if T and (dy.data_ptr() in written or x.data_ptr() in written):
            raise ValueError("dy and x are read after the layer's backward buffers are written: pass copies of these")
        st = stream if stream is not None else torch.cuda.current_stream()
        weighted = self.post_weight is not None
        L.moe_combine_norm_backward(
            dy, b.inv_perm, b.topk_w, b.d, s.n_shared, shared_w, self.post_norm, self.post_weight, self.eps,
            self.scale, T, s.k, s.H, bb.dD, bb.dw, f.d_shared_w if shared_w is not None else None, bb.dDq, bb.dDs,
            f.d_post_weight if weighted else None, f.ws, f.ws_bytes, st)
        layer._experts_backward(f.n, b, bb, False, st, _run)
        layer._router_backward(f.n, b, bb, seq_len, alpha, st, _run)
        L.moe_norm_backward(bb.dx_total, f.sum if held.added else x, self.weight, f.rstd, dy, self.residual_scale, T,
                            s.H, f.dx, f.d_weight if self.weight is not None else None, f.ws, f.ws_bytes, st)
        return f, bb

    def capture(self, x, add=None, **forward_kw):
        """One forward captured as a HIP graph on the buffers of this T and type,
        as MoELayer.capture."""
        side = torch.cuda.Stream()   # default priority
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.forward(x, add, stream=side, **forward_kw)   # warm-up outside the capture
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = CapturedForward()
        with torch.cuda.graph(graph):
            self.forward(x, add, stream=torch.cuda.current_stream(), **forward_kw)
        graph.bufs = self.layer.buffers(x.shape[0])
        graph.held = graph.bufs.held
        return graph
