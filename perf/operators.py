"""Cases, plain forms and calls of the gate and the 8-bit-integer expert operators.

Operators:
  gate            moe_gate: softmax or sigmoid scores of given router logits, an
                  optional bias for the choice only, group-limited top-k,
                  optionally renormalised and scaled weights, expert counts
  gate_backward   moe_gate_backward: the gradient of those weights (and of the
                  dense scores) with respect to the logits
  quant_rows      int8_quant_rows: bf16 activations to int8, one scale a token
  quant_channels  int8_quant_channels: fp32 weights to int8, one scale an
                  output channel
  gemm            grouped_int8_gemm: the experts' product with both scales
  swiglu          grouped_int8_gemm_swiglu: gate+up product and SwiGLU

The plain forms use elementary torch operations in 32 bits, and in 64 where a
choice hangs on values next to each other: the order of the experts and the
rounding of a quotient to a whole number.
"""
import math

import torch

own = False

SOFTMAX, SIGMOID = 0, 1


def listed():
    return [
        # one decode step of 128 sequences: biased sigmoid scores, 4 of 8 groups
        dict(name="gate decode", op="gate", T=128, E=256, type="f32", score=SIGMOID, bias=True,
             n_group=8, topk_group=4, group_top=2, k=8, renorm=True, scale=2.5, scores=False),
        # a prefill or training batch: softmax scores kept for a balance loss
        dict(name="gate prefill", op="gate", T=16384, E=256, type="f32", score=SOFTMAX, bias=False,
             n_group=1, topk_group=1, group_top=1, k=8, renorm=False, scale=1.0, scores=True),
        # the training step's gradient, a dense loss on the scores among it
        dict(name="gate backward train", op="gate_backward", T=16384, E=256, type="f32",
             score=SOFTMAX, k=8, renorm=True, scale=1.0, d_scores=True),
        # a short odd batch of a smaller layer with bf16 logits
        dict(name="gate backward odd", op="gate_backward", T=1031, E=60, type="bf16",
             score=SIGMOID, k=4, renorm=False, scale=1.5, d_scores=False),
        # activations of one decode step, and of a prefill's expert rows
        dict(name="quant rows decode", op="quant_rows", M=128, K=7168, ld=7168),
        dict(name="quant rows prefill", op="quant_rows", M=147456, K=2048, ld=2048),
        # an odd number of experts' weights, quantised when a model is loaded
        dict(name="quant channels", op="quant_channels", G=33, N=4096, K=7168),
        # one token through one dense matrix: latency
        dict(name="gemm one token", op="gemm", T=1, groups=1, k=1, shared=False, N=4096, K=7168),
        # down projections of 256 experts and the shared one, decode and prefill
        dict(name="gemm down decode", op="gemm", T=128, groups=256, k=8, shared=True, N=7168, K=2048),
        dict(name="gemm down prefill", op="gemm", T=16384, groups=256, k=8, shared=True, N=7168, K=2048),
        # gate and up projections with SwiGLU: decode, and a ragged middle-sized batch
        dict(name="swiglu decode", op="swiglu", T=128, groups=256, k=8, shared=True, N=2048, K=7168),
        dict(name="swiglu ragged", op="swiglu", T=4099, groups=64, k=6, shared=True, N=1416, K=7152),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_backward", "quant_rows", "quant_channels", "gemm", "gemm",
                     "swiglu", "swiglu"])
    if op in ("gate", "gate_backward"):
        c = dict(op=op, T=_log(rng, 1, 16384), type=rng.choice(["f32", "bf16"]),
                 score=rng.choice([SOFTMAX, SIGMOID]), renorm=rng.random() < 0.5,
                 scale=rng.choice([1.0, 1.5, 2.5]))
        if op == "gate_backward":
            c["E"] = rng.randint(2, 512)
            c["k"] = rng.randint(1, min(8, c["E"]))
            c["d_scores"] = rng.random() < 0.5
            return c
        c["n_group"] = rng.choice([1, 1, 2, 4, 5, 8])
        c["E"] = c["n_group"] * rng.randint(2, 512 // c["n_group"])
        c["topk_group"] = rng.randint((c["n_group"] + 1) // 2, c["n_group"])
        c["group_top"] = rng.choice([1, 2])
        c["k"] = rng.randint(1, min(8, c["topk_group"] * (c["E"] // c["n_group"])))
        c["bias"], c["scores"] = rng.random() < 0.6, rng.random() < 0.4
        return c
    if op == "quant_rows":
        K = 8 * rng.randint(1, 1024)
        return dict(op=op, M=_log(rng, 1, 30000), K=K, ld=K + 8 * rng.choice([0, 0, 3]))
    if op == "quant_channels":
        return dict(op=op, G=_log(rng, 1, 32), N=rng.randint(1, 4096), K=8 * rng.randint(1, 896))
    groups = _log(rng, 1, 128)
    return dict(op=op, T=_log(rng, 1, 3500), groups=groups, k=rng.randint(1, min(8, groups)),
                shared=rng.random() < 0.5, N=8 * rng.randint(4, 512), K=16 * rng.randint(2, 440))


# ---- inputs ------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _int8_normal(shape, sigma, g):
    """Codes of normal values scaled to int8, made a few matrices at a time."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").mul_(sigma).round_().clamp_(-127, 127)
    return out


def prepare(case, seed):
    c, g = case, _gen(seed)
    dev = dict(device="cuda")
    op = c["op"]
    s = dict(case=c)
    if op in ("gate", "gate_backward"):
        T, E, k = c["T"], c["E"], c["k"]
        dtype = torch.float32 if c["type"] == "f32" else torch.bfloat16
        s["logits"] = (torch.randn((T, E), generator=g, **dev) * 1.7).to(dtype)
        if op == "gate":
            lim = 0.01 if c["score"] == SIGMOID else 0.5 / E
            s["bias"] = (torch.rand(E, generator=g, **dev) * 2 - 1) * lim if c["bias"] else None
            s["idx"] = torch.empty((T, k), dtype=torch.int32, **dev)
            s["w"] = torch.empty((T, k), **dev)
            s["counts"] = torch.empty(E, dtype=torch.int32, **dev)
            s["scores"] = torch.empty((T, E), **dev) if c["scores"] else None
        else:
            s["idx"] = s["logits"].float().topk(k).indices.sort().values.to(torch.int32)
            s["dw"] = torch.randn((T, k), generator=g, **dev)
            s["ds"] = torch.randn((T, E), generator=g, **dev) * 0.01 if c["d_scores"] else None
            s["dl"] = torch.empty((T, E), dtype=dtype, **dev)
    elif op == "quant_rows":
        M, K, ld = c["M"], c["K"], c["ld"]
        row = torch.exp(torch.randn((M, 1), generator=g, **dev))  # tokens of different sizes
        s["x"] = (torch.randn((M, ld), generator=g, **dev) * row).to(torch.bfloat16)
        s["q"] = torch.empty((M, K), dtype=torch.int8, **dev)
        s["s"] = torch.empty(M, **dev)
    elif op == "quant_channels":
        G, N, K = c["G"], c["N"], c["K"]
        s["w"] = torch.randn((G, N, K), generator=g, **dev) * 0.02
        s["q"] = torch.empty((G, N, K), dtype=torch.int8, **dev)
        s["s"] = torch.empty((G, N), **dev)
    else:
        T, E, k, K = c["T"], c["groups"], c["k"], c["K"]
        G = E + c["shared"]
        N = c["N"] * (2 if op == "swiglu" else 1)
        # some experts are more popular than others; each token has k of them
        like = torch.rand((T, E), generator=g, **dev) + 0.3 * torch.rand(E, generator=g, **dev)
        expert = like.topk(k).indices.sort().values.reshape(-1)
        order = expert.sort(stable=True).indices
        counts = torch.bincount(expert, minlength=E)
        source = order // k
        if c["shared"]:
            counts = torch.cat([counts, torch.tensor([T], **dev)])
            source = torch.cat([source, torch.arange(T, **dev)])
        s["rows"] = int(source.numel())
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, **dev), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts[:E].max())  # a host program knows a bound of its batch
        s["index"] = source.to(torch.int32) if op == "swiglu" else None
        a_rows = T if op == "swiglu" else s["rows"]
        s["a"] = _int8_normal((a_rows, K), 31.0, g)
        s["sa"] = torch.exp(torch.randn(a_rows, generator=g, **dev) * 0.5) * 0.03
        s["b"] = _int8_normal((G, N, K), 33.0, g)
        s["sb"] = (0.5 + torch.rand((G, N), generator=g, **dev)) * (1.0 / (33.0 * math.sqrt(K)))
        s["out"] = torch.empty((s["rows"], c["N"]), dtype=torch.bfloat16, **dev)
    return s


# ---- one pass ------------------------------------------------------------------

def run(state):
    if own:
        return _call(state)
    return _PLAIN[state["case"]["op"]](state)


def _call(s):
    import fp8_block_scaled_bias_amd as M
    c = s["case"]
    op = c["op"]
    if op == "gate":
        M.moe_gate(s["logits"], c["T"], c["E"], s["bias"], c["score"], c["n_group"], c["topk_group"],
                   c["group_top"], c["k"], c["renorm"], c["scale"], s["idx"], s["w"], s["counts"],
                   scores=s["scores"])
        return dict(idx=s["idx"], w=s["w"], counts=s["counts"], scores=s["scores"])
    if op == "gate_backward":
        M.moe_gate_backward(s["logits"], c["T"], c["E"], c["score"], c["k"], c["renorm"], c["scale"],
                            s["idx"], s["dw"], s["dl"], d_scores=s["ds"])
        return dict(d_logits=s["dl"])
    if op == "quant_rows":
        M.int8_quant_rows(s["x"], c["M"], c["K"], c["ld"], s["q"], s["s"])
        return dict(codes=s["q"], scale=s["s"])
    if op == "quant_channels":
        M.int8_quant_channels(s["w"], c["G"], c["N"], c["K"], s["q"], s["s"])
        return dict(codes=s["q"], scale=s["s"])
    G = c["groups"] + c["shared"]
    fn = M.grouped_int8_gemm_swiglu if op == "swiglu" else M.grouped_int8_gemm
    fn(s["a"], s["sa"], s["index"], s["b"], s["sb"], s["offsets"], G, s["rows"], c["N"], c["K"], s["out"])
    return dict(out=s["out"])


def _scores(logits, score):
    if score == SIGMOID:
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    return e / e.sum(dim=1, keepdim=True)


def _gate(s):
    c, bias = s["case"], s["bias"]
    T, E, k, n = c["T"], c["E"], c["k"], c["n_group"]
    scores = _scores(s["logits"].float(), c["score"])
    wide = s["logits"].double()
    if n > 1 or bias is not None:
        exact = _scores(wide, c["score"])
        if bias is not None:
            exact = exact + bias.double()
    key = wide if bias is None else exact  # a score grows with its logit
    if n > 1:
        group = (exact if c["group_top"] == 2 else key).view(T, n, E // n)
        group = group.sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(dim=2)
        first = group.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        kept = torch.zeros((T, n), dtype=torch.bool, device="cuda").scatter_(1, first, True)
        key = torch.where(kept.repeat_interleave(E // n, dim=1), key, -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k].sort(dim=1).values
    w = scores.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    counts.index_add_(0, idx.reshape(-1), torch.ones(T * k, dtype=torch.int32, device="cuda"))
    return dict(idx=idx.to(torch.int32), w=w * c["scale"], counts=counts,
                scores=scores if c["scores"] else None)


def _gate_backward(s):
    c, idx = s["case"], s["idx"].long()
    p = _scores(s["logits"].float(), c["score"])
    chosen, dw = p.gather(1, idx), s["dw"] * c["scale"]
    if c["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        dw = (dw - (dw * chosen / total).sum(dim=1, keepdim=True)) / total
    ds = torch.zeros_like(p) if s["ds"] is None else s["ds"].clone()
    ds.scatter_add_(1, idx, dw)
    if c["score"] == SIGMOID:
        dl = ds * p * (1 - p)
    else:
        dl = p * (ds - (ds * p).sum(dim=1, keepdim=True))
    return dict(d_logits=dl.to(s["dl"].dtype))


def _quantise(v):
    """Along the last axis; the quotient in 64 bits, where its rounding is decided."""
    scale = (v.abs().amax(dim=-1, keepdim=True) / 127).float()
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    codes = (v.double() / scale.double()).round().clamp(-127, 127).to(torch.int8)
    return dict(codes=codes, scale=scale.squeeze(-1))


def _quant_rows(s):
    return _quantise(s["x"][:, :s["case"]["K"]].float())


def _quant_channels(s):
    return _quantise(s["w"])


def _products(s):
    """[rows, N] products in the codes' units: sums of whole numbers, in 32 bits."""
    c, b, offs = s["case"], s["b"], s["offsets"].long()
    a, sa, R, E = s["a"], s["sa"], s["rows"], c["groups"]
    if s["index"] is not None:
        a, sa = a[s["index"].long()], sa[s["index"].long()]
    group = torch.searchsorted(offs[1:], torch.arange(R, device="cuda"), right=True)
    if R < E:  # fewer rows than matrices: each row with its own
        acc = torch.bmm(b[group].float(), a.float()[:, :, None])[:, :, 0]
    else:  # the groups' rows padded to the longest group's
        rows = offs[:E, None] + torch.arange(s["most"], device="cuda")
        there = rows < offs[1:E + 1, None]
        pad = a[rows.clamp(max=R - 1)].float().transpose(1, 2).contiguous()
        acc = torch.bmm(b[:E].float(), pad).transpose(1, 2)[there]
        if c["shared"]:
            acc = torch.cat([acc, a[-c["T"]:].float() @ b[E].float().t().contiguous()])
    return acc * sa[:, None] * s["sb"][group]


def _gemm(s):
    return dict(out=_products(s).to(torch.bfloat16))


def _swiglu(s):
    gate, up = _products(s).chunk(2, dim=1)
    return dict(out=(gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16))


_PLAIN = dict(gate=_gate, gate_backward=_gate_backward, quant_rows=_quant_rows,
              quant_channels=_quant_channels, gemm=_gemm, swiglu=_swiglu)


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    c, op = case, case["op"]
    if op in ("gate", "gate_backward"):
        T, E, k = c["T"], c["E"], c["k"]
        size = 4 if c["type"] == "f32" else 2
        if op == "gate":
            return dict(bytes=T * E * size + 8 * T * k + 4 * E + 4 * E * c["bias"]
                        + 4 * T * E * c["scores"], flops=6 * T * E)
        return dict(bytes=2 * T * E * size + 8 * T * k + 4 * T * E * c["d_scores"], flops=8 * T * E)
    if op == "quant_rows":
        return dict(bytes=3 * c["M"] * c["K"] + 4 * c["M"], flops=3 * c["M"] * c["K"])
    if op == "quant_channels":
        n = c["G"] * c["N"]
        return dict(bytes=5 * n * c["K"] + 4 * n, flops=3 * n * c["K"])
    T, E, k, K = c["T"], c["groups"], c["k"], c["K"]
    R = T * (k + c["shared"])
    # experts that T tokens of k each reach, when all are alike
    reached = E * (1 - (1 - k / E) ** T) + c["shared"]
    N = c["N"] * (2 if op == "swiglu" else 1)
    a_rows = T if op == "swiglu" else R
    return dict(bytes=reached * N * (K + 4) + a_rows * (K + 4) + 2 * R * c["N"] + 4 * (E + 2)
                + (4 * R if op == "swiglu" else 0), flops=2 * R * N * K)


# ---- from the definitions, in 64 bits ------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "gate":
        T, E, k, n = c["T"], c["E"], c["k"], c["n_group"]
        l = s["logits"].double()
        score = torch.sigmoid(l) if c["score"] == SIGMOID else torch.softmax(l, dim=1)
        if s["bias"] is None:
            order = l
        else:
            order = score + s["bias"].double()
        if n > 1:
            size = E // n
            if c["group_top"] == 1:
                worth = order.reshape(T * n, size).max(dim=1).values.reshape(T, n)
            else:
                both = score if s["bias"] is None else order
                worth = both.reshape(T * n, size).topk(2, dim=1).values.sum(dim=1).reshape(T, n)
            # a group is kept if fewer than topk_group others come before it
            i = torch.arange(n, device="cuda")
            before = (worth[:, None, :] > worth[:, :, None]) | (
                (worth[:, None, :] == worth[:, :, None]) & (i[None, None, :] < i[None, :, None]))
            out = before.sum(dim=2) >= c["topk_group"]
            order = order.masked_fill(out.reshape(T, n, 1).expand(T, n, size).reshape(T, E), -math.inf)
        chosen = torch.zeros((T, E), dtype=torch.bool, device="cuda")
        at = torch.arange(T, device="cuda")
        for _ in range(k):  # the largest that is left, the lowest index among equals
            left = order.masked_fill(chosen, -math.inf)
            best = (left == left.max(dim=1, keepdim=True).values) & ~chosen
            chosen[at, best.int().argmax(dim=1)] = True
        idx = chosen.nonzero()[:, 1].reshape(T, k)
        w = score[chosen].reshape(T, k)
        if c["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
        return dict(idx=idx.to(torch.int32), w=c["scale"] * w, counts=chosen.sum(dim=0).to(torch.int32),
                    scores=score if c["scores"] else None)
    if op == "gate_backward":
        l = s["logits"].double().requires_grad_(True)
        score = torch.sigmoid(l) if c["score"] == SIGMOID else torch.softmax(l, dim=1)
        w = torch.gather(score, 1, s["idx"].long())
        if c["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
        loss = (c["scale"] * w * s["dw"].double()).sum()
        if s["ds"] is not None:
            loss = loss + (score * s["ds"].double()).sum()
        loss.backward()
        return dict(d_logits=l.grad)
    if op in ("quant_rows", "quant_channels"):
        v = s["w"] if op == "quant_channels" else s["x"][:, :c["K"]]
        scale = v.double().abs().amax(dim=-1) / 127
        scale[scale == 0] = 1.0
        return dict(codes=None, scale=scale)
    offs = s["offsets"].tolist()
    out = torch.empty((s["rows"], c["N"]), dtype=torch.float64, device="cuda")
    for g in range(len(offs) - 1):
        r0, r1 = offs[g], offs[g + 1]
        if r0 == r1:
            continue
        rows = slice(r0, r1) if s["index"] is None else s["index"][r0:r1].long()
        a = s["a"][rows].double() * s["sa"][rows].double()[:, None]
        b = s["b"][g].double() * s["sb"][g].double()[:, None]
        y = a @ b.t()
        if op == "swiglu":
            y = torch.nn.functional.silu(y[:, :c["N"]]) * y[:, c["N"]:]
        out[r0:r1] = y
    return dict(out=out)
