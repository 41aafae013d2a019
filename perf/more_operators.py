"""Cases, plain forms and calls of the bf16 gated feed-forward experts and of the
norms before and after a block.

Operators:
  glu            grouped_bf16_gemm_glu: gate and up projections, activation and
                 product of the experts in one kernel, gate/up kept on demand
  gemm           grouped_bf16_gemm: the down projection (or any linear layer)
  dgrad_glu      grouped_bf16_gemm_dgrad_glu: the down projection's input
                 gradient and the activation's backward in one kernel
  dgrad          grouped_bf16_gemm_dgrad: input gradient, weights as stored
  wgrad          grouped_bf16_wgrad: each group's weight gradient
  norm           moe_norm: residual add, RMS norm, and the experts' operand
                 (E4M3 in 1x128 tiles, or int8 rows) in one pass
  norm_backward  moe_norm_backward: input and weight gradients
  combine        moe_combine_norm: the gate-weighted sum of the experts' rows and
                 the shared one, its norm, the scaled residual sum
  combine_backward  moe_combine_norm_backward: the experts' output gradients
                 (with E4M3 codes on demand), the gates' and the norm weight's

The plain forms use elementary torch operations in 32 bits, products in 32 bits
too, and round once at the end.
"""
import math

import torch

own = False

SILU, GELU = 0, 1
E4M3 = 1  # moe_norm's codes: 1x128 tiles
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token through the gated half of one dense block: latency
        dict(name="glu one token", op="glu", T=1, groups=1, k=1, shared=False, I=2048, K=7168, act=SILU, keep=False),
        # one decode step of 128 sequences: 256 experts and the shared one
        dict(name="glu decode", op="glu", T=128, groups=256, k=8, shared=True, I=2048, K=7168, act=SILU, keep=False),
        # a training batch that keeps its gate and up outputs for the backward
        dict(name="glu train", op="glu", T=8192, groups=64, k=6, shared=True, I=2048, K=7168, act=GELU, keep=True),
        # down projections of a prefill
        dict(name="gemm prefill", op="gemm", T=16384, groups=256, k=8, shared=True, N=7168, K=2048),
        # the training step's gradients, part by part
        dict(name="dgrad glu train", op="dgrad_glu", T=8192, groups=64, k=6, shared=True, N=7168, I=2048, act=SILU),
        dict(name="wgrad train", op="wgrad", T=8192, groups=64, k=6, shared=True, N=4096, K=7168, gather=True),
        # a short ragged batch of a smaller layer
        dict(name="dgrad odd", op="dgrad", T=1031, groups=16, k=4, shared=False, N=2832, K=2040),
        # the norm before the block: one decode step, its codes on the way
        dict(name="norm decode", op="norm", T=128, H=7168, type="bf16", add=True, codes=True),
        # a prefill whose residual stream is held in 32 bits
        dict(name="norm prefill", op="norm", T=16384, H=7168, type="f32", add=True, codes=True),
        # the training step's gradient through that norm, the residual's gradient added
        dict(name="norm backward train", op="norm_backward", T=16384, H=7168, type="bf16", res=True),
        # the norm after the block over 8 experts a token and the shared one
        dict(name="combine prefill", op="combine", T=16384, k=8, H=7168, type="bf16", shared=True,
             gated=False, norm=True, weight=True),
        # its gradient, with the codes that the experts' backward reads
        dict(name="combine backward train", op="combine_backward", T=16384, k=8, H=7168, type="bf16",
             shared=True, gated=False, norm=True, weight=True, codes=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glu", "glu", "gemm", "gemm", "dgrad_glu", "dgrad", "wgrad", "norm", "norm_backward",
                     "combine", "combine_backward"])
    if op in ("norm", "norm_backward"):
        c = dict(op=op, T=_log(rng, 1, 16000), type=rng.choice(["bf16", "f32"]))
        if op == "norm":
            c["codes"] = rng.random() < 0.5
            c["H"] = 128 * rng.randint(1, 56) if c["codes"] else 8 * rng.randint(8, 896)
            c["add"] = rng.random() < 0.6
        else:
            c["H"], c["res"] = 8 * rng.randint(8, 896), rng.random() < 0.7
        return c
    if op in ("combine", "combine_backward"):
        c = dict(op=op, T=_log(rng, 1, 16000), k=rng.randint(1, 8), type=rng.choice(["bf16", "f32"]),
                 shared=rng.random() < 0.6, norm=rng.random() < 0.7, weight=rng.random() < 0.7)
        c["gated"] = c["shared"] and rng.random() < 0.5
        c["H"] = 8 * rng.randint(8, 896)
        if op == "combine_backward":
            c["codes"] = rng.random() < 0.5
            if c["codes"]:
                c["H"] = 128 * rng.randint(1, 56)
        return c
    groups = _log(rng, 1, 96)
    c = dict(op=op, T=_log(rng, 1, 6000), groups=groups, k=rng.randint(1, min(8, groups)),
             shared=rng.random() < 0.5)
    if op in ("glu", "dgrad_glu"):
        c["I"], c["act"] = 8 * rng.randint(4, 256), rng.choice([SILU, GELU])
        if op == "glu":
            c["K"], c["keep"] = 8 * rng.randint(4, 896), rng.random() < 0.5
        else:
            c["N"] = 8 * rng.randint(4, 896)
        return c
    c["N"], c["K"] = 8 * rng.randint(4, 512), 8 * rng.randint(4, 512)
    if op == "wgrad":
        c["gather"] = rng.random() < 0.5
    return c


# ---- inputs ------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, sigma, g):
    """bf16 normal values, made a few matrices at a time."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").mul_(sigma)
    return out


def prepare(case, seed):
    c, g = case, _gen(seed)
    op, s = c["op"], dict(case=case)
    dev = dict(device="cuda")
    bf = torch.bfloat16
    if op in ("norm", "norm_backward"):
        T, H, dtype = c["T"], c["H"], TYPES[c["type"]]
        size = torch.exp(torch.randn((T, 1), generator=g, **dev) * 0.5)  # tokens of different sizes
        s["x"] = (torch.randn((T, H), generator=g, **dev) * size).to(dtype)
        s["weight"] = 1 + 0.2 * torch.randn(H, generator=g, **dev)
        if op == "norm":
            s["add"] = _normal((T, H), 0.3, g) if c["add"] else None
            s["sum"] = torch.empty((T, H), dtype=dtype, **dev) if c["add"] else None
            s["n"] = torch.empty((T, H), dtype=bf, **dev)
            s["rstd"] = torch.empty(T, **dev)
            s["q"] = s["qs"] = None
            if c["codes"]:
                s["q"] = torch.empty((T, H), dtype=torch.uint8, **dev)
                s["qs"] = torch.empty((T, H // 128), **dev)
            return s
        s["rstd"] = (s["x"].double().square().mean(dim=1) + EPS).rsqrt().float()
        s["dn"] = _normal((T, H), 0.02, g)
        s["res"] = (torch.randn((T, H), generator=g, **dev) * 0.02).to(dtype) if c["res"] else None
        s["dx"] = torch.empty((T, H), dtype=dtype, **dev)
        s["dw"] = torch.empty(H, **dev)
        s["ws"] = None
        return s
    if op in ("combine", "combine_backward"):
        T, k, H, dtype = c["T"], c["k"], c["H"], TYPES[c["type"]]
        s["D"] = _normal((T * (k + c["shared"]), H), 0.5, g)
        s["S"] = s["D"][T * k:] if c["shared"] else None
        s["perm"] = torch.randperm(T * k, generator=g, **dev).to(torch.int32)
        w = torch.rand((T, k), generator=g, **dev) + 0.1
        s["w"] = w / w.sum(dim=1, keepdim=True)
        s["sw"] = torch.rand(T, generator=g, **dev) if c["gated"] else None
        s["weight"] = 1 + 0.2 * torch.randn(H, generator=g, **dev) if c["weight"] else None
        if op == "combine":
            s["x"] = torch.randn((T, H), generator=g, **dev).to(dtype)
            s["y"] = torch.empty((T, H), dtype=dtype, **dev)
            s["rstd"] = torch.empty(T, **dev) if c["norm"] else None
            return s
        s["dy"] = (torch.randn((T, H), generator=g, **dev) * 0.02).to(dtype)
        s["dD"] = torch.empty_like(s["D"])
        s["dw"] = torch.empty((T, k), **dev)
        s["dsw"] = torch.empty(T, **dev) if c["gated"] else None
        s["dweight"] = torch.empty(H, **dev) if c["weight"] else None
        R = s["D"].shape[0]
        s["q"] = torch.empty((R, H), dtype=torch.uint8, **dev) if c["codes"] else None
        s["qs"] = torch.empty((R, H // 128), **dev) if c["codes"] else None
        s["ws"] = None
        return s
    T, E, k = c["T"], c["groups"], c["k"]
    G = E + c["shared"]
    # some experts are more popular than others; each token has k of them
    like = torch.rand((T, E), generator=g, **dev) + 0.3 * torch.rand(E, generator=g, **dev)
    expert = like.topk(k).indices.sort().values.reshape(-1)
    order = expert.sort(stable=True).indices
    counts = torch.bincount(expert, minlength=E)
    source = order // k
    if c["shared"]:
        counts = torch.cat([counts, torch.tensor([T], **dev)])
        source = torch.cat([source, torch.arange(T, **dev)])
    R = s["rows"] = int(source.numel())
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, **dev), counts.cumsum(0)]).to(torch.int32)
    s["most"] = int(counts[:E].max())  # a host program knows a bound of its batch
    s["index"] = None
    if op == "glu":
        I, K = c["I"], c["K"]
        s["index"] = source.to(torch.int32)
        s["a"] = _normal((T, K), 1.0, g)
        s["b"] = _normal((G, 2 * I, K), 1 / math.sqrt(K), g)
        s["h"] = torch.empty((R, I), dtype=bf, **dev)
        s["gu"] = torch.empty((R, 2 * I), dtype=bf, **dev) if c["keep"] else None
    elif op == "dgrad_glu":
        N, I = c["N"], c["I"]
        s["a"] = _normal((R, N), 0.02, g)
        s["b"] = _normal((G, N, I), 1 / math.sqrt(I), g)
        s["gu"] = _normal((R, 2 * I), 1.0, g)
        s["out"] = torch.empty((R, 2 * I), dtype=bf, **dev)
    elif op == "wgrad":
        N, K = c["N"], c["K"]
        s["index"] = source.to(torch.int32) if c["gather"] else None
        s["dy"] = _normal((R, N), 0.02, g)
        s["a"] = _normal((T if c["gather"] else R, K), 1.0, g)
        s["out"] = torch.empty((G, N, K), **dev)
    else:  # gemm: C [R, N] of A [R, K]; dgrad: dA [R, K] of dC [R, N]
        N, K = c["N"], c["K"]
        s["a"] = _normal((R, K if op == "gemm" else N), 1.0 if op == "gemm" else 0.02, g)
        s["b"] = _normal((G, N, K), 1 / math.sqrt(K), g)
        s["out"] = torch.empty((R, N if op == "gemm" else K), dtype=bf, **dev)
    return s


# ---- one pass ------------------------------------------------------------------

def run(state):
    if own:
        return _call(state)
    return _PLAIN[state["case"]["op"]](state)


def _codes(q):
    return None if q is None else q.view(torch.float8_e4m3fn)


def _call(s):
    import fp8_block_scaled_bias_amd as M
    c = s["case"]
    op = c["op"]
    if op == "norm":
        T, H = c["T"], c["H"]
        M.moe_norm(s["x"], s["add"], s["weight"], T, H, EPS, s["sum"], s["n"], s["rstd"], E4M3 if c["codes"] else 0,
                   s["q"], s["qs"])
        return dict(sum=s["sum"], n=s["n"], rstd=s["rstd"], codes=_codes(s["q"]), scale=s["qs"])
    if op == "norm_backward":
        T, H = c["T"], c["H"]
        if s["ws"] is None:  # a program keeps its workspace
            s["ws_bytes"] = M.moe_norm_backward_workspace_bytes(T, H)
            s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
        M.moe_norm_backward(s["dn"], s["x"], s["weight"], s["rstd"], s["res"], 1.0, T, H, s["dx"], s["dw"],
                            s["ws"], s["ws_bytes"])
        return dict(dx=s["dx"], d_weight=s["dw"])
    if op == "combine":
        M.moe_combine_norm(s["D"], s["perm"], s["w"], s["S"], s["sw"], s["x"], 1.0, c["norm"], s["weight"], EPS,
                           0.5, c["T"], c["k"], c["H"], s["y"], s["rstd"])
        return dict(y=s["y"], rstd=s["rstd"])
    if op == "combine_backward":
        T, k, H = c["T"], c["k"], c["H"]
        if s["ws"] is None:
            s["ws_bytes"] = M.moe_combine_norm_backward_workspace_bytes(T, H)
            s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
        M.moe_combine_norm_backward(s["dy"], s["perm"], s["w"], s["D"], int(c["shared"]), s["sw"], c["norm"],
                                    s["weight"], EPS, 0.5, T, k, H, s["dD"], s["dw"], s["dsw"], s["q"], s["qs"],
                                    s["dweight"], s["ws"], s["ws_bytes"])
        return dict(dD=s["dD"], dw=s["dw"], dsw=s["dsw"], d_weight=s["dweight"],
                    codes=_codes(s["q"]), scale=s["qs"])
    G, R = c["groups"] + c["shared"], s["rows"]
    if op == "glu":
        M.grouped_bf16_gemm_glu(s["a"], s["index"], s["b"], s["offsets"], G, R, c["I"], c["K"], c["act"], s["h"],
                                s["gu"])
        return dict(h=s["h"], gu=s["gu"])
    if op == "dgrad_glu":
        M.grouped_bf16_gemm_dgrad_glu(s["a"], s["b"], s["gu"], s["offsets"], G, R, c["N"], c["I"], c["act"],
                                      s["out"])
        return dict(d_gu=s["out"])
    if op == "wgrad":
        M.grouped_bf16_wgrad(s["dy"], s["a"], s["index"], s["offsets"], G, R, c["N"], c["K"], s["out"])
        return dict(dw=s["out"])
    if op == "dgrad":
        M.grouped_bf16_gemm_dgrad(s["a"], s["b"], s["offsets"], G, R, c["N"], c["K"], s["out"])
        return dict(dx=s["out"])
    M.grouped_bf16_gemm(s["a"], s["index"], s["b"], s["offsets"], G, R, c["N"], c["K"], s["out"])
    return dict(out=s["out"])


def _padded(s, v):
    """The routed groups' rows of v, in 32 bits, padded to the longest group's:
    [groups, most, columns], zeros where a group has no row; and which are rows."""
    E, offs = s["case"]["groups"], s["offsets"].long()
    rows = offs[:E, None] + torch.arange(s["most"], device="cuda")
    there = rows < offs[1:E + 1, None]
    return v[rows.clamp(max=s["rows"] - 1)].float() * there[:, :, None], there


def _products(s, flip):
    """[rows, .] products of each row with its group's matrix, as stored or flipped."""
    c, b, offs = s["case"], s["b"], s["offsets"].long()
    a, R, E, T = s["a"], s["rows"], c["groups"], c["T"]
    if s["index"] is not None:
        a = a[s["index"].long()]
    if R < E:  # fewer rows than matrices: each row with its own
        group = torch.searchsorted(offs[1:], torch.arange(R, device="cuda"), right=True)
        m, v = b[group].float(), a.float()
        return torch.bmm(v[:, None, :], m)[:, 0] if flip else torch.bmm(m, v[:, :, None])[:, :, 0]
    pad, there = _padded(s, a)
    m = b[:E].float()
    out = torch.bmm(pad, m) if flip else torch.bmm(m, pad.transpose(1, 2).contiguous()).transpose(1, 2)
    out = out[there]
    if c["shared"]:
        m, v = b[E].float(), a[R - T:].float()
        out = torch.cat([out, v @ m if flip else v @ m.t().contiguous()])
    return out


def _slope(g, act):
    """Activation g * sigmoid(z(g)) and its derivative: z = g, or twice the
    argument of the tanh form of GELU."""
    z, dz = g, torch.ones_like(g)
    if act == GELU:
        r = 2 * math.sqrt(2 / math.pi)
        z, dz = r * (g + 0.044715 * g * g * g), r * (1 + 3 * 0.044715 * g * g)
    p = 1 / (1 + torch.exp(-z))
    return g * p, p + g * p * (1 - p) * dz


def _glu(s):
    gu = _products(s, False)
    gate, up = gu.chunk(2, dim=1)
    h = _slope(gate, s["case"]["act"])[0] * up
    return dict(h=h.to(torch.bfloat16), gu=gu.to(torch.bfloat16) if s["case"]["keep"] else None)


def _gemm(s):
    return dict(out=_products(s, False).to(torch.bfloat16))


def _dgrad(s):
    return dict(dx=_products(s, True).to(torch.bfloat16))


def _dgrad_glu(s):
    dh = _products(s, True)
    gate, up = s["gu"].float().chunk(2, dim=1)
    act, slope = _slope(gate, s["case"]["act"])
    return dict(d_gu=torch.cat([dh * up * slope, dh * act], dim=1).to(torch.bfloat16))


def _wgrad(s):
    c, a, R = s["case"], s["a"], s["rows"]
    if s["index"] is not None:
        a = a[s["index"].long()]
    dy, _ = _padded(s, s["dy"])
    out = torch.bmm(dy.transpose(1, 2).contiguous(), _padded(s, a)[0])
    if c["shared"]:
        last = s["dy"][R - c["T"]:].float().t().contiguous() @ a[R - c["T"]:].float()
        out = torch.cat([out, last[None]])
    return dict(dw=out)


def _e4m3(v):
    """E4M3 codes and scales of v, 1x128 tiles."""
    tiles = v.view(v.shape[0], -1, 128)
    scale = tiles.abs().amax(dim=2) / 448
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return (tiles / scale[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(v.shape), scale


def _norm(s):
    c, x = s["case"], s["x"]
    total = None
    if c["add"]:  # the stream as it is stored is what the norm sees
        total = x = (x.float() + s["add"].float()).to(x.dtype)
    v = x.float()
    rstd = 1 / torch.sqrt(v.square().mean(dim=1) + EPS)
    n = v * rstd[:, None] * s["weight"]
    codes, scale = _e4m3(n) if c["codes"] else (None, None)
    return dict(sum=total, n=n.to(torch.bfloat16), rstd=rstd, codes=codes, scale=scale)


def _norm_backward(s):
    g, hat = s["dn"].float(), s["x"].float() * s["rstd"][:, None]
    gw = g * s["weight"]
    dx = s["rstd"][:, None] * (gw - hat * (gw * hat).mean(dim=1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return dict(dx=dx.to(s["x"].dtype), d_weight=(g * hat).sum(dim=0))


def _rows(s):
    """The experts' rows of each token, [T, k (+ 1), H], and their weights."""
    c = s["case"]
    T, k, H = c["T"], c["k"], c["H"]
    rows, w = s["D"][s["perm"].long()].float().view(T, k, H), s["w"]
    if c["shared"]:
        rows = torch.cat([rows, s["S"].float()[:, None]], dim=1)
        w = torch.cat([w, (torch.ones_like(w[:, 0]) if s["sw"] is None else s["sw"])[:, None]], dim=1)
    return rows, w


def _combine(s):
    c = s["case"]
    rows, w = _rows(s)
    z = (rows * w[:, :, None]).sum(dim=1)
    rstd = None
    if c["norm"]:
        rstd = 1 / torch.sqrt(z.square().mean(dim=1) + EPS)
        z = z * rstd[:, None]
    if s["weight"] is not None:
        z = z * s["weight"]
    return dict(y=(s["x"].float() + 0.5 * z).to(s["x"].dtype), rstd=rstd)


def _combine_backward(s):
    c, g = s["case"], s["dy"].float() * 0.5
    T, k = c["T"], c["k"]
    rows, w = _rows(s)
    z, rstd, d_weight = (rows * w[:, :, None]).sum(dim=1), None, None
    if c["norm"]:
        rstd = (1 / torch.sqrt(z.square().mean(dim=1) + EPS))[:, None]
        z = z * rstd
    if s["weight"] is not None:
        d_weight, g = (g * z).sum(dim=0), g * s["weight"]
    if c["norm"]:
        g = rstd * (g - z * (g * z).mean(dim=1, keepdim=True))
    dw = (rows * g[:, None]).sum(dim=2)
    spread = g[:, None] * w[:, :, None]
    d = torch.empty_like(s["D"], dtype=torch.float32)
    d[s["perm"].long()] = spread[:, :k].reshape(T * k, -1)
    if c["shared"]:
        d[T * k:] = spread[:, k]
    codes, scale = _e4m3(d) if c["codes"] else (None, None)
    return dict(dD=d.to(torch.bfloat16), dw=dw[:, :k].contiguous(), dsw=dw[:, k].contiguous() if c["gated"] else None,
                d_weight=d_weight, codes=codes, scale=scale)


_PLAIN = dict(glu=_glu, gemm=_gemm, dgrad_glu=_dgrad_glu, dgrad=_dgrad, wgrad=_wgrad, norm=_norm,
              norm_backward=_norm_backward, combine=_combine, combine_backward=_combine_backward)


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    c, op, T = case, case["op"], case["T"]
    if op in ("norm", "norm_backward"):
        n, size = T * c["H"], 4 if c["type"] == "f32" else 2
        if op == "norm":
            coded = n + n // 32 if c["codes"] else 0
            return dict(bytes=n * (size + 2) + (n * (size + 2) if c["add"] else 0) + coded + 4 * (T + c["H"]),
                        flops=4 * n)
        return dict(bytes=n * (2 + 2 * size + (size if c["res"] else 0)) + 4 * T + 8 * c["H"], flops=9 * n)
    if op in ("combine", "combine_backward"):
        n, size, m = T * c["H"], 4 if c["type"] == "f32" else 2, c["k"] + c["shared"]
        small = 8 * T * c["k"] + 4 * T * c["gated"] + 4 * c["H"] * c["weight"]
        if op == "combine":
            return dict(bytes=n * (2 * m + 2 * size) + small + 4 * T * c["norm"], flops=n * (2 * m + 6))
        coded = m * (n + n // 32) if c["codes"] else 0
        return dict(bytes=n * (4 * m + size) + coded + small + 4 * T * (c["k"] + c["gated"]) + 4 * c["H"] * c["weight"],
                    flops=n * (5 * m + 10))
    E, k = c["groups"], c["k"]
    R = T * (k + c["shared"])
    # experts that T tokens of k each reach, when all are alike
    reached = E * (1 - (1 - k / E) ** T) + c["shared"]
    offsets = 4 * (E + 2)
    if op == "glu":
        I, K = c["I"], c["K"]
        return dict(bytes=reached * 4 * I * K + 2 * T * K + 4 * R + 2 * R * I * (3 if c["keep"] else 1) + offsets,
                    flops=4 * R * I * K)
    if op == "dgrad_glu":
        N, I = c["N"], c["I"]
        return dict(bytes=reached * 2 * N * I + 2 * R * N + 8 * R * I + offsets, flops=2 * R * N * I)
    N, K = c["N"], c["K"]
    if op == "wgrad":
        a = T if c["gather"] else R
        return dict(bytes=4 * (E + c["shared"]) * N * K + 2 * R * N + 2 * a * K + (4 * R if c["gather"] else 0) + offsets,
                    flops=2 * R * N * K)
    return dict(bytes=reached * 2 * N * K + 2 * R * (N + K) + offsets, flops=2 * R * N * K)


# ---- from the definitions, in 64 bits ------------------------------------------

def _activation(g, act):
    return torch.nn.functional.silu(g) if act == SILU else torch.nn.functional.gelu(g, approximate="tanh")


def exact(case, seed):
    s = prepare(case, seed)
    c, op, T = case, case["op"], case["T"]
    if op == "norm":
        x = s["x"].double()
        total = None
        if c["add"]:
            total = x + s["add"].double()
            x = total.to(s["x"].dtype).double()
        rms = (x.square().sum(dim=1) / c["H"] + EPS).sqrt()
        n = x / rms[:, None] * s["weight"].double()
        scale = n.reshape(T, -1, 128).abs().max(dim=2).values / 448 if c["codes"] else None
        return dict(sum=total, n=n, rstd=1 / rms, codes=None, scale=scale)
    if op == "norm_backward":
        x = s["x"].double().requires_grad_(True)
        w = s["weight"].double().requires_grad_(True)
        n = x / (x.square().mean(dim=1, keepdim=True) + EPS).sqrt() * w
        dx, dw = torch.autograd.grad(n, (x, w), s["dn"].double())
        return dict(dx=dx if s["res"] is None else dx + s["res"].double(), d_weight=dw)
    if op in ("combine", "combine_backward"):
        k, back = c["k"], op == "combine_backward"
        D = s["D"].double()
        w = s["w"].double()
        sw = s["sw"].double() if c["gated"] else None
        weight = s["weight"].double() if c["weight"] else None
        leaf = [v.requires_grad_(back) for v in (D, w, sw, weight) if v is not None]
        z = 0
        for j in range(k):
            z = z + w[:, j, None] * D[s["perm"].view(T, k)[:, j].long()]
        if c["shared"]:
            z = z + (D[T * k:] if sw is None else sw[:, None] * D[T * k:])
        rms = (z.square().mean(dim=1, keepdim=True) + EPS).sqrt()
        out = z / rms if c["norm"] else z
        if weight is not None:
            out = out * weight
        if not back:
            return dict(y=s["x"].double() + 0.5 * out, rstd=1 / rms[:, 0] if c["norm"] else None)
        grads = list(torch.autograd.grad(0.5 * out, leaf, s["dy"].double()))
        dD, dw = grads[0], grads[1]
        rest = grads[2:]
        dsw = rest.pop(0) if sw is not None else None
        scale = None
        if c["codes"]:
            scale = dD.reshape(dD.shape[0], -1, 128).abs().max(dim=2).values / 448
        return dict(dD=dD, dw=dw, dsw=dsw, d_weight=rest.pop(0) if weight is not None else None, codes=None,
                    scale=scale)
    offs, R = s["offsets"].tolist(), s["rows"]
    wide = dict(dtype=torch.float64, device="cuda")
    if op == "glu":
        out = dict(h=torch.empty((R, c["I"]), **wide), gu=torch.empty((R, 2 * c["I"]), **wide) if c["keep"] else None)
    elif op == "wgrad":
        out = dict(dw=torch.zeros(s["out"].shape, **wide))
    else:
        out = {dict(gemm="out", dgrad="dx", dgrad_glu="d_gu")[op]: torch.empty(s["out"].shape, **wide)}
    for g in range(len(offs) - 1):
        r0, r1 = offs[g], offs[g + 1]
        if r0 == r1:
            continue
        rows = slice(r0, r1) if s["index"] is None else s["index"][r0:r1].long()
        a = s["a"][rows].double()
        if op == "wgrad":
            out["dw"][g] = s["dy"][r0:r1].double().t() @ a
            continue
        b = s["b"][g].double()
        if op == "glu":
            y = a @ b.t()
            out["h"][r0:r1] = _activation(y[:, :c["I"]], c["act"]) * y[:, c["I"]:]
            if c["keep"]:
                out["gu"][r0:r1] = y
        elif op == "gemm":
            out["out"][r0:r1] = a @ b.t()
        elif op == "dgrad":
            out["dx"][r0:r1] = a @ b
        else:
            gu = s["gu"][r0:r1].double().requires_grad_(True)
            h = _activation(gu[:, :c["I"]], c["act"]) * gu[:, c["I"]:]
            out["d_gu"][r0:r1] = torch.autograd.grad(h, gu, a @ b)[0]
    return out
