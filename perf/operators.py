"""The operators of the serving step around one DeepSeek-V3/R1 FFN layer, as measured:

  moe_few   the whole MoE layer for a few tokens (router, experts, shared expert, combine) in one launch, alone or as
            the pre-norm block  out = h + MoE(RMSNorm(h) gamma)
  linear    out = x W^T of a bf16 x with block-scaled e4m3 weights; x is quantised in 1x128 tiles on the way, alone,
            with a residual, or behind the pre-norm
  gemm      the same product of e4m3 codes that are quantised already (several projections of one x)

Weights are e4m3 codes with one scale per 128x128 block (binary32, or a power of two: UE8M0), row-major or stored as
128x128-byte tiles; the MoE layer also takes bf16 weights.  `run` computes the plain form in torch, or with `own` makes
the framework's calls.  `exact` restates each operator in 64 bits."""
from __future__ import annotations

import math

import torch

own = False
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases --
def listed():
    few = dict(op="moe_few", d=7168, E=256, k=8, de=2048, shared=1, scale=1.0, precision="fp8", layout="tiled", prenorm=False)
    lin = dict(op="linear", precision="fp8", layout="tiled", out="bf16", residual=False, prenorm=False)
    gem = dict(op="gemm", precision="fp8", layout="tiled", out="bf16", residual=False, prenorm=False)
    return [
        # a small layer, two tokens: nothing but latency (launches, barriers)
        dict(few, name="moe-small-2", T=2, d=512, E=16, k=4, de=256, precision="bf16", layout="rowmajor"),
        # one user's decode step at the full layer: 9 experts' weights and little else
        dict(few, name="moe-full-1", T=1),
        # the same step as a transformer block runs it, with the power-of-two scales
        dict(few, name="moe-full-3-prenorm", T=3, precision="fp8_ue8m0", prenorm=True),
        # verifying a few drafted tokens: about 100 of 257 experts
        dict(few, name="moe-full-16", T=16, scale=2.5),
        # bf16 weights, no shared expert, an odd number of tokens
        dict(few, name="moe-bf16-5", T=5, d=2048, E=64, k=6, de=1408, shared=0, precision="bf16"),
        # a projection in a decode step
        dict(lin, name="linear-1", T=1, K=7168, N=2112, layout="rowmajor"),
        # the same behind the pre-norm, a few tokens, row-major weights
        dict(lin, name="linear-13-prenorm", T=13, K=7168, N=1536, layout="rowmajor", prenorm=True),
        # the output projection of a serving batch, with its residual
        dict(lin, name="linear-64-residual", T=64, K=16384, N=7168, residual=True),
        # logits in 32 bits over an odd vocabulary
        dict(lin, name="linear-7-logits", T=7, K=7168, N=64007, layout="rowmajor", out="f32"),
        # a prompt through a projection
        dict(lin, name="linear-4096", T=4096, K=7168, N=4096),
        # codes that several projections share: ragged batch, odd width, UE8M0
        dict(gem, name="gemm-37-odd", T=37, K=1536, N=4099, layout="rowmajor", precision="fp8_ue8m0"),
        dict(gem, name="gemm-300", T=300, K=2048, N=7168, out="f32"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["moe_few", "linear", "gemm"])
    precision = rng.choice(["fp8", "fp8", "fp8_ue8m0"])
    layout = rng.choice(["tiled", "rowmajor"])
    if op == "moe_few":
        d, de, E = 256 * _between(rng, 2, 28), 128 * _between(rng, 1, 16), _between(rng, 8, 256)
        return dict(op=op, T=_between(rng, 1, 16), d=d, E=E, k=rng.randint(1, min(8, E)), de=de, shared=rng.randint(0, 1),
                    scale=rng.choice([1.0, 2.5]), precision=rng.choice([precision, precision, "bf16"]), layout=layout, prenorm=rng.random() < 0.3)
    N = 128 * _between(rng, 2, 128)
    if layout == "rowmajor" and rng.random() < 0.6:
        N += rng.randint(1, 127)
    K = 128 * _between(rng, 1, 128)
    T = _between(rng, 1, 2048)
    prenorm = op == "linear" and K % 256 == 0 and rng.random() < 0.3
    return dict(op=op, T=T, K=K, N=N, precision=precision, layout=layout, out=rng.choice(["bf16", "f32"]),
                residual=not prenorm and rng.random() < 0.3, prenorm=prenorm)


# ----------------------------------------------------------------- inputs --
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _codes(g, rows, cols, std, ue):
    """Weights as a checkpoint holds them: e4m3 codes of normal values whose block maximum is 448 (about 4.1 standard
    deviations of a 128x128 block), and the blocks' scales."""
    q = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        v = torch.randn(n, cols, generator=g, device=DEV, dtype=torch.bfloat16).mul_(109.0).clamp_(-448.0, 448.0)
        q[r : r + n] = v.to(E4M3).view(torch.uint8)
    s = (torch.rand(-(-rows // 128), cols // 128, generator=g, device=DEV) * 0.2 + 0.9) * (std / 109.0)
    return q, torch.exp2(torch.ceil(torch.log2(s))) if ue else s


def _scores64(x, w_router):
    return torch.sigmoid(x.double() @ w_router.double().T)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    c, ue = dict(case), case["precision"] == "fp8_ue8m0"
    if c["op"] != "moe_few":
        T, K, N = c["T"], c["K"], c["N"]
        w, ws = _codes(g, N, K, 1.0 / math.sqrt(K), ue)
        s = {"case": c, "w": w, "w_scales": ws}
        x = (_normal(g, T, K) * (0.5 + torch.rand(T, 1, generator=g, device=DEV))).bfloat16()
        if c["op"] == "gemm":
            s["a"], s["a_scales"] = _quantise(x.float(), ue)
            s["a"] = s["a"].view(torch.uint8)
        else:
            s["x"] = x
        s["gamma"] = (1.0 + 0.1 * _normal(g, K)).bfloat16() if c["prenorm"] else None
        s["residual"] = _normal(g, T, N).bfloat16() if c["residual"] else None
        s["y"] = torch.empty(T, N, dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device=DEV)
        if own:
            import sparse_moe_transformer_fwd_b200 as moe

            s["shape"] = moe.make_linear_shape(T, K, N, c["precision"], c["layout"], s["y"].dtype)
            s["ws"] = moe.alloc_linear_workspace(s["shape"], DEV)
        return s
    T, d, E, k, de, S = c["T"], c["d"], c["E"], c["k"], c["de"], c["E"] + c["shared"]
    s = {"case": c, "w_router": (_normal(g, E, d) / math.sqrt(d)).bfloat16()}
    s["bias"] = torch.rand(E, generator=g, device=DEV) * 0.2 - 0.1
    s["gamma"] = (1.0 + 0.1 * _normal(g, d)).bfloat16() if c["prenorm"] else None
    # Of more rows than wanted, the first whose selection has no two values within rounding of each other: between such
    # values either choice is right.
    x = _normal(g, 8 * T + 24, d).bfloat16()
    sel = (_scores64(_prenorm64(x, s["gamma"]) if c["prenorm"] else x, s["w_router"]) + s["bias"].double()).topk(min(E, k + 1)).values
    apart = (sel[:, :-1] - sel[:, 1:]).min(1).values if sel.shape[1] > 1 else torch.ones(len(x), device=DEV)
    s["x"] = x[torch.sort((apart < 1e-5).int(), stable=True).indices[:T]].contiguous()
    if c["precision"] == "bf16":
        s["w13"] = torch.randn(S * 2 * de, d, generator=g, device=DEV, dtype=torch.bfloat16).mul_(1.0 / math.sqrt(d))
        s["w2"] = torch.randn(S * d, de, generator=g, device=DEV, dtype=torch.bfloat16).mul_(1.0 / math.sqrt(de))
        s["w13_scales"] = s["w2_scales"] = None
    else:
        s["w13"], s["w13_scales"] = _codes(g, S * 2 * de, d, 1.0 / math.sqrt(d), ue)
        s["w2"], s["w2_scales"] = _codes(g, S * d, de, 1.0 / math.sqrt(de), ue)
    s["out"] = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    s["topk"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
    if own:
        import sparse_moe_transformer_fwd_b200 as moe

        s["shape"] = moe.make_shape(T, d, E, k, de, c["shared"], c["scale"], c["precision"], c["layout"])
        s["ws"] = moe.alloc_few_workspace(s["shape"], DEV)
    return s


# -------------------------------------------------------------- plain form --
def _quantise(v, ue):
    """1x128 tiles of binary32 values: e4m3 codes and scales (amax / 448, or the least power of two that keeps the
    codes within 448).  The codes' borders are set in binary32 by the format's definition."""
    t = v.reshape(*v.shape[:-1], -1, 128)
    amax = t.abs().amax(-1, keepdim=True)
    if ue:
        m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
        k = torch.clamp(e - 9 + (m > 0.875).int(), min=-127)
        scale, inv = torch.ldexp(torch.ones_like(amax), k), torch.ldexp(torch.ones_like(amax), -k)
    else:
        scale, inv = amax / 448.0, 448.0 / amax
    zero = amax == 0
    scale, inv = torch.where(zero, torch.ones_like(scale), scale), torch.where(zero, torch.zeros_like(inv), inv)
    return (t * inv).to(E4M3).reshape(v.shape), scale.squeeze(-1)


def _real(codes, scale):
    """The values that 1x128 tiles stand for."""
    return (codes.float().reshape(*codes.shape[:-1], -1, 128) * scale.unsqueeze(-1)).reshape(codes.shape)


def _rows(w, scales, layout, first, count):
    """Rows first .. first + count - 1 (first a multiple of 128, a tensor or a number) of stored weights, in binary32."""
    rows, cols = w.shape
    per = 128 if scales is not None else 64  # columns of a 128-byte tile
    bands, wide = -(-count // 128), cols // per
    band = first // 128 + torch.arange(bands, device=w.device)
    if layout == "tiled":
        t = w.reshape(-1, wide, 128, per)[band]
    else:
        at = torch.clamp((band[:, None] * 128 + torch.arange(128, device=w.device)).reshape(-1), max=rows - 1)
        t = w[at].reshape(bands, 128, wide, per).transpose(1, 2)
    t = t.float() if scales is None else t.view(E4M3).float() * scales[band][:, :, None, None]
    return t.transpose(1, 2).reshape(bands * 128, cols)[:count]


def _prenorm(h, gamma, eps=1e-6):
    f = h.float()
    rstd = torch.rsqrt((f * f).double().mean(-1, keepdim=True) + eps).float()  # x is rounded to 8 bits right after: borders
    return ((f * rstd) * gamma.float()).bfloat16()


def _run_linear(s):
    c, ue = s["case"], s["case"]["precision"] == "fp8_ue8m0"
    if c["op"] == "gemm":
        a = _real(s["a"].view(E4M3), s["a_scales"])
    else:
        a = _real(*_quantise((_prenorm(s["x"], s["gamma"]) if c["prenorm"] else s["x"]).float(), ue))
    y = a @ _rows(s["w"], s["w_scales"], c["layout"], 0, c["N"]).T
    return (y + s["residual"].float() if c["residual"] else y).to(s["y"].dtype)


def _run_few(s):
    c = s["case"]
    d, E, k, de = c["d"], c["E"], c["k"], c["de"]
    ue, fp8 = c["precision"] == "fp8_ue8m0", c["precision"] != "bf16"
    x = _prenorm(s["x"], s["gamma"]) if c["prenorm"] else s["x"]
    score = _scores64(x, s["w_router"])
    topk = torch.sort(score + s["bias"].double(), dim=1, descending=True, stable=True).indices[:, :k]
    gate = torch.gather(score, 1, topk)
    gate = (gate / gate.sum(1, keepdim=True) * c["scale"]).float()
    a = _real(*_quantise(x.float(), ue)) if fp8 else x.float()
    out = s["x"].float() if c["prenorm"] else torch.zeros(c["T"], d, device=x.device)
    for t in range(c["T"]):  # every token reads its own experts
        for j in range(k + c["shared"]):
            e = topk[t, j] if j < k else E
            gu = a[t] @ _rows(s["w13"], s["w13_scales"], c["layout"], e * 2 * de, 2 * de).T
            h = gu[:de] * torch.sigmoid(gu[:de]) * gu[de:]
            h = _real(*_quantise(h, ue)) if fp8 else h.bfloat16().float()
            y = h @ _rows(s["w2"], s["w2_scales"], c["layout"], e * d, d).T
            out[t] += (gate[t, j] if j < k else 1.0) * y
    return {"out": out.bfloat16(), "topk": topk.int()}


# ------------------------------------------------------- framework's calls --
def _own_linear(s):
    import sparse_moe_transformer_fwd_b200 as moe

    c = s["case"]
    if c["op"] == "gemm":
        moe.fp8_block_gemm(s["shape"], s["a"], s["a_scales"], s["w"], s["w_scales"], s["y"], s["ws"], residual=s["residual"])
    elif c["prenorm"]:
        moe.moe_linear_prenorm(s["shape"], s["x"], s["gamma"], 1e-6, s["w"], s["w_scales"], s["y"], s["ws"])
    else:
        moe.moe_linear(s["shape"], s["x"], s["w"], s["w_scales"], s["y"], s["ws"], residual=s["residual"])
    return s["y"]


def _own_few(s):
    import sparse_moe_transformer_fwd_b200 as moe

    w = (s["w_router"], s["bias"], s["w13"], s["w13_scales"], s["w2"], s["w2_scales"], s["out"], s["ws"])
    if s["case"]["prenorm"]:
        moe.moe_forward_few_prenorm(s["shape"], s["x"], s["gamma"], 1e-6, *w, topk_idx_out=s["topk"])
    else:
        moe.moe_forward_few(s["shape"], s["x"], *w, topk_idx_out=s["topk"])
    return {"out": s["out"], "topk": s["topk"]}


def run(state):
    if state["case"]["op"] == "moe_few":
        return _own_few(state) if own else _run_few(state)
    return _own_linear(state) if own else _run_linear(state)


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    eb = 2 if c["precision"] == "bf16" else 1
    if c["op"] != "moe_few":
        T, K, N = c["T"], c["K"], c["N"]
        a = T * K * 2 if c["op"] == "linear" else T * K + 4 * T * K // 128
        o = 4 if c["out"] == "f32" else 2
        b = N * K + 4 * (-(-N // 128)) * (K // 128) + a + T * N * (o + 2 * c["residual"]) + 2 * K * c["prenorm"]
        return {"bytes": b, "flops": 2.0 * T * K * N}
    T, d, E, k, de = c["T"], c["d"], c["E"], c["k"], c["de"]
    touched = E * (1.0 - (1.0 - k / E) ** T) + c["shared"]  # experts that T tokens meet, on average
    expert = 3 * d * de * eb + (0 if eb == 2 else 4 * 3 * (d // 128) * (de // 128))
    b = touched * expert + E * d * 2 + E * 4 + T * (4 * d + 4 * k) + 2 * d * c["prenorm"]
    return {"bytes": b, "flops": 2.0 * T * (k + c["shared"]) * 3 * d * de + 2.0 * T * E * d}


# ------------------------------------------------------------ in 64 bits --
def _e4m3_64(v):
    """The nearest e4m3 value (ties to even, none above 448), in 64 bits."""
    e = torch.frexp(v)[1] - 1
    q = torch.ldexp(torch.ones_like(v), torch.clamp(e, min=-6) - 3)
    return torch.clamp(torch.round(v / q) * q, -448.0, 448.0)


def _tiles64(v, ue):
    """What the quantiser's tiles stand for.  Inputs are bf16 here, or 64-bit values of H; the factor 448 / amax and
    its product are binary32 by the format's definition."""
    out = torch.empty_like(v)
    for i in range(0, v.shape[-1], 128):
        t = v[..., i : i + 128]
        amax = t.abs().amax(-1, keepdim=True)
        if ue:
            k = torch.clamp(torch.ceil(torch.log2(amax / 448.0)), min=-127.0)
            k = torch.where(amax * torch.exp2(-k) > 448.0, k + 1, k)
            code, scale = _e4m3_64(t * torch.exp2(-k)), torch.exp2(k)
        else:
            inv = 448.0 / amax.float()
            code, scale = _e4m3_64((t.float() * inv).double()), (amax.float() / 448.0).double()
        out[..., i : i + 128] = torch.where(amax > 0, code * scale, torch.zeros_like(t))
    return out


def _matrix64(w, scales, layout, r0, n):
    """Rows r0 .. r0 + n - 1 of stored weights, in 64 bits, one 128-row band after the other."""
    rows, cols = w.shape
    per = 64 if scales is None else 128
    m = torch.empty(n, cols, dtype=torch.float64, device=w.device)
    flat = w.reshape(-1)
    for b in range(0, n, 128):
        h = min(128, n - b, rows - r0 - b)
        if layout == "tiled":
            tiles = flat[(r0 + b) * cols : (r0 + b + 128) * cols].reshape(cols // per, 128, per)
            band = torch.cat(list(tiles), dim=1)[:h]
        else:
            band = w[r0 + b : r0 + b + h]
        band = band.double() if scales is None else band.view(E4M3).double() * scales[(r0 + b) // 128].double().repeat_interleave(128)
        m[b : b + h] = band
    return m


def _prenorm64(h, gamma):
    """bf16((h rstd) gamma) with rstd from 64 bits; the two products are binary32 by the block's definition."""
    rstd = 1.0 / torch.sqrt(h.double().square().sum(-1, keepdim=True) / h.shape[-1] + 1e-6)
    return (h.float() * rstd.float() * gamma.float()).bfloat16()


def exact(case, seed):
    c = case
    if c["op"] != "moe_few" and c["T"] * c["K"] * c["N"] > 4e11:
        return None
    s = prepare(case, seed)
    ue, fp8 = c["precision"] == "fp8_ue8m0", c["precision"] != "bf16"
    if c["op"] != "moe_few":
        if c["op"] == "gemm":
            a = s["a"].view(E4M3).double() * s["a_scales"].double().repeat_interleave(128, dim=1)
        else:
            a = _tiles64((_prenorm64(s["x"], s["gamma"]) if c["prenorm"] else s["x"]).double(), ue)
        y = torch.empty(c["T"], c["N"], dtype=torch.float64, device=a.device)
        for n in range(0, c["N"], 8192):
            m = min(8192, c["N"] - n)
            y[:, n : n + m] = a @ _matrix64(s["w"], s["w_scales"], c["layout"], n, m).T
        return y + s["residual"].double() if c["residual"] else y
    x = _prenorm64(s["x"], s["gamma"]) if c["prenorm"] else s["x"]
    score = 1.0 / (1.0 + torch.exp(-(x.double() @ s["w_router"].double().T)))
    chosen = torch.topk(score + s["bias"].double(), c["k"], dim=1).indices
    g = torch.gather(score, 1, chosen)
    g = g * c["scale"] / g.sum(1, keepdim=True)
    a = _tiles64(x.double(), ue) if fp8 else x.double()
    out = s["x"].double() if c["prenorm"] else torch.zeros(c["T"], c["d"], dtype=torch.float64, device=x.device)
    de, d = c["de"], c["d"]
    for e in sorted(set(chosen.flatten().tolist())) + ([c["E"]] if c["shared"] else []):
        tok = (chosen == e).any(1).nonzero().flatten() if e < c["E"] else torch.arange(c["T"], device=x.device)
        wt = (g * (chosen == e)).sum(1)[tok] if e < c["E"] else torch.ones(c["T"], dtype=torch.float64, device=x.device)
        gu = a[tok] @ _matrix64(s["w13"], s["w13_scales"], c["layout"], e * 2 * de, 2 * de).T
        h = gu[:, :de] / (1.0 + torch.exp(-gu[:, :de])) * gu[:, de:]
        h = _tiles64(h, ue) if fp8 else h.bfloat16().double()
        out[tok] += wt[:, None] * (h @ _matrix64(s["w2"], s["w2_scales"], c["layout"], e * d, d).T)
    return {"out": out, "topk": None}
