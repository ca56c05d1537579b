"""moe_forward_few and its pre-norm block against a 64-bit evaluation.

Routing is the oracle's, bit for bit.  Outputs: the reference takes the same
e4m3 (or bf16) operands as the library and evaluates the rest in 64 bits, so
they differ by
  - the rounding of a bf16 output: at most 2^-8 of the value;
  - sums: the tensor core and binary32 promotion keep G, U and Y to 2^-13 of
    the sum of their terms' magnitudes (the other GEMMs of the library are held
    to the same), and the fast exponential and division of silu to a few ulp;
  - H elements whose rounding to a code (or to bf16) such an error can turn:
    those whose quantiser input lies within 2^-12 (relative) of a border are
    allowed their step, propagated through |W2| and the gates."""
import numpy as np
import pytest
import torch

import oracle
import sparse_moe_transformer_fwd_b200 as moe

from _gpu_util import from_u16, u16
from test_gpu_linear import quant_rcp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BAND = 2.0 ** -12


def _e4m3(v):
    e = torch.frexp(v)[1] - 1
    q = torch.ldexp(torch.ones_like(v), torch.clamp(e, min=-6) - 3)
    return torch.clamp(torch.round(v / q) * q, -448.0, 448.0)


def _round_h(h, precision):
    """What H stands for after its rounding, and how far a code turned by BAND moves it."""
    if precision == "bf16":
        r = lambda v: v.float().bfloat16().double()
        return r(h), (r(h * (1 + BAND)) - r(h * (1 - BAND))).abs()
    t = h.reshape(*h.shape[:-1], -1, 128)
    amax = t.abs().amax(-1, keepdim=True)
    if precision == "fp8_ue8m0":
        def scales(a):
            k = torch.ceil(torch.log2(a / 448.0)).clamp(min=-127.0)
            k = torch.where(a * torch.exp2(-k) > 448.0, k + 1, k)
            return torch.exp2(k), torch.exp2(-k)
    else:
        def scales(a):
            return a / 448.0, 448.0 / a
    zero = amax == 0
    a = torch.where(zero, torch.ones_like(amax), amax)
    val = []
    for f in (1.0, 1 - BAND, 1 + BAND):
        for g in (1.0, 1 - BAND, 1 + BAND):  # the tile's maximum moves its scale (a whole step, power-of-two scales)
            s, inv = scales(a * g)
            val.append(torch.where(zero, torch.zeros_like(t), _e4m3(t * f * inv) * s))
    v = torch.stack(val)
    return val[0].reshape(h.shape), (v.amax(0) - v.amin(0)).reshape(h.shape)


class Layer:
    """A layer, its library form, and its operands' values in 64 bits."""

    def __init__(self, d, E, k, de, n_shared, precision, layout, seed, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        S = E + n_shared
        self.E, self.k, self.n_shared, self.precision, self.scale = E, k, n_shared, precision, scale
        self.wr = (torch.randn(E, d, generator=g) / d ** 0.5).bfloat16()
        self.bias = torch.rand(E, generator=g) * 0.2 - 0.1
        w13 = (torch.randn(S, 2 * de, d, generator=g) / d ** 0.5).bfloat16()
        w2 = (torch.randn(S, d, de, generator=g) / de ** 0.5).bfloat16()
        self.lib = moe.MoELayer(self.wr.to(DEV), self.bias.to(DEV), w13.to(DEV), w2.to(DEV), top_k=k,
                                n_shared=n_shared, routed_scale=scale, precision=precision, weight_layout=layout)
        ue = precision == "fp8_ue8m0"

        def values(w):
            if precision == "bf16":
                return [m.double().to(DEV) for m in w]
            return [torch.from_numpy(oracle.dequant(*oracle.block_quant(u16(m), 128, ue8m0=ue), 128)).to(DEV) for m in w]

        self.w13, self.w2 = values(w13), values(w2)

    def route(self, x):
        return oracle.route(oracle.router_logits(u16(x), u16(self.wr)), self.bias.numpy(), self.k, self.scale)[:2]

    def reference(self, x, residual=None):
        """-> idx, out in 64 bits, tolerance."""
        idx, gates = self.route(x)
        if self.precision == "bf16":
            a = x.double()
        else:
            q, s = oracle.block_quant(u16(x), 1, ue8m0=True) if self.precision == "fp8_ue8m0" else quant_rcp(u16(x))
            a = torch.from_numpy(oracle.dequant(q, s, 1))
        a = a.to(DEV)
        T, de = x.shape[0], self.w2[0].shape[1]
        out = residual.double().to(DEV) if residual is not None else torch.zeros(T, x.shape[1], dtype=torch.float64, device=DEV)
        tol = out.abs() * 2.0 ** -24
        for e in sorted(set(idx.flatten().tolist())) + ([self.E] if self.n_shared else []):
            if e < self.E:
                tok = np.nonzero((idx == e).any(1))[0]
                w = torch.tensor([float(gates[t][list(idx[t]).index(e)]) for t in tok], dtype=torch.float64, device=DEV)
            else:
                tok, w = np.arange(T), torch.ones(T, dtype=torch.float64, device=DEV)
            at, w13, w2 = a[tok], self.w13[e], self.w2[e]
            gu, mag = at @ w13.T, at.abs() @ w13.abs().T
            G, U, dG, dU = gu[:, :de], gu[:, de:], mag[:, :de] * 2.0 ** -13, mag[:, de:] * 2.0 ** -13
            sig = 1 / (1 + torch.exp(-G))
            H, slack = _round_h(G * sig * U, self.precision)
            # rounding noise of G and U through silu (slope at most 1.1) where no border is near
            slack = slack + (1.1 * dG * U.abs() + (G * sig).abs() * dU) * 2.0 ** -5
            out[tok] += w[:, None] * (H @ w2.T)
            tol[tok] += w[:, None].abs() * (slack @ w2.abs().T + (H.abs() @ w2.abs().T) * 2.0 ** -13)
        return idx, out, tol + (out.abs() + tol) * 2.0 ** -8


def _check(got, want, tol):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    worst = (err / tol.clamp_min(1e-300)).max().item()
    rel = (got.double() - want).norm().item() / max(want.norm().item(), 1e-300)
    assert worst <= 1.0 and rel <= 2.0 ** -6, (worst, rel)


def _x(T, d, seed):
    return torch.randn(T, d, generator=torch.Generator().manual_seed(seed)).bfloat16()


# (T, d, E, k, d_expert, n_shared): one and sixteen tokens, one K block of H
# (128 in e4m3), an odd number, more experts than blocks, every expert, few
CASES = [
    (1, 512, 16, 4, 256, 1), (2, 256, 16, 2, 128, 1), (16, 512, 16, 4, 384, 1), (7, 1024, 64, 8, 256, 0),
    (5, 256, 300, 6, 128, 1), (16, 256, 40, 32, 128, 1), (3, 768, 4, 4, 640, 0), (9, 256, 1, 1, 128, 0),
    (13, 512, 1023, 8, 128, 1),
]


@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d-d%d-E%d-k%d-de%d-s%d" % c)
def test_few_vs_64bit(case, precision):
    T, d, E, k, de, sh = case
    L = Layer(d, E, k, de, sh, precision, "tiled" if T % 2 else "rowmajor", seed=T + E, scale=2.5 if T == 7 else 1.0)
    x = _x(T, d, T)
    idx = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    out = L.lib.forward_few(x.to(DEV), topk_idx_out=idx)
    assert L.lib.check_status(T) == 0
    want_idx, want, tol = L.reference(x)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    _check(out, want, tol)


@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0", "bf16"])
@pytest.mark.parametrize("T", [1, 6, 16])
def test_few_prenorm(T, precision):
    d = 768
    L = Layer(d, 24, 4, 256, 1, precision, "tiled", seed=3)
    h = (_x(T, d, 8).float() * 3).bfloat16()
    gamma = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(1))).bfloat16()
    idx = torch.empty(T, 4, dtype=torch.int32, device=DEV)
    out = L.lib.forward_few_prenorm(h.to(DEV), gamma.to(DEV), 1e-6, topk_idx_out=idx)
    assert L.lib.check_status(T) == 0
    x = from_u16(oracle.rmsnorm(u16(h), u16(gamma), 1e-6)[0], "cpu").reshape(T, d)
    want_idx, want, tol = L.reference(x, residual=h)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    _check(out, want, tol)


@pytest.mark.parametrize("T", [1, 16])
def test_rough_selection_that_misses(T):
    """Every expert's router row is a permutation of one row and x is constant,
    so the exact logits differ by the order of summation alone: the rough
    logits select other experts, and the missed ones are still computed."""
    d, E, k = 1024, 96, 8
    L = Layer(d, E, k, 128, 1, "fp8", "tiled", seed=2)
    g = torch.Generator().manual_seed(4)
    row = torch.randn(d, generator=g).bfloat16()
    L.wr = torch.stack([row[torch.randperm(d, generator=g)] for _ in range(E)])
    L.bias = torch.zeros(E)
    L.lib.w_router, L.lib.bias = L.wr.to(DEV), L.bias.to(DEV)
    x = torch.linspace(0.5, 1.5, T).bfloat16()[:, None].repeat(1, d).contiguous()
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    for _ in range(3):
        out = L.lib.forward_few(x.to(DEV), topk_idx_out=idx)
        assert L.lib.check_status(T) == 0
        want_idx, want, tol = L.reference(x)
        assert np.array_equal(idx.cpu().numpy(), want_idx)
        _check(out, want, tol)


def test_equal_logits_take_the_lowest_experts():
    L = Layer(256, 32, 4, 128, 1, "fp8", "tiled", seed=2)
    L.lib.w_router.zero_()
    L.lib.bias.zero_()
    idx = torch.empty(2, 4, dtype=torch.int32, device=DEV)
    L.lib.forward_few(_x(2, 256, 1).to(DEV), topk_idx_out=idx)
    assert idx.tolist() == [[0, 1, 2, 3]] * 2


def test_same_routing_as_the_layer_and_near_its_output():
    """Full-size experts, against moe_forward on the same weights: equal
    routing; outputs apart by roundings.  bf16 and power-of-two scales: the
    same codes of x, so what differs is the bf16 rounding of Y there and of out
    (2^-8 each) and the order of sums.  fp32 scales: the two quantisers' factors
    differ in their last bit, which turns codes of x that lie on a border.  A
    border takes a product of two 8-bit significands whose bits below the code's
    four are 1000...: at most 2^-4 of the elements, each moved by a step of at
    most 2^-3 of its value, so G and U change by sqrt(2^-4) 2^-3 = 2^-5 of their
    size (rms) at most.  A relative change eps of H's quantiser input turns its
    code with probability eps / step and moves it by step <= 2^-3: sqrt(eps
    2^-3) = 2^-4 (rms)."""
    d, E, k, de = 7168, 24, 8, 2048
    g = torch.Generator(device=DEV).manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16)
    for precision in ("fp8", "fp8_ue8m0", "bf16"):
        layer = moe.MoELayer(n(E, d) / 85, torch.rand(E, generator=g, device=DEV) * 0.2 - 0.1, n(E + 1, 2 * de, d) / 85,
                             n(E + 1, d, de) / 45, top_k=k, precision=precision)
        for T in (1, 5, 16):
            x = n(T, d)
            i0, i1 = (torch.empty(T, k, dtype=torch.int32, device=DEV) for _ in range(2))
            a, b = layer(x, topk_idx_out=i0), layer.forward_few(x, topk_idx_out=i1)
            assert layer.check_status(T) == 0
            assert torch.equal(i0, i1)
            apart = ((a.float() - b.float()).norm() / a.float().norm()).item()
            assert apart <= (2.0 ** -4 if precision == "fp8" else 2.0 ** -7), (precision, T, apart)
        del layer


def test_special_values():
    """A zero token, and tokens with an infinity or NaN, whose rows alone carry it."""
    T, d = 6, 512
    L = Layer(d, 16, 4, 256, 1, "fp8", "tiled", seed=5)
    x = _x(T, d, 3)
    x[0] = 0
    x[1, :256] = 0
    idx, want, tol = L.reference(x)
    out = L.lib.forward_few(x.to(DEV))
    _check(out, want, tol)
    assert torch.all(out[0] == 0)
    y = x.clone()
    y[2, 5], y[4, 9] = float("inf"), float("nan")
    out2 = L.lib.forward_few(y.to(DEV))
    keep = [0, 1, 3, 5]
    assert torch.equal(out2[keep], out[keep])
    assert L.lib.check_status(T) == 0


@pytest.mark.parametrize("precision", ["fp8", "bf16"])
def test_repeats_streams_and_graphs(precision):
    """Bit-identical repeats, whatever order the blocks ran in; on a side
    stream; two captured graphs that share the workspace, replayed in turn with
    new inputs between eager calls of other shapes."""
    d, k = 512, 4
    L = Layer(d, 32, k, 256, 1, precision, "tiled", seed=6)
    T = 8
    xs = {n: _x(n, d, n).to(DEV) for n in (1, T)}
    want = {n: L.lib.forward_few(xs[n]).clone() for n in xs}
    for _ in range(20):
        for n in xs:
            assert torch.equal(L.lib.forward_few(xs[n]), want[n])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = L.lib.forward_few(xs[T])
    side.synchronize()
    assert torch.equal(out, want[T])
    ws = torch.zeros(moe.moe_few_workspace_size(L.lib.shape(16)), dtype=torch.uint8, device=DEV)
    call = lambda n, x, o: moe.moe_forward_few(L.lib.shape(n), x, L.lib.w_router, L.lib.bias, L.lib.w13, L.lib.w13s,
                                               L.lib.w2, L.lib.w2s, o, ws)
    static = {n: (xs[n].clone(), torch.empty_like(want[n])) for n in xs}
    graphs = {}
    for n in xs:
        torch.cuda.synchronize()
        graphs[n] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[n]):
            call(n, *static[n])
    for seed in (1, 2, 3):
        for n in xs:
            new = _x(n, d, 10 + seed).to(DEV)
            ref = L.lib.forward_few(new).clone()
            static[n][0].copy_(new)
            graphs[n].replay()
            o = torch.empty_like(want[1])
            call(1, xs[1], o)
            torch.cuda.synchronize()
            assert torch.equal(static[n][1], ref)
            assert torch.equal(o, want[1])
    del graphs
    assert moe.moe_check_status(ws) == 0 and L.lib.check_status(T) == 0


def test_a_block_of_the_model():
    """The operators as a decode step runs them: pre-norm projection, output
    projection with the residual, pre-norm MoE layer; eager and captured."""
    T, d, N = 5, 512, 640
    L = Layer(d, 16, 4, 256, 1, "fp8", "tiled", seed=7)
    g = torch.Generator().manual_seed(1)
    proj = moe.Fp8Linear((torch.randn(N, d, generator=g) / d ** 0.5).bfloat16().to(DEV))
    back = moe.Fp8Linear((torch.randn(d, N, generator=g) / N ** 0.5).bfloat16().to(DEV))
    gamma = (1 + 0.1 * torch.randn(d, generator=g)).bfloat16()
    gd = gamma.to(DEV)

    def step(h):
        mid = back(proj.forward_prenorm(h, gd), residual=h)
        return mid, L.lib.forward_few_prenorm(mid, gd)

    h = _x(T, d, 2).to(DEV)
    mid, out = step(h)
    x = from_u16(oracle.rmsnorm(u16(mid), u16(gamma), 1e-6)[0], "cpu").reshape(T, d)
    _, want, tol = L.reference(x, residual=mid)
    _check(out, want, tol)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gmid, gout = step(h)
    for seed in (3, 4):
        h.copy_(_x(T, d, seed))
        graph.replay()
        torch.cuda.synchronize()
        m, o = step(h)
        assert torch.equal(gmid, m) and torch.equal(gout, o)
    del graph
    assert L.lib.check_status(T) == 0 and proj.check_status(T) == 0 and back.check_status(T) == 0


def test_launches_and_refusals():
    L = Layer(256, 8, 2, 128, 1, "fp8", "tiled", seed=1)
    x = _x(4, 256, 1).to(DEV)
    gamma = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    L.lib.forward_few(x)
    assert moe.moe_last_launch_names() == ["moe_few"]
    L.lib.forward_few_prenorm(x, gamma)
    assert moe.moe_last_launch_names() == ["few_prenorm", "moe_few"]
    L.lib.forward_few(x[:0])
    assert moe.moe_last_launch_count() == 0
    with pytest.raises(moe.MoeError, match="at most 16"):
        L.lib.forward_few(_x(17, 256, 1).to(DEV))
    ws, out = L.lib.few_workspace(4), torch.empty_like(x)
    call = lambda **o: moe.moe_forward_few(
        L.lib.shape(4), o.get("x", x), L.lib.w_router, L.lib.bias, o.get("w13", L.lib.w13), L.lib.w13s, L.lib.w2,
        L.lib.w2s, o.get("out", out), o.get("ws", ws))
    with pytest.raises(moe.MoeError):
        call(ws=ws[:4096])
    for bad in (dict(x=x[:3]), dict(out=out[:, :128].contiguous()), dict(w13=L.lib.w13[:4]), dict(x=x.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(moe.MoeError):
        L.lib.forward_few_prenorm(x, gamma, eps=-1.0)
