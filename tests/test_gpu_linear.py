"""The block-scaled linear (moe_linear, moe_linear_prenorm, fp8_block_gemm)
against a 64-bit evaluation of the same codes.

Tolerances.  The codes and scales of both operands are exact inputs of the
reference (for moe_linear they come from quant_rcp below, the documented
arithmetic, which the library matches bit for bit), so the outputs differ by the kernel's sums
only: per 128-wide K block the tensor core's sum of e4m3 products, a binary32
scale product (2^-24 relative), and one binary32 fused multiply-add per K
block.  With S = sum_kb s_a s_w sum |a w| (all terms positive):
  - each of the KB additions, and each partial-sum addition of a split tile,
    rounds a value of at most S: KB + 16 roundings of 2^-24 S;
  - the scale product and its use: 2 * 2^-24 S;
  - the tensor core sums a K block in chunks of 32 with an alignment that
    keeps at least 2^-13 of the chunk's largest term: the products of e4m3
    codes have 8 significand bits, and the library's other kernels rely on
    sums good to 2^-13 S.
bf16 outputs add half a bf16 step: at most 2^-8 of the value."""
import numpy as np
import pytest
import torch

import oracle
import sparse_moe_transformer_fwd_b200 as moe

from _gpu_util import from_u16, u16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def _values(codes_u8, scales, block_rows):
    """float64 values of [rows, cols] codes in block_rows x 128 blocks."""
    v = oracle.e4m3_decode_table()[codes_u8].astype(np.float64)
    s = np.repeat(np.repeat(scales.astype(np.float64), 128, axis=1), block_rows, axis=0)[: v.shape[0]]
    return v * s


def _check(got, a, w, residual=None):
    a, w = torch.from_numpy(a).to(DEV), torch.from_numpy(w).to(DEV)
    want = a @ w.T
    S = a.abs() @ w.abs().T
    if residual is not None:
        want = want + residual.double()
        S = S + residual.double().abs()
    KB = a.shape[1] // 128
    tol = S * (2.0 ** -13 + (KB + 18) * 2.0 ** -24)
    if got.dtype == torch.bfloat16:
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    worst = ((got.double() - want).abs() / (tol + 1e-300)).max().item()
    rel = ((got.double() - want).norm() / want.norm().clamp_min(1e-300)).item()
    assert worst <= 1.0, (worst, rel)
    # far tighter on the whole: a wrong scale or K block is 2^-4 and more
    assert rel <= (2.0 ** -8 if got.dtype == torch.bfloat16 else 2e-5), rel


def _inputs(T, K, N, precision, layout, seed, gen=None):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, K, generator=g) * (0.5 + torch.rand(T, 1, generator=g))).bfloat16()
    w = (torch.randn(N, K, generator=g) / K ** 0.5).bfloat16()
    lin = moe.Fp8Linear(w.to(DEV), precision=precision, weight_layout=layout)
    wq, ws = oracle.block_quant(u16(w), 128, ue8m0=precision == "fp8_ue8m0")
    return x, lin, _values(wq, ws, 128), g


def quant_rcp(v):
    """e4m3 codes and scales of 1x128 tiles by one binary32 reciprocal: scale amax * (1/448), codes of
    v * (448 * (1/amax))."""
    f = np.float32
    t = oracle.bf16_to_f32(v).reshape(v.shape[0], -1, 128)
    amax = np.abs(t).max(-1, keepdims=True)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.minimum((f(1) / amax) * f(448), np.finfo(f).max)
        scale = np.where(amax == 0, f(1), amax * f(1.0 / 448.0)).astype(f)
        codes = oracle.e4m3_encode(np.where(amax == 0, f(0), t * inv).astype(f))
    return codes.reshape(v.shape), np.ascontiguousarray(scale[..., 0])


def _quant(x, precision):
    q, s = oracle.block_quant(u16(x), 1, ue8m0=True) if precision == "fp8_ue8m0" else quant_rcp(u16(x))
    return q, s, _values(q, s, 1)


# few tokens (16-, 32- and 64-column tiles, each end), split and whole tiles,
# short last row blocks, odd N, one K block; then the tiled GEMM: direct, split
# K, padded N, binary32
CASES = [
    (1, 7168, 576), (1, 128, 1), (2, 128, 130), (16, 1536, 2112), (17, 512, 1000), (32, 256, 4099),
    (33, 2048, 640), (64, 7168, 1536), (64, 384, 33), (3, 18432, 257), (5, 256, 40000),
    (65, 1536, 512), (100, 512, 384), (128, 384, 130), (256, 2048, 768), (257, 512, 256), (300, 1152, 520),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0"])
@pytest.mark.parametrize("T,K,N", CASES)
def test_linear_vs_64bit(T, K, N, precision, out_dtype):
    x, lin, w, _ = _inputs(T, K, N, precision, "rowmajor", seed=T + K + N)
    lin.out_dtype = out_dtype
    out = lin(x.to(DEV))
    assert lin.check_status(T) == 0
    q, s, a = _quant(x, precision)
    _check(out, a, w)
    out2 = lin.quantized(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV))
    assert lin.check_status(T) == 0
    assert torch.equal(out, out2)


@pytest.mark.parametrize("T,K,N", [(1, 7168, 1536), (13, 512, 128), (40, 1536, 640), (200, 512, 384),
                                   (300, 512, 512)])
def test_tiled_weights_match_rowmajor(T, K, N):
    outs = []
    for layout in ("tiled", "rowmajor"):
        x, lin, w, _ = _inputs(T, K, N, "fp8", layout, seed=7)
        outs.append(lin(x.to(DEV)))
        assert lin.check_status(T) == 0
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("T,N,out_dtype", [(1, 640, torch.bfloat16), (50, 999, torch.bfloat16),
                                           (9, 999, torch.float32), (90, 512, torch.bfloat16),
                                           (300, 512, torch.bfloat16), (300, 999, torch.float32)])
def test_residual(T, N, out_dtype):
    x, lin, w, g = _inputs(T, 512, N, "fp8", "rowmajor", seed=11)
    lin.out_dtype = out_dtype
    res = torch.randn(T, N, generator=g).bfloat16().to(DEV)
    out = lin(x.to(DEV), residual=res)
    _check(out, _quant(x, "fp8")[2], w, res)
    if out_dtype == torch.bfloat16:  # in place
        buf = res.clone()
        lin(x.to(DEV), out=buf, residual=buf)
        assert torch.equal(buf, out)


@pytest.mark.parametrize("T", [1, 16, 40, 300])
@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0"])
def test_prenorm(T, precision):
    K, N = 1024, 768
    h, lin, w, g = _inputs(T, K, N, precision, "tiled", seed=5)
    gamma = (1 + 0.1 * torch.randn(K, generator=g)).bfloat16()
    out = lin.forward_prenorm(h.to(DEV), gamma.to(DEV), 1e-6)
    assert lin.check_status(T) == 0
    x = from_u16(oracle.rmsnorm(u16(h), u16(gamma), 1e-6)[0], "cpu").reshape(T, K)
    _check(out, _quant(x, precision)[2], w)


def test_extreme_tiles():
    """Zero rows and tiles, one huge element per tile, tiny inputs; a
    token's own infinities and NaN stay its own."""
    T, K, N = 20, 512, 300
    x, lin, w, _ = _inputs(T, K, N, "fp8", "rowmajor", seed=3)
    x[0] = 0
    x[1, 128:256] = 0
    x[2, ::128] = 3e4
    x[3] = x[3] * 1e-30
    x[4, :128] = 0
    x[4, 5] = 1e-37  # below 448 / FLT_MAX: a code, not NaN
    out = lin(x.to(DEV))
    _check(out, _quant(x, "fp8")[2], w)
    assert torch.all(out[0] == 0)
    y = x.clone()
    y[5, 7] = float("inf")
    y[9, 300] = float("nan")
    out2 = lin(y.to(DEV))
    keep = [t for t in range(T) if t not in (5, 9)]
    assert torch.equal(out2[keep], out[keep])


@pytest.mark.parametrize("T,N", [(1, 640), (64, 999), (200, 999)])
def test_repeats_and_graph_replay_bitidentical(T, N):
    x, lin, w, g = _inputs(T, 2048, N, "fp8", "rowmajor", seed=9)
    xs = x.to(DEV)
    first = lin(xs).clone()
    for _ in range(5):
        assert torch.equal(lin(xs), first)
    static, out = xs.clone(), torch.empty_like(first)
    lin(static, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin(static, out=out)
    for seed in (1, 2):
        new = torch.randn(T, 2048, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)
        want = lin(new).clone()
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    del graph
    assert lin.check_status(T) == 0


def test_one_workspace_for_many_shapes():
    """Counters are left zero and lie clear of every other region, so one
    workspace serves linears of any shape, on a side stream too."""
    shapes = [(64, 7168, 640), (1, 512, 40000), (300, 512, 999), (7, 1536, 130), (64, 256, 64007)]
    lins = [_inputs(T, K, N, "fp8", "rowmajor", seed=K + N) for T, K, N in shapes]
    ws = torch.zeros(max(moe.moe_linear_workspace_size(l.shape(T)) for (T, _, _), (_, l, _, _) in zip(shapes, lins)),
                     dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    for _ in range(2):
        for (T, K, N), (x, lin, w, _) in zip(shapes, lins):
            want = lin(x.to(DEV))
            out = torch.empty_like(want)
            xd = x.to(DEV)
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                moe.moe_linear(lin.shape(T), xd, lin.w, lin.w_scales, out, ws)
            side.synchronize()
            assert torch.equal(out, want), (T, K, N)
    assert moe.moe_check_status(ws) == 0


def test_weights_written_just_before():
    """The kernel before the call may still be writing the weights and codes
    when the call is enqueued: nothing is read ahead of it."""
    T, K, N = 300, 2048, 7168
    g = torch.Generator().manual_seed(2)
    w = (torch.randn(N, K, generator=g) / 45).bfloat16().to(DEV)
    x = torch.randn(T, K, generator=g).bfloat16().to(DEV)
    lin = moe.Fp8Linear(w)
    a, s = torch.empty(T, K, dtype=torch.uint8, device=DEV), torch.empty(T, K // 128, device=DEV)
    moe.fp8_block_quant(x, 1, a, s)
    want = lin.quantized(a, s).clone()
    for _ in range(3):
        lin.w.zero_()
        torch.cuda.synchronize()
        moe.fp8_block_quant(w, 128, lin.w, lin.w_scales, layout=moe.MOE_LAYOUT_TILED)
        assert torch.equal(lin.quantized(a, s), want)


def test_launches():
    x, lin, w, _ = _inputs(8, 512, 640, "fp8", "tiled", seed=1)
    lin(x.to(DEV))  # up to 16 tokens: quantised in the product's kernel
    assert moe.moe_last_launch_names() == ["linear_stream"]
    lin.forward_prenorm(x.to(DEV), torch.ones(512, dtype=torch.bfloat16, device=DEV))
    assert moe.moe_last_launch_names() == ["linear_prenorm_quant", "linear_stream"]
    lin(torch.zeros(17, 512, dtype=torch.bfloat16, device=DEV))
    assert moe.moe_last_launch_names() == ["linear_quant", "linear_stream"]
    x, lin, w, _ = _inputs(17, 7168, 256, "fp8", "tiled", seed=1)  # two tiles, cut into parts of K
    lin(x.to(DEV))
    assert moe.moe_last_launch_names() == ["linear_quant", "linear_stream"]
    lin(x.to(DEV)[:4])  # added by the tile's last block
    assert moe.moe_last_launch_names() == ["linear_stream"]
    lin(x.to(DEV)[:0])
    assert moe.moe_last_launch_count() == 0


def test_refusals():
    x, lin, w, _ = _inputs(4, 512, 640, "fp8", "tiled", seed=1)
    xd, out, ws = x.to(DEV), torch.empty(4, 640, dtype=torch.bfloat16, device=DEV), lin.workspace(4)
    sh = lin.shape(4)
    with pytest.raises(moe.MoeError):  # workspace too small
        moe.moe_linear(sh, xd, lin.w, lin.w_scales, out, ws[:1024])
    with pytest.raises(ValueError):  # too few elements
        moe.moe_linear(sh, xd[:3], lin.w, lin.w_scales, out, ws)
    with pytest.raises(ValueError):
        moe.moe_linear(sh, xd, lin.w, lin.w_scales, out[:, :600].contiguous(), ws)
    with pytest.raises(ValueError):  # not contiguous
        moe.moe_linear(sh, torch.empty(4, 1024, dtype=torch.bfloat16, device=DEV)[:, ::2], lin.w, lin.w_scales, out, ws)
    with pytest.raises(ValueError):  # a CPU tensor
        moe.moe_linear(sh, x, lin.w, lin.w_scales, out, ws)
    with pytest.raises(TypeError):  # out dtype
        moe.moe_linear(sh, xd, lin.w, lin.w_scales, out.float(), ws)
    with pytest.raises(moe.MoeError):
        moe.moe_linear_prenorm(sh, xd, torch.ones(512, dtype=torch.bfloat16, device=DEV), -1.0, lin.w, lin.w_scales, out, ws)
