"""What the linear makes of its inputs, against no restatement of the kernel:
the values that x's codes stand for, and weights that the kernel before the call
is still writing."""
import numpy as np
import pytest
import torch

import oracle
import sparse_moe_transformer_fwd_b200 as moe

from _gpu_util import u16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0"])
@pytest.mark.parametrize("T", [1, 5, 16, 17, 40, 300])
def test_codes_are_the_nearest(T, precision):
    """Weights that are the identity give scale * code of each element of x (one
    product, exact; one binary32 rounding of scale * code).  With the real
    quotient x / scale of a correctly rounded scale amax / 448:
      - scale amax * (1/448) is off by the constant's and the product's rounding,
        2 * 2^-24 relative, and the factor 448 * (1/amax) by the reciprocal's and
        the product's, 2 * 2^-24, its product with x by 2^-24 more;
      - so the value in hand when the code is chosen is within 3 * 2^-24 (and
        second-order terms: 2^-22 in all) of the quotient 448 x / amax, and the
        code is the nearest one unless that lies so near the middle of two.
    Power-of-two scales: the factor is exact, so the code is the nearest."""
    K = 1024
    ue = precision == "fp8_ue8m0"
    g = torch.Generator().manual_seed(T)
    x = (torch.randn(T, K, generator=g) * torch.exp(3 * torch.randn(T, 1, generator=g))).bfloat16()
    x[0, :128] = 0
    x[T // 2, 128:256] = x[T // 2, 128:256] * 1e-30
    lin = moe.Fp8Linear(torch.zeros(K, K, dtype=torch.bfloat16, device=DEV), precision=precision,
                        weight_layout="rowmajor", out_dtype=torch.float32)
    lin.w.copy_(torch.eye(K, dtype=torch.uint8, device=DEV) * 0x38)  # 1.0
    lin.w_scales.fill_(1.0)
    got = lin(x.to(DEV)).cpu().double().numpy().reshape(T, -1, 128)
    assert lin.check_status(T) == 0
    v = x.double().numpy().reshape(T, -1, 128)
    amax = np.abs(v).max(-1, keepdims=True)
    assert np.all(got[np.broadcast_to(amax == 0, got.shape)] == 0)
    live = np.broadcast_to(amax > 0, got.shape)
    if ue:
        scale = oracle.block_quant(u16(x), 1, ue8m0=True)[1].astype(np.float64)[..., None]
        want = v / scale
    else:
        scale = np.where(amax > 0, amax, 448.0) / 448.0
        want = v * 448.0 / np.where(amax > 0, amax, 1.0)
    codes = np.unique(oracle.e4m3_decode_table().astype(np.float64)[np.r_[0:127]])
    codes = np.unique(np.concatenate([codes, -codes]))
    value = got / scale  # a code, within the scale's and the output's roundings
    nearest = codes[np.abs(codes[None] - value.reshape(-1, 1)).argmin(1)].reshape(value.shape)
    assert np.all(np.abs(value - nearest)[live] <= (4 * 2.0 ** -24 * np.abs(nearest))[live])
    middle = (codes[1:] + codes[:-1]) / 2
    right = codes[np.abs(codes[None] - want.reshape(-1, 1)).argmin(1)].reshape(value.shape)
    near = np.abs(middle[None] - want.reshape(-1, 1)).min(1).reshape(value.shape) <= np.abs(want) * (0.0 if ue else 2.0 ** -22)
    wrong = live & (nearest != right) & ~near
    # exactly in the middle (ue: x / scale can be): either neighbour is as near
    wrong &= np.abs(np.abs(nearest - want) - np.abs(right - want)) > 0
    assert not wrong.any(), (nearest[wrong][:5], right[wrong][:5], want[wrong][:5])


@pytest.mark.parametrize("kind", ["linear", "prenorm", "quantized"])
@pytest.mark.parametrize("T,K,N,layout", [(1, 7168, 7168, "rowmajor"), (13, 7168, 7168, "tiled"), (40, 7168, 7168, "tiled"),
                                          (64, 4096, 9001, "rowmajor"), (300, 7168, 7168, "rowmajor"), (1500, 4096, 7168, "tiled"),
                                          (600, 4096, 7001, "rowmajor")])
def test_weights_written_just_before_every_call(T, K, N, layout, kind):
    """The kernel before the call may still be writing the weights and their
    scales: whatever the call's first launch is, none reads them ahead of it."""
    g = torch.Generator(DEV).manual_seed(T)
    w = (torch.randn(N, K, generator=g, device=DEV) / K ** 0.5).bfloat16()
    x = torch.randn(T, K, generator=g, device=DEV).bfloat16()
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).bfloat16()
    lin = moe.Fp8Linear(w, weight_layout=layout)
    a, s = torch.empty(T, K, dtype=torch.uint8, device=DEV), torch.empty(T, K // 128, device=DEV)
    moe.fp8_block_quant(x, 1, a, s)
    call = {"linear": lambda: lin(x), "prenorm": lambda: lin.forward_prenorm(x, gamma), "quantized": lambda: lin.quantized(a, s)}[kind]
    want = call().clone()
    for _ in range(3):
        lin.w.zero_()
        lin.w_scales.zero_()
        torch.cuda.synchronize()
        moe.fp8_block_quant(w, 128, lin.w, lin.w_scales,
                            layout=moe.MOE_LAYOUT_TILED if layout == "tiled" else moe.MOE_LAYOUT_ROWMAJOR)
        assert torch.equal(call(), want)
    assert lin.check_status(T) == 0


@pytest.mark.parametrize("T,K", [(1, 8320), (5, 16384), (40, 12416), (2, 131072), (300, 8192), (300, 9088)])
def test_long_rows_behind_the_prenorm(T, K):
    """Rows longer than the statistics' piece in shared memory: the same codes as of
    the pre-norm worked out apart, so the same output."""
    g = torch.Generator(DEV).manual_seed(K)
    h = torch.randn(T, K, generator=g, device=DEV).bfloat16()
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).bfloat16()
    lin = moe.Fp8Linear((torch.randn(264, K, generator=g, device=DEV) / K ** 0.5).bfloat16(), weight_layout="rowmajor")
    x, _ = oracle.rmsnorm(u16(h), u16(gamma), 1e-6)
    x = torch.from_numpy(np.ascontiguousarray(x).reshape(T, K).view(np.int16)).view(torch.bfloat16).to(DEV)
    assert torch.equal(lin.forward_prenorm(h, gamma), lin(x))
    assert lin.check_status(T) == 0


@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0"])
@pytest.mark.parametrize("T,N", [(9, 640), (20, 300), (300, 1000), (700, 999)])
def test_infinities_and_nan_stay_in_their_rows(T, N, precision):
    g = torch.Generator(DEV).manual_seed(T)
    x = torch.randn(T, 1024, generator=g, device=DEV).bfloat16()
    lin = moe.Fp8Linear((torch.randn(N, 1024, generator=g, device=DEV) / 32).bfloat16(), precision=precision, weight_layout="rowmajor")
    want = lin(x)
    y = x.clone()
    y[1, 7], y[T // 2, 300], y[T - 1] = float("inf"), float("nan"), float("-inf")
    got = lin(y)
    bad = [1, T // 2, T - 1]
    keep = [t for t in range(T) if t not in bad]
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[bad]).all()
    res = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
    res[2], res[3, 5] = float("inf"), float("nan")
    got = lin(x, residual=res)
    assert torch.equal(got[[0, 1]], want[[0, 1]]) and torch.isinf(got[2]).all()
    assert torch.isnan(got[3, 5]) and torch.isfinite(got[3, :5]).all() and torch.isfinite(got[3, 6:]).all()
    assert lin.check_status(T) == 0
