"""Which sums a linear's output is made of, bit for bit.  Whatever kernel takes a
batch and however its tiles are cut, a bf16 output is the binary32 sum rounded
once, and a residual is added once, to the finished binary32 sum.  So the output
in binary32 without a residual says what the others are; there is no tolerance."""
import pytest
import torch

import sparse_moe_transformer_fwd_b200 as moe

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None

# streamed in one round, in a cluster's parts, in parts beside whole tiles; tiled:
# whole tiles, cut ones and both; rows of vectors and ragged ones, a last column
# tile of one 128-row block and of less, a last row tile of few rows
CASES = [(3, 512, 640), (16, 7168, 576), (40, 1536, 999), (64, 16384, 1100), (200, 1152, 384), (300, 2048, 7168),
         (700, 1152, 999), (513, 7168, 4096), (2048, 2048, 2560), (2300, 1152, 2531), (1100, 3584, 9000), (2176, 4096, 2312),
         (2049, 8192, 2568), (600, 7168, 7001), (520, 4096, 7296)]


def _linear(T, K, N, precision, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(T, K, generator=g, device=DEV).bfloat16()
    w = (torch.randn(N, K, generator=g, device=DEV) / K ** 0.5).bfloat16()
    return x, moe.Fp8Linear(w, precision=precision, weight_layout="rowmajor"), g


def _call(lin, x, dtype, residual=None):
    lin.out_dtype = dtype
    out = lin(x, residual=residual)
    assert lin.check_status(x.shape[0]) == 0
    return out


@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0"])
@pytest.mark.parametrize("T,K,N", CASES)
def test_bf16_is_the_binary32_sum_rounded(T, K, N, precision):
    """Neither the output's type nor the batch's size changes how K is summed."""
    x, lin, _ = _linear(T, K, N, precision, T + K + N)
    want = _call(lin, x, torch.float32)
    assert torch.equal(_call(lin, x, torch.bfloat16), want.bfloat16())


@pytest.mark.parametrize("T,K,N", [(2200, 65536, 1832), (600, 7168, 7001), (1024, 7168, 4096)])
def test_long_sums_of_positive_terms(T, K, N):
    """Power-of-two scales, all terms positive, so that bits lost in the sum all
    go one way.  -bf16(sum) as the residual leaves what the sum itself is off by.
    Per K block at most 2^-13 of its terms is allowed elsewhere for the tensor
    core; here the mean error counts: the roundings of K/128 binary32 additions
    are at most 2^-24 of the sum each and of either sign, so their mean over the
    output is below (K/128) 2^-24 / 16, and what the tensor core drops of a K
    block's 128 terms below 128 2^-24 of that block: 2^-17 of the sum."""
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.randn(T, K, generator=g, device=DEV).bfloat16().abs()
    w = (torch.randn(N, K, generator=g, device=DEV) / K ** 0.5).bfloat16().abs()
    lin = moe.Fp8Linear(w, precision="fp8_ue8m0", weight_layout="rowmajor")
    r = lin(x)
    off = lin(x, residual=-r).double() + r.double()
    q, s = torch.empty(T, K, dtype=torch.uint8, device=DEV), torch.empty(T, K // 128, device=DEV)
    moe.fp8_block_quant(x, 1, q, s, ue8m0=True)
    n = min(N, 256)
    e4m3 = lambda c: c.view(torch.float8_e4m3fn).double()
    a = e4m3(q) * s.double().repeat_interleave(128, 1)
    want = a @ (e4m3(lin.w[:n]) * lin.w_scales.double().repeat_interleave(128, 1).repeat_interleave(128, 0)[:n]).T
    mean = ((off[:, :n] - want) / want).mean().item()
    assert abs(mean) <= 2.0 ** -17 + (K // 128) * 2.0 ** -28, mean


@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0"])
@pytest.mark.parametrize("T,K,N", CASES)
def test_residual_is_added_to_the_finished_sum(T, K, N, precision):
    """A residual a thousand times the product: were it in the sum from the start,
    each of the K/128 additions would round at its exponent."""
    x, lin, g = _linear(T, K, N, precision, T + K + N)
    res = (torch.randn(T, N, generator=g, device=DEV) * 1024).bfloat16()
    want = _call(lin, x, torch.float32) + res.float()
    assert torch.equal(_call(lin, x, torch.float32, res), want)
    assert torch.equal(_call(lin, x, torch.bfloat16, res), want.bfloat16())
    buf = res.clone()  # in place
    lin(x, out=buf, residual=buf)
    assert torch.equal(buf, want.bfloat16())
