"""CPU checks of moe_forward_few, moe_linear and fp8_block_gemm at the C ABI
and in the binding: what they refuse, they refuse on the host, before a kernel
is enqueued."""
import ctypes

import pytest
import torch

import sparse_moe_transformer_fwd_b200 as moe
from sparse_moe_transformer_fwd_b200 import _native as N

FAKE = ctypes.c_void_p(0x7F0000001000)  # never dereferenced on the host
MISALIGNED = ctypes.c_void_p(0x7F0000001008)
UNALIGNED_WS = ctypes.c_void_p(0x7F0000001080)


def _few(**kw):
    a = dict(T=4, d_model=7168, n_experts=256, top_k=8, d_expert=2048, n_shared=1, routed_scale=1.0, precision="fp8")
    a.update(kw)
    return moe.make_shape(**a)


def _call_few(shape, nbytes, **o):
    g = lambda n: o.get(n, FAKE)
    return moe.lib().moe_forward_few(ctypes.byref(shape), g("x"), g("w_router"), g("bias"), g("w13"), g("w13s"), g("w2"),
                                     g("w2s"), g("out"), o.get("idx"), g("ws"), nbytes, None)


def _call_few_prenorm(shape, nbytes, gamma=FAKE, eps=1e-6):
    return moe.lib().moe_forward_few_prenorm(ctypes.byref(shape), FAKE, gamma, ctypes.c_float(eps), FAKE, FAKE, FAKE,
                                             FAKE, FAKE, FAKE, FAKE, None, FAKE, nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(T=17), dict(T=-1), dict(T=1 << 30), dict(d_model=7000), dict(d_model=384), dict(d_expert=100), dict(top_k=0),
    dict(top_k=33), dict(top_k=300), dict(n_shared=2), dict(n_experts=1024), dict(precision=7), dict(weight_layout=2),
    dict(d_model=1025 * 128 * 2)], ids=str)
def test_few_bad_shapes(bad):
    s = _few(**bad)
    assert moe.lib().moe_few_workspace_size(ctypes.byref(s)) == 0
    assert moe.moe_last_error()
    assert _call_few(s, 1 << 40) == N.MOE_ERR_INVALID_ARG


def test_few_host_side_errors():
    s = _few()
    need = moe.moe_few_workspace_size(s)
    assert need > 2 * 4 * 9 * 7168 * 4  # the experts' rows in binary32
    assert _call_few(s, need - 1) == N.MOE_ERR_WORKSPACE
    assert "needs" in moe.moe_last_error()
    for name in ("x", "w_router", "bias", "w13", "w2", "out", "w13s", "w2s"):
        assert _call_few(s, need, **{name: None}) == N.MOE_ERR_INVALID_ARG, name
        assert _call_few(s, need, **{name: MISALIGNED}) == N.MOE_ERR_INVALID_ARG, name
    assert _call_few(s, need, ws=None) == N.MOE_ERR_INVALID_ARG
    assert _call_few(s, need, ws=UNALIGNED_WS) == N.MOE_ERR_INVALID_ARG
    assert _call_few(s, need, idx=MISALIGNED) == N.MOE_ERR_INVALID_ARG
    assert _call_few_prenorm(s, need, gamma=None) == N.MOE_ERR_INVALID_ARG
    assert _call_few_prenorm(s, need, gamma=MISALIGNED) == N.MOE_ERR_INVALID_ARG
    for eps in (-1.0, float("nan")):
        assert _call_few_prenorm(s, need, eps=eps) == N.MOE_ERR_INVALID_ARG
    assert moe.lib().moe_forward_few(None, *[FAKE] * 8, None, FAKE, need, None) == N.MOE_ERR_INVALID_ARG
    e = _few(T=0)
    assert _call_few(e, moe.moe_few_workspace_size(e), x=None, out=None) == N.MOE_OK
    assert moe.moe_last_launch_count() == 0


def test_few_workspace_grows_with_the_batch():
    """One workspace of the largest batch serves all of them."""
    for precision in ("fp8", "fp8_ue8m0", "bf16"):
        sizes = [moe.moe_few_workspace_size(_few(T=T, precision=precision)) for T in range(17)]
        assert sizes == sorted(sizes) and all(n % 256 == 0 for n in sizes)


def _linear(**kw):
    a = dict(T=8, K=7168, N=1536)
    a.update(kw)
    return moe.make_linear_shape(**a)


def _call_gemm(shape, nbytes, **o):
    g = lambda n: o.get(n, FAKE)
    return moe.lib().fp8_block_gemm(ctypes.byref(shape), g("a"), g("a_scales"), g("w"), g("w_scales"), o.get("residual"),
                                    g("out"), g("ws"), nbytes, None)


def _call_linear(shape, nbytes, **o):
    g = lambda n: o.get(n, FAKE)
    return moe.lib().moe_linear(ctypes.byref(shape), g("x"), g("w"), g("w_scales"), o.get("residual"), g("out"), g("ws"),
                                nbytes, None)


def _call_linear_prenorm(shape, nbytes, gamma=FAKE, eps=1e-6, **o):
    g = lambda n: o.get(n, FAKE)
    return moe.lib().moe_linear_prenorm(ctypes.byref(shape), g("x"), gamma, ctypes.c_float(eps), g("w"), g("w_scales"),
                                        g("out"), g("ws"), nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=(1 << 30) + 1), dict(T=1 << 29), dict(K=0), dict(K=100), dict(K=192), dict(K=(1 << 20) + 128),
    dict(N=0), dict(N=-5), dict(N=(1 << 20) + 1, weight_layout="rowmajor"), dict(N=1 << 20, K=1 << 19), dict(N=1500),
    dict(precision="fp8", weight_layout=2), dict(precision=N.MOE_BF16), dict(precision=9)], ids=str)
def test_linear_bad_shapes(bad):
    s = _linear(**bad)
    assert moe.lib().moe_linear_workspace_size(ctypes.byref(s)) == 0
    assert moe.moe_last_error()
    for call in (_call_gemm, _call_linear, _call_linear_prenorm):
        assert call(s, 1 << 50) == N.MOE_ERR_INVALID_ARG


def test_linear_out_f32_is_a_flag():
    s = _linear()
    s.out_f32 = 2
    assert moe.lib().moe_linear_workspace_size(ctypes.byref(s)) == 0
    with pytest.raises(TypeError):
        moe.make_linear_shape(1, 128, 128, out_dtype=torch.float16)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_linear_host_side_errors(T):
    s = _linear(T=T)
    need = moe.moe_linear_workspace_size(s)
    for call in (_call_gemm, _call_linear, _call_linear_prenorm):
        assert call(s, need - 1) == N.MOE_ERR_WORKSPACE
        for name in ("w", "w_scales", "out"):
            for p in (None, MISALIGNED):
                assert call(s, need, **{name: p}) == N.MOE_ERR_INVALID_ARG, name
        assert call(s, need, ws=None) == N.MOE_ERR_INVALID_ARG
        assert call(s, need, ws=UNALIGNED_WS) == N.MOE_ERR_INVALID_ARG
    for p in (None, MISALIGNED):
        assert _call_gemm(s, need, a=p) == N.MOE_ERR_INVALID_ARG
        assert _call_gemm(s, need, a_scales=p) == N.MOE_ERR_INVALID_ARG
        assert _call_linear(s, need, x=p) == N.MOE_ERR_INVALID_ARG
        assert _call_linear_prenorm(s, need, x=p) == N.MOE_ERR_INVALID_ARG
        assert _call_linear_prenorm(s, need, gamma=p) == N.MOE_ERR_INVALID_ARG
    for call in (_call_gemm, _call_linear):
        assert call(s, need, residual=MISALIGNED) == N.MOE_ERR_INVALID_ARG
    for eps in (-1e-6, float("nan")):
        assert _call_linear_prenorm(s, need, eps=eps) == N.MOE_ERR_INVALID_ARG


def test_linear_empty_batch():
    s = _linear(T=0)
    need = moe.moe_linear_workspace_size(s)
    assert need > 0
    none = dict(w=None, w_scales=None, out=None)
    assert _call_gemm(s, need, a=None, a_scales=None, **none) == N.MOE_OK
    assert _call_linear(s, need, x=None, **none) == N.MOE_OK
    assert _call_linear_prenorm(s, need, x=None, **none) == N.MOE_OK
    assert moe.moe_last_launch_count() == 0


def test_linear_extremes_are_shapes():
    """The largest sizes of each dimension, and one of everything."""
    for kw in (dict(T=1, K=128, N=1, weight_layout="rowmajor"), dict(N=1 << 20, K=1024), dict(N=1024, K=1 << 20),
               dict(T=1 << 23, K=7168, N=7168), dict(T=1 << 29, K=128, N=128)):
        assert moe.moe_linear_workspace_size(_linear(**kw)) > 0, kw


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    b = torch.zeros(1 << 16, dtype=torch.uint8)
    f = torch.zeros(1 << 10)
    s = moe.make_linear_shape(4, 256, 256)
    with pytest.raises(ValueError):
        moe.moe_linear(s, x, b, f, x, b)
    with pytest.raises(ValueError):
        moe.moe_linear_prenorm(s, x, x, 1e-6, b, f, x, b)
    with pytest.raises(ValueError):
        moe.fp8_block_gemm(s, b, f, b, f, x, b)
    with pytest.raises(TypeError):
        moe.moe_linear(s, None, b, f, x, b)
    s = moe.make_shape(4, 256, 16, 4, 128)
    with pytest.raises(ValueError):
        moe.moe_forward_few(s, x, x, f, b, f, b, f, x, b)
    with pytest.raises(ValueError):
        moe.moe_forward_few_prenorm(s, x, x, 1e-6, x, f, b, f, b, f, x, b)
