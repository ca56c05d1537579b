"""Calls of the block-scaled linear and of moe_forward_few at their edges:
borders between the kernels and their column groups, outputs and weights beyond
2^31 elements, padded outputs, overlapping calls, shared workspaces, a wait that
runs out.  Tolerances are those of the operators' own tests."""
import os
import subprocess
import sys

import pytest
import torch

import oracle
import sparse_moe_transformer_fwd_b200 as moe

from _gpu_util import u16
from test_gpu_few import Layer, _check as _check_few, _x
from test_gpu_linear import _check, _inputs, _quant, _values

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


# groups of 64 columns, whole and ragged; the last batch that streams and the
# first that cannot; few rows of weights (cut into parts) and two rounds of them
@pytest.mark.parametrize("T,K,N", [(65, 1536, 200), (127, 7168, 257), (128, 512, 640), (129, 384, 1000), (191, 7168, 128),
                                   (512, 2048, 131), (513, 2048, 131), (64, 256, 40000), (130, 128, 20000), (2, 256, 40064),
                                   (700, 384, 999)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_borders_with_residual(T, K, N, out_dtype):
    x, lin, w, g = _inputs(T, K, N, "fp8", "rowmajor", seed=T + N)
    lin.out_dtype = out_dtype
    res = torch.randn(T, N, generator=g).bfloat16().to(DEV)
    a = _quant(x, "fp8")[2]
    xd = x.to(DEV)
    out = lin(xd, residual=res)
    _check(out, a, w, residual=res)
    _check(lin(xd), a, w)
    for _ in range(3):  # counters are back at zero
        assert torch.equal(lin(xd, residual=res), out)
    assert lin.check_status(T) == 0


# the tiled GEMM: padded and odd widths, one round of tiles and more (the rest
# cut in ranges of K), the block-scaled MMA where it applies
@pytest.mark.parametrize("T,K,N", [(700, 512, 640), (700, 1152, 999), (2048, 2048, 2560), (2300, 1152, 2531), (1000, 128, 72),
                                   (600, 7168, 136)])
@pytest.mark.parametrize("precision", ["fp8", "fp8_ue8m0"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_tiled(T, K, N, precision, out_dtype):
    x, lin, w, g = _inputs(T, K, N, precision, "rowmajor", seed=T + N)
    lin.out_dtype = out_dtype
    res = torch.randn(T, N, generator=g).bfloat16().to(DEV)
    a = _quant(x, precision)[2]
    xd = x.to(DEV)
    _check(lin(xd), a, w)
    out = lin(xd, residual=res)
    _check(out, a, w, residual=res)
    assert torch.equal(lin(xd, residual=res), out)
    assert lin.check_status(T) == 0


@pytest.mark.parametrize("T", [1, 3, 16, 40, 100, 300, 700])
@pytest.mark.parametrize("N", [640, 999])
def test_residual_in_place_and_rows_behind_the_batch(T, N):
    """The residual's memory as the output; a buffer longer than the batch keeps
    what lies behind."""
    x, lin, w, g = _inputs(T, 1536, N, "fp8", "rowmajor", seed=T)
    res = torch.randn(T + 5, N, generator=g).bfloat16().to(DEV)
    xd = torch.cat([x, torch.full((5, 1536), float("nan"), dtype=torch.bfloat16)]).to(DEV)
    want = lin(xd[:T], residual=res[:T].clone())
    buf = res.clone()
    sh = lin.shape(T)
    moe.moe_linear(sh, xd, lin.w, lin.w_scales, buf, lin.workspace(T), residual=buf)
    assert torch.equal(buf[:T], want) and torch.equal(buf[T:], res[T:])
    f32 = torch.full((T + 5, N), 7.0, device=DEV)
    sf = moe.make_linear_shape(T, 1536, N, "fp8", "rowmajor", torch.float32)
    moe.moe_linear(sf, xd, lin.w, lin.w_scales, f32, moe.alloc_linear_workspace(sf, DEV))
    assert torch.all(f32[T:] == 7.0)


def _big(rows, cols, seed):
    return torch.randn(rows, cols, device=DEV, dtype=torch.bfloat16, generator=torch.Generator(DEV).manual_seed(seed))


@pytest.mark.parametrize("T,K,N", [(300001, 7168, 128), (524300, 128, 4096), (262200, 128, 8200)])
def test_activations_beyond_32_bits(T, K, N):
    """T * K or T * N past 2^31: the first and last rows."""
    x = _big(T, K, 1)
    w = (torch.randn(N, K, generator=torch.Generator().manual_seed(2)) / K ** 0.5).bfloat16()
    lin = moe.Fp8Linear(w.to(DEV), weight_layout="rowmajor")
    out = lin(x)
    assert lin.check_status(T) == 0
    wv = _values(*oracle.block_quant(u16(w), 128), 128)
    for rows in (slice(0, 3), slice(T // 2, T // 2 + 3), slice(T - 3, T)):
        _check(out[rows], _quant(x[rows].cpu(), "fp8")[2], wv)
    del x, out, lin
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,layout", [(2, "tiled"), (2, "rowmajor"), (80, "tiled"), (300, "rowmajor")])
def test_weights_beyond_32_bits(T, layout):
    """N * K past 2^31: the last output columns."""
    N, K = 300032, 7168
    w = _big(N, K, 3)
    lin = moe.Fp8Linear(w, weight_layout=layout)
    tail = w[-256:].cpu()
    del w
    x = _x(T, K, 5)
    out = lin(x.to(DEV))
    assert lin.check_status(T) == 0
    _check(out[:, -256:], _quant(x, "fp8")[2], _values(*oracle.block_quant(u16(tail), 128), 128))
    del out, lin
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,K,N", [(3, 1 << 20, 130), (40, 1 << 17, 40), (1, 128, 1 << 20), (20, 256, (1 << 19) + 5), (600, 1 << 16, 24)])
def test_longest_sizes(T, K, N):
    """The limits of K and N: many parts of one tile, many rounds of short ones."""
    x, lin, w, _ = _inputs(T, K, N, "fp8", "rowmajor", seed=7)
    out = lin(x.to(DEV))
    assert lin.check_status(T) == 0
    _check(out, _quant(x, "fp8")[2], w)
    assert torch.equal(lin(x.to(DEV)), out)


def test_graphs_that_share_a_workspace():
    """Captured calls of different shapes on one workspace, replayed in turn."""
    shapes = [(2, 7168, 640), (40, 512, 999), (3, 256, 40064), (300, 1536, 256)]
    lins = [_inputs(T, K, N, "fp8", "rowmajor", seed=K) for T, K, N in shapes]
    ws = torch.zeros(max(moe.moe_linear_workspace_size(l.shape(s[0])) for s, (_, l, _, _) in zip(shapes, lins)),
                     dtype=torch.uint8, device=DEV)
    static = [(x.to(DEV), torch.empty(T, N, dtype=torch.bfloat16, device=DEV)) for (T, _, N), (x, _, _, _) in zip(shapes, lins)]
    graphs = []
    torch.cuda.synchronize()
    for (T, _, _), (_, lin, _, _), (x, out) in zip(shapes, lins, static):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            moe.moe_linear(lin.shape(T), x, lin.w, lin.w_scales, out, ws)
            moe.moe_linear(lin.shape(T), x, lin.w, lin.w_scales, out, ws)
    for seed in range(3):
        for (T, K, _), (_, lin, _, _), (x, out), graph in zip(shapes, lins, static, graphs):
            x.copy_(_x(T, K, seed))
            out.zero_()
            graph.replay()
            want = lin(x)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    del graphs
    assert moe.moe_check_status(ws) == 0


def test_first_call_on_another_stream():
    """A new object's workspace is zero before the first call reads it, whatever
    stream that call is on."""
    w = (torch.randn(640, 7168, generator=torch.Generator().manual_seed(1)) / 85).bfloat16().to(DEV)
    x = _x(3, 7168, 1).to(DEV)
    want = moe.Fp8Linear(w)(x)
    L = Layer(512, 16, 4, 256, 1, "fp8", "tiled", seed=5)
    xf = _x(4, 512, 2).to(DEV)
    wantf = L.lib.forward_few(xf)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    junk = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        lin = moe.Fp8Linear(w)
        L.lib._few_ws.clear()
        out, outf = torch.empty_like(want), torch.empty_like(wantf)
        del junk  # the workspace may come from memory that was not zero
        torch.cuda.synchronize()
        lin(x, out=out, stream=side)
        L.lib.forward_few(xf, out=outf, stream=side)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(outf, wantf)
        junk = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)


def test_overlapping_calls():
    """Calls on two streams at once, a workspace each."""
    L = Layer(1024, 64, 8, 256, 1, "fp8", "tiled", seed=9)
    g = torch.Generator().manual_seed(1)
    lin = moe.Fp8Linear((torch.randn(2112, 1024, generator=g) / 32).bfloat16().to(DEV), weight_layout="rowmajor")
    xs = [_x(T, 1024, T).to(DEV) for T in (2, 9)]
    want = [(L.lib.forward_few(x).clone(), lin(x).clone()) for x in xs]
    ws = [(moe.alloc_few_workspace(L.lib.shape(9), DEV), moe.alloc_linear_workspace(lin.shape(9), DEV)) for _ in xs]
    outs = [(torch.empty_like(a), torch.empty_like(b)) for a, b in want]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    m = L.lib
    for _ in range(30):
        for x, s, (fw, lw), (o, p) in zip(xs, streams, ws, outs):
            moe.moe_linear(lin.shape(x.shape[0]), x, lin.w, lin.w_scales, p, lw, stream=s)
            moe.moe_forward_few(m.shape(x.shape[0]), x, m.w_router, m.bias, m.w13, m.w13s, m.w2, m.w2s, o, fw, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])
    for fw, lw in ws:
        assert moe.moe_check_status(fw) == 0 and moe.moe_check_status(lw) == 0


def test_capture_needs_a_workspace_made_before():
    lin = moe.Fp8Linear((torch.randn(128, 128) / 12).bfloat16().to(DEV))
    x = _x(2, 128, 1).to(DEV)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            lin(x)
    assert torch.isfinite(lin(x).float()).all()


def test_few_same_tokens_and_rows_behind():
    """The same token sixteen times gives the same row sixteen times; rows of a
    longer output keep what they held."""
    L = Layer(512, 32, 8, 256, 1, "fp8", "tiled", seed=2)
    x = _x(1, 512, 4).repeat(16, 1)
    out = torch.full((20, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    m = L.lib
    moe.moe_forward_few(m.shape(16), x.to(DEV), m.w_router, m.bias, m.w13, m.w13s, m.w2, m.w2s, out, m.few_workspace(16))
    assert torch.all(out[:16] == out[0]) and torch.all(out[16:] == 3.0)
    _, want, tol = L.reference(x)
    _check_few(out[:16], want, tol)


def test_few_routes_any_values_as_moe_route():
    """Infinities, NaN, zeros and huge values in x: the experts moe_route selects."""
    L = Layer(512, 64, 8, 128, 1, "fp8", "tiled", seed=3)
    x = _x(8, 512, 6)
    x[1, 3], x[2, 5], x[3, 7], x[4] = float("inf"), float("-inf"), float("nan"), 0
    x[5], x[6] = x[5] * 1e30, x[6] * 1e-30
    xd = x.to(DEV)
    idx = torch.empty(8, 8, dtype=torch.int32, device=DEV)
    L.lib.forward_few(xd, topk_idx_out=idx)
    sh, ref, gates = L.lib.shape(8), torch.empty_like(idx), torch.empty(8, 8, device=DEV)
    moe.moe_route(sh, xd, L.lib.w_router, L.lib.bias, ref, gates, L.lib.workspace(8))
    assert torch.equal(idx, ref)
    assert L.lib.check_status(8) == 0


def test_few_wait_that_runs_out(monkeypatch):
    """The exact routing waits for a block that does not exist: the call reports
    MOE_ERR_TIMEOUT through the status word, leaves its counters zero, and the
    next call is right."""
    L = Layer(512, 16, 4, 256, 1, "fp8", "tiled", seed=4)
    x = _x(3, 512, 1)
    monkeypatch.setenv("MOE_FAULT_INJECT", "few_scored")
    L.lib.forward_few(x.to(DEV))
    monkeypatch.delenv("MOE_FAULT_INJECT")
    assert moe.moe_check_status(L.lib.few_workspace(3)) == moe._native.MOE_ERR_TIMEOUT
    out = L.lib.forward_few(x.to(DEV))
    assert L.lib.check_status(3) == 0
    _check_few(out, *L.reference(x)[1:])


def test_first_calls_of_a_process_captured():
    """Nothing that the first call sets up stands in the way of a capture."""
    code = """
import torch, sparse_moe_transformer_fwd_b200 as moe
d, E, de, T = 256, 8, 128, 3
g = torch.Generator("cuda").manual_seed(0)
r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
L = moe.MoELayer(r(E, d), torch.zeros(E, device="cuda"), r(E + 1, 2 * de, d), r(E + 1, d, de), top_k=2)
lin = moe.Fp8Linear(r(640, 7168))
x, y = r(T, d), r(T, 7168)
out, lout = torch.empty(T, d, device="cuda").bfloat16(), torch.empty(T, 640, device="cuda").bfloat16()
L.few_workspace(T), lin.workspace(T)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    L.forward_few(x, out=out)
    lin(y, out=lout)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, L.forward_few(x)) and torch.equal(lout, lin(y))
assert L.check_status(T) == 0 and lin.check_status(T) == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "captured" in p.stdout, p.stderr[-2000:]


def test_checked_calls_from_c():
    """The binding's C functions make a good call, decline (None) whatever the
    call does not take, and hold on to nothing."""
    lin = moe.Fp8Linear((torch.randn(256, 512) / 20).bfloat16().to(DEV))
    x, out, ws, sh = _x(4, 512, 1).to(DEV), torch.empty(4, 256, dtype=torch.bfloat16, device=DEV), lin.workspace(4), lin.shape(4)
    fast = moe._native._fast("linear")
    good = dict(kind=1, shape=sh, x=x, second=None, eps=0.0, w=lin.w, w_scales=lin.w_scales, residual=None, out=out, ws=ws,
                stream=None)
    call = lambda **o: fast(*{**good, **o}.values())
    assert call() == 0 and torch.equal(out, lin(x))
    assert call(stream=torch.cuda.Stream()) == 0
    held = (x, out, ws, lin.w, lin.w_scales, sh)
    before = [sys.getrefcount(t) for t in held]
    bad = dict(x=[x.cpu(), x.float(), x[:, ::2], x[:3], None, 3], w=[lin.w[:100], lin.w.cpu(), lin.w.int()],
               w_scales=[lin.w_scales.double()], residual=[out.float(), out[:3]], out=[out[:3], out.float(), out.t()],
               ws=[None, ws.float()], shape=[L_shape(), 5, None], eps=["a"], kind=[None], stream=[7])
    for name, values in bad.items():
        for v in values:
            assert call(**{name: v}) is None, (name, v)
    for _ in range(100):
        call()
    del v, values
    bad.clear()
    assert [sys.getrefcount(t) for t in held] == before
    few = moe._native._fast("few")
    L = Layer(256, 8, 2, 128, 1, "fp8", "tiled", seed=1).lib
    x = _x(4, 256, 1).to(DEV)
    out = torch.empty_like(x)
    good = dict(prenorm=False, shape=L.shape(4), x=x, gamma=None, eps=0.0, w_router=L.w_router, bias=L.bias, w13=L.w13, s13=L.w13s,
                w2=L.w2, s2=L.w2s, out=out, ws=L.few_workspace(4), idx=None, stream=None)
    call = lambda **o: few(*{**good, **o}.values())
    assert call() == 0 and torch.equal(out, L.forward_few(x))
    for name in ("x", "w_router", "bias", "w13", "s13", "w2", "s2", "out", "ws"):
        assert call(**{name: good[name].cpu()}) is None, name
        assert call(**{name: good[name].reshape(-1)[:-1] if name != "ws" else good[name].float()}) is None, name
    assert call(idx=torch.empty(8, dtype=torch.int64, device=DEV)) is None
    assert few(1, 2, 3) is None and fast() is None


def L_shape():
    return moe.make_shape(4, 256, 8, 2, 128)
