"""Fp8Linear and MoELayer.forward_few as objects that a program shares: between
streams, threads, graphs and batch sizes.  Overlapping calls give what each
gives alone, bit for bit."""
import copy
import pickle
import threading

import pytest
import torch

import sparse_moe_transformer_fwd_b200 as moe

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def _linear(K=2048, N=1536, seed=1, **kw):
    g = torch.Generator(DEV).manual_seed(seed)
    return moe.Fp8Linear((torch.randn(N, K, generator=g, device=DEV) / K ** 0.5).bfloat16(), **kw)


def _layer(d=1024, E=64, k=8, de=256, precision="fp8", seed=2):
    g = torch.Generator(DEV).manual_seed(seed)
    n = lambda *s: (torch.randn(*s, generator=g, device=DEV) / s[-1] ** 0.5).bfloat16()
    return moe.MoELayer(n(E, d), torch.zeros(E, device=DEV), n(E + 1, 2 * de, d), n(E + 1, d, de), top_k=k,
                        precision=precision)


def _x(T, K, seed):
    return torch.randn(T, K, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).bfloat16()


# (tokens, call): several launches that share the workspace's quantised x, partial
# sums, item counters, pre-normed tokens
CALLS = {
    "linear-40": (40, lambda o, x, g, **kw: o(x, **kw)),
    "linear-300": (300, lambda o, x, g, **kw: o(x, **kw)),
    "linear-prenorm-13": (13, lambda o, x, g, **kw: o.forward_prenorm(x, g, **kw)),
    "few-9": (9, lambda o, x, g, **kw: o.forward_few(x, **kw)),
    "few-prenorm-4": (4, lambda o, x, g, **kw: o.forward_few_prenorm(x, g, **kw)),
}


def _setup(name, count):
    T, call = CALLS[name]
    obj, K = (_layer(), 1024) if name.startswith("few") else (_linear(), 2048)
    xs, gamma = [_x(T, K, i) for i in range(count)], _x(1, K, 99).reshape(-1)
    want = [call(obj, x, gamma).clone() for x in xs]
    torch.cuda.synchronize()
    return obj, T, lambda x, **kw: call(obj, x, gamma, **kw), xs, want


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("passed", [False, True], ids=["current", "argument"])
def test_two_streams_of_one_object(name, passed):
    obj, T, call, xs, want = _setup(name, 4)
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(25):
        for x, o, s in zip(xs, outs, streams):
            if passed:
                call(x, out=o, stream=s)
            else:
                with torch.cuda.stream(s):
                    call(x, out=o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    assert obj.check_status(T) == 0


@pytest.mark.parametrize("name", ["linear-300", "linear-prenorm-13", "few-prenorm-4"])
def test_threads_on_one_stream(name):
    """The launches of two threads' calls do not mix."""
    obj, T, call, xs, want = _setup(name, 4)
    outs = [[torch.empty_like(w) for _ in range(50)] for w in want]
    torch.cuda.synchronize()
    errors = []

    def work(x, out):
        try:
            for o in out:
                call(x, out=o)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(xs, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for out, w in zip(outs, want):
        assert all(torch.equal(o, w) for o in out)
    assert obj.check_status(T) == 0


@pytest.mark.parametrize("name", CALLS)
def test_replays_beside_eager_calls(name):
    """A captured call and eager ones at once; two graphs of two capture streams at once."""
    obj, T, call, xs, want = _setup(name, 3)
    outs = [torch.empty_like(w) for w in want]
    graphs, replay_on = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in (0, 1):
        call(xs[2], out=outs[2])  # a workspace for the capture to take over
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=torch.cuda.Stream()):
            call(xs[i], out=outs[i])
    for _ in range(25):
        for g, s in zip(graphs, replay_on):
            with torch.cuda.stream(s):
                g.replay()
        call(xs[2], out=outs[2])
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    assert obj.check_status(T) == 0
    del graphs


def test_captures_after_one_eager_call():
    """Two captures, on two streams, after one eager call: the second one's
    workspace is its graph's own."""
    lin = _linear()
    xs = [_x(40, 2048, i) for i in range(2)]
    want = [lin(x).clone() for x in xs]
    graphs, outs = [], [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=torch.cuda.Stream()):
            lin(x, out=o)
            lin(x, out=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    assert torch.equal(lin(xs[0]), want[0])
    assert lin.check_status(40) == 0
    del graphs
    with pytest.raises(RuntimeError, match="before the capture"):  # larger than any so far
        big = _x(3000, 2048, 1)
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            lin(big)


def test_one_workspace_for_every_batch_size():
    """The memory of one object is that of its largest call on each stream."""
    lin = _linear()
    sizes = [1, 7, 64, 300, 513, 1024, 2000, 5, 1999]
    xs = {T: _x(T, 2048, T) for T in sizes}
    first = lin(xs[2000])  # what the first call sets up
    assert lin.check_status(2000) == 0
    want = {T: _linear()(xs[T]).clone() for T in sizes}
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(2):
        for T in sizes:
            assert torch.equal(lin(xs[T]), want[T])
    assert torch.cuda.memory_allocated() == before
    assert lin.workspace(1).data_ptr() == lin.workspace(2000).data_ptr()
    layer = _layer()
    layer.forward_few(_x(16, 1024, 1))
    ws = layer.few_workspace(16)
    assert all(layer.few_workspace(T).data_ptr() == ws.data_ptr() for T in range(1, 17))
    del first


def test_a_growing_workspace_under_load():
    """The workspace is replaced by a larger one while calls on the old one are
    still running, and its memory is used again."""
    lin = _linear(K=7168, N=7168)
    sizes = [2, 20, 100, 400, 700, 1500]
    xs = {T: _x(T, 7168, T) for T in sizes}
    want = {T: lin(xs[T]).clone() for T in reversed(sizes)}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    fresh = _linear(K=7168, N=7168)
    outs = {}
    with torch.cuda.stream(side):
        for T in sizes:
            outs[T] = [fresh(xs[T]) for _ in range(3)]
            torch.full((fresh.workspace(T).numel(),), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for T in sizes:
        assert all(torch.equal(o, want[T]) for o in outs[T]), T
    assert fresh.check_status(1500) == 0


def test_outputs_are_the_calls_streams_memory():
    """An output that a call makes on stream= comes out of that stream's memory: a
    block that the current stream frees later and takes again is not one that the
    call still writes, and the other way round."""
    lin, layer = _linear(), _layer()
    dense = moe.DenseFFN(_x(512, 1024, 1), _x(1024, 256, 2))
    x, y, gamma = _x(40, 2048, 1), _x(9, 1024, 2), _x(1, 1024, 3).reshape(-1)
    calls = [lambda **kw: lin(x, **kw), lambda **kw: lin.forward_prenorm(x, x[0].contiguous(), **kw),
             lambda **kw: layer.forward_few(y, **kw), lambda **kw: layer.forward_few_prenorm(y, gamma, **kw),
             lambda **kw: layer(y, **kw), lambda **kw: layer.forward_prenorm(y, gamma, **kw),
             lambda **kw: dense(y, **kw), lambda **kw: dense.forward_prenorm(y, gamma, **kw)]
    side = torch.cuda.Stream()

    class Handle:  # what else has a stream's handle
        cuda_stream = side.cuda_stream

    for call in calls:
        want = call()
        for stream in (side, Handle()):
            torch.cuda.synchronize()
            out = call(stream=stream)
            side.synchronize()
            assert torch.equal(out, want)
            at, shape = out.data_ptr(), out.shape
            del out
            again = [torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
            assert at not in [t.data_ptr() for t in again]
            with torch.cuda.stream(side):
                assert torch.empty(shape, dtype=torch.bfloat16, device=DEV).data_ptr() == at


def test_shapes_that_objects_refuse():
    """Tensors with enough elements in other rows: a batch in more dimensions than
    two, longer rows, columns of another width."""
    lin, layer = _linear(K=512, N=640), _layer(d=512)
    x, gamma = _x(4, 512, 1), _x(1, 512, 3).reshape(-1)
    q, s = torch.empty(4, 512, dtype=torch.uint8, device=DEV), torch.empty(4, 4, device=DEV)
    moe.fp8_block_quant(x, 1, q, s)
    wide = torch.zeros(4, 1024, dtype=torch.bfloat16, device=DEV)
    cube = _x(8, 512, 2).reshape(2, 4, 512)
    for bad in (wide, cube, wide.reshape(2, -1)):
        for call in (lin, layer.forward_few, lambda t: lin.forward_prenorm(t, gamma),
                     lambda t: layer.forward_few_prenorm(t, gamma)):
            with pytest.raises(ValueError, match="expected \\[T, 512\\]"):
                call(bad)
    with pytest.raises(ValueError, match="a_scales"):
        lin.quantized(q, torch.zeros(4, 8, device=DEV))
    with pytest.raises(ValueError, match="a: shape"):
        lin.quantized(torch.zeros(4, 1024, dtype=torch.uint8, device=DEV), s)
    for name in ("out", "residual"):
        with pytest.raises(ValueError, match=name):
            lin(x, **{name: wide})
    with pytest.raises(ValueError, match="gamma"):
        lin.forward_prenorm(x, wide[0])
    with pytest.raises(ValueError, match="gamma"):
        layer.forward_few_prenorm(x, wide[0])
    with pytest.raises(ValueError, match="out"):
        layer.forward_few(x, out=wide)
    with pytest.raises(ValueError, match="topk_idx_out"):
        layer.forward_few(x, topk_idx_out=torch.zeros(4, 16, dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError):
        lin(None)
    # what says the same rows in another way, and longer outputs, are taken
    want = lin(x)
    assert torch.equal(lin(x.reshape(4, 1, 512)), want)
    out = torch.full((6, 640), 3.0, dtype=torch.bfloat16, device=DEV)
    lin(x, out=out, residual=torch.zeros_like(out))
    assert torch.equal(out[:4], want) and torch.all(out[4:] == 3.0)
    flat = torch.empty(4 * 640, dtype=torch.bfloat16, device=DEV)
    lin(x, out=flat)
    assert torch.equal(flat.reshape(4, 640), want)
    assert torch.equal(lin.forward_prenorm(x, gamma.reshape(1, 512)), lin.forward_prenorm(x, gamma))


@pytest.mark.parametrize("T", [1, 5, 16, 17, 64, 300])
def test_in_place(T):
    """The output in the input's memory, and in what follows it: projections of equal
    widths, the residual as well, behind the pre-norm; codes beside the output."""
    K = 1536
    lin, gamma = _linear(K=K, N=K), _x(1, K, 3).reshape(-1)
    x = _x(T, K, 1)
    want = lin(x), lin(x, residual=x), lin.forward_prenorm(x, gamma)
    for w, call in zip(want, (lambda b: lin(b, out=b), lambda b: lin(b, out=b, residual=b),
                              lambda b: lin.forward_prenorm(b, gamma, out=b))):
        for _ in range(3):
            buf = x.clone()
            call(buf)
            assert torch.equal(buf, w)
    long = torch.zeros(T + 1, K, dtype=torch.bfloat16, device=DEV)
    long[:T] = x
    lin(long[:T], out=long[1:])
    assert torch.equal(long[1:], want[0])
    both = torch.empty(T * K * 3, dtype=torch.uint8, device=DEV)
    s = torch.empty(T, K // 128, device=DEV)
    moe.fp8_block_quant(x, 1, both[: T * K], s)
    codes, out = both[: T * K].reshape(T, K), both[T * K :].view(torch.bfloat16).reshape(T, K)
    clean = lin.quantized(codes.clone(), s)
    assert torch.equal(lin.quantized(codes, s, out=out), clean)
    with pytest.raises(moe.MoeError, match="overlaps"):
        lin.quantized(codes, s, out=both[: 2 * T * K].view(torch.bfloat16).reshape(T, K))
    assert lin.check_status() == 0


@pytest.mark.parametrize("precision", ["fp8", "bf16"])
@pytest.mark.parametrize("T", [1, 7, 16])
def test_few_in_place(T, precision):
    layer, gamma = _layer(precision=precision), _x(1, 1024, 3).reshape(-1)
    x = _x(T, 1024, 1)
    want = layer.forward_few(x), layer.forward_few_prenorm(x, gamma)
    for _ in range(5):
        a, b = x.clone(), x.clone()
        layer.forward_few(a, out=a)
        layer.forward_few_prenorm(b, gamma, out=b)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert layer.check_status(T) == 0


def test_copies_and_pickles():
    """An object's copy has workspaces of its own."""
    lin, layer = _linear(K=512, N=640), _layer(d=512)
    x, y = _x(40, 512, 1), _x(4, 512, 2)
    want = lin(x), layer.forward_few(y)
    for again in (copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))):
        a, b = again(lin), again(layer)
        assert torch.equal(a(x), want[0]) and torch.equal(b.forward_few(y), want[1])
        assert a.workspace(40).data_ptr() != lin.workspace(40).data_ptr()
        assert a.check_status() == 0 and b.check_status(4) == 0
