"""GPU tests of layers with an epilogue and of the block on several streams and in
several graphs at once.  Needs a B200."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    import hadamard_rotated_bit_token_b200 as hq_mod
    from hadamard_rotated_bit_token_b200 import build as hq_build
    hq_build.build()
    hq_mod.load_library()
    return hq_mod


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _calls(hq, kind, g):
    """A call of inputs X [T, C] and its X's shape."""
    C = 512
    W = _bf(g, C, C, scale=C ** -0.5)
    if kind == "group_wise":
        layer = hq.GroupWiseQuantLinear(hq.GwDesc(C, C, 64, 32), W)
        block = hq.PointwiseBlock(hq.GroupNorm(C, 32, act=hq.HQ_ACT_SILU), layer)
        return block, (2, 400, C)
    per_tensor = kind == "per_tensor"
    desc = hq.LayerDesc(C, C, 128, a_bits=8, w_bits=8, centering=hq.HQ_CENTER_NONE,
                        act_gran=hq.HQ_PER_TENSOR_DYNAMIC if per_tensor else hq.HQ_PER_TOKEN)
    layer = hq.HadamardQuantLinear(desc, W)
    if kind == "epilogue":
        return (lambda X: layer.forward(X, epilogue=hq.Epilogue(hq.HQ_ACT_GELU, X))), (3000, C)
    if kind == "plain":
        return layer, (3000, C)
    return hq.PointwiseBlock(hq.GroupNorm(C, 32), layer, residual=True), (2, 1500, C)


KINDS = ["plain", "epilogue", "per_token", "per_tensor", "group_wise"]


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(hq, kind):
    """Calls of one layer with equal numbers of tokens, many in flight on two
    streams: each gives what it gives alone."""
    g = _gen(len(kind))
    call, shape = _calls(hq, kind, g)
    Xs = [_bf(g, *shape, scale=s) for s in (1.0, 3.0)]
    want = [call(X).clone() for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    outs = []
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs.append((i, call(Xs[i])))
    torch.cuda.synchronize()
    assert all(torch.equal(Y, want[i]) for i, Y in outs)
    assert hq.hq_check_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_two_graphs_at_once(hq, kind):
    """Two graphs of one layer, replayed at the same time on two streams."""
    g = _gen(len(kind) + 7)
    call, shape = _calls(hq, kind, g)
    Xs = [_bf(g, *shape, scale=s) for s in (1.0, 3.0)]
    want = [call(X).clone() for X in Xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for X in Xs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call(X))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in Xs]
    for _ in range(20):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    # and an eager call beside them
    eager = call(Xs[0])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert torch.equal(eager, want[0])
    assert hq.hq_check_device_error() == 0


def test_buffers_hold_what_the_last_call_on_this_stream_left(hq):
    g = _gen(3)
    T, C = 70, 256
    layer = hq.HadamardQuantLinear(hq.LayerDesc(C, C, 128), _bf(g, C, C))
    X1, X2 = _bf(g, T, C), _bf(g, T, C)
    layer(X1)
    codes = layer.buffers(T)["a_codes"].clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        layer(X2)
    torch.cuda.synchronize()
    assert torch.equal(layer.buffers(T)["a_codes"], codes)
    layer(X2)
    assert not torch.equal(layer.buffers(T)["a_codes"], codes)


@pytest.mark.parametrize("shape", [(0, 5, 256), (2, 0, 256), (0, 256), (1, 256), (1, 1, 1, 256)])
def test_block_of_no_or_one_pixel(hq, shape):
    g = _gen(4)
    C = 256
    layer = hq.HadamardQuantLinear(hq.LayerDesc(C, C, 128, a_bits=8, w_bits=8), _bf(g, C, C))
    X = _bf(g, *shape)
    Y = hq.PointwiseBlock(hq.GroupNorm(C, 32), layer, residual=True)(X)
    assert Y.shape == X.shape and bool(Y.isfinite().all())
    Y = hq.PointwiseBlock(hq.GroupNorm(C, 32), layer, act=hq.HQ_ACT_RELU)(X)
    assert Y.shape == X.shape and bool((Y >= 0).all())
    assert hq.hq_check_device_error() == 0
