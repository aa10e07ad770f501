"""GPU tests of the operators beside the quantized layer (include/hq_ops.h)
against their plain 64-bit forms (ops_ref).  Needs a B200."""
import pytest

torch = pytest.importorskip("torch")

from ops_ref import (ACTS, GELU, GELU_TANH, NONE, RELU, SILU, check_rounded, dense64,  # noqa: E402
                     epilogue64, group_norm64, linear64, pack_i4, rel_frob)

pytestmark = pytest.mark.gpu

# a bf16 rounding alone leaves a root-mean-square error of 0.0016 to 0.0017
# relative to the result's norm
ROUND_FROB = 0.0019


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


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _bf(t):
    return t.to(torch.bfloat16)


def _guarded(T, N):
    """Y [T, N] inside a larger buffer of a poison value: (Y, check)."""
    buf = torch.full((T + 3, N), 123.0, dtype=torch.bfloat16, device="cuda")
    Y = buf[1:T + 1]
    if (Y.data_ptr() & 15) != 0:
        Y = buf[2:T + 2]
    lo = (Y.data_ptr() - buf.data_ptr()) // (2 * N)

    def check():
        assert bool((buf[:lo] == 123.0).all()) and bool((buf[lo + T:] == 123.0).all()), \
            "rows outside Y were written"
    return Y, check


# ------------------------------------------------------------------ hq_dense
DENSE_SHAPES = [
    (1, 8, 8), (1, 256, 1152), (2, 1152, 6912), (3, 72, 40), (7, 520, 264), (16, 1000, 72),
    (17, 136, 1144), (33, 64, 128), (64, 4608, 1152), (65, 1152, 136), (127, 200, 328),
    (128, 128, 256), (129, 1160, 776), (257, 4096, 512), (1000, 2600, 1160), (2049, 320, 320),
    (300, 8, 2048), (4100, 1152, 1152),
    # few tokens and narrow layers: every split and token tile of the K split
    (5, 4096, 4096), (9, 64, 128), (10, 192, 136), (24, 8192, 512), (31, 320, 1000),
    (48, 2304, 3456), (96, 1600, 144), (200, 4608, 264), (400, 72, 72), (12, 15000, 8),
]


@pytest.mark.parametrize("T,K,N", DENSE_SHAPES)
def test_dense_integers_are_exact(hq, T, K, N):
    """Integer operands whose sums fp32 holds exactly: any wrong, missing or
    doubled product shows."""
    g = _gen(T * 7 + K + N)
    X = _bf(torch.randint(-3, 4, (T, K), generator=g, device="cuda").float())
    W = _bf(torch.randint(-3, 4, (N, K), generator=g, device="cuda").float())
    b = _bf(torch.randint(-8, 9, (N,), generator=g, device="cuda").float())
    Y, check = _guarded(T, N)
    hq.hq_dense(hq.DenseDesc(K, N), X, W, b, None, Y)
    assert hq.hq_check_device_error() == 0
    z = X.double() @ W.double().t() + b.double()
    assert torch.equal(Y, z.float().bfloat16())
    check()


@pytest.mark.parametrize("T,K,N", DENSE_SHAPES)
@pytest.mark.parametrize("form", range(3))
def test_dense_epilogue(hq, T, K, N, form):
    g = _gen(T + K * 3 + N * 5 + form)
    X, W = _bf(_randn(g, T, K)), _bf(_randn(g, N, K) * K ** -0.5)
    act = (SILU, GELU, GELU_TANH, RELU, NONE)[(T + form) % 5]
    b = _bf(_randn(g, N)) if form != 1 else None
    R = _bf(_randn(g, T, N)) if form != 0 else None
    rows = (0, 1, max(1, T // 3))[form]
    G = _bf(_randn(g, -(-T // rows), N)) if rows else None
    Y, check = _guarded(T, N)
    hq.hq_dense(hq.DenseDesc(K, N), X, W, b, hq.Epilogue(act, R, G, rows), Y)
    assert hq.hq_check_device_error() == 0
    z, ztol = dense64(X, W, b)
    y, tol = epilogue64(z, ztol, act, R, G, rows)
    check_rounded(Y, y, tol, f"dense {T}x{K}x{N} act {act}")
    if T * N > 4000:
        assert rel_frob(Y, y) < ROUND_FROB
    check()


@pytest.mark.parametrize("act", sorted(ACTS.values()))
@pytest.mark.parametrize("T", [1, 13, 400])
def test_dense_activation_values(hq, act, T):
    """Every activation over its range, tails, zeros and the largest values, T
    rows a call: a product with the identity hands bf16 values through
    unchanged."""
    K = N = 64
    vals = torch.cat((torch.linspace(-12, 12, 40 * N - 12), torch.tensor(
        [0.0, -0.0, 1e-30, -1e-30, 30.0, -30.0, 88.0, -88.0, 1e4, -1e4, 3e38, -3e38])))
    I = _bf(torch.eye(K, device="cuda"))
    for V in _bf(vals.cuda()).view(-1, N).repeat(10 if T > 40 else 1, 1).split(T):
        Y = torch.empty(V.shape[0], N, dtype=torch.bfloat16, device="cuda")
        hq.hq_dense(hq.DenseDesc(K, N), V, I, None, hq.Epilogue(act), Y)
        y, tol = epilogue64(V.double(), torch.zeros_like(V.double()), act)
        check_rounded(Y, y, tol, f"act {act}")
    assert hq.hq_check_device_error() == 0


def test_dense_nonfinite(hq):
    """A NaN or infinity reaches only its own row (or its own column), and relu
    keeps a NaN."""
    for T in (5, 200):
        K, N = 128, 192
        g = _gen(T)
        X, W = _bf(_randn(g, T, K)), _bf(_randn(g, N, K))
        X[1, 3] = float("nan")
        X[2, 7] = float("inf")
        for act in (NONE, RELU):
            Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
            hq.hq_dense(hq.DenseDesc(K, N), X, W, None, hq.Epilogue(act), Y)
            assert bool(Y[1].isnan().all())
            big = (W[:, 7].float() * float("inf"))
            want = torch.where(big < 0, torch.zeros_like(big), big) if act == RELU else big
            assert torch.equal(Y[2].float().nan_to_num(1.0, 2.0, 3.0),
                               want.nan_to_num(1.0, 2.0, 3.0))
            rest = [i for i in range(T) if i not in (1, 2)]
            assert bool(Y[rest].isfinite().all())
        # a NaN weight: its own column only, under every activation
        X, W = _bf(_randn(g, T, K)), _bf(_randn(g, N, K))
        W[8, 5] = float("nan")
        W[33, 5] = float("nan")
        for act in sorted(ACTS.values()):
            Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
            hq.hq_dense(hq.DenseDesc(K, N), X, W, None, hq.Epilogue(act), Y)
            cols = Y.isnan().any(dim=0).nonzero().flatten().tolist()
            assert cols == [8, 33] and bool(Y[:, [8, 33]].isnan().all())


@pytest.mark.parametrize("T", [1, 4, 40, 130, 1500])
def test_dense_in_place_residual_and_determinism(hq, T):
    K, N = 520, 712
    g = _gen(T)
    X, W, b = _bf(_randn(g, T, K)), _bf(_randn(g, N, K) * 0.05), _bf(_randn(g, N))
    R = _bf(_randn(g, T, N))
    d = hq.DenseDesc(K, N)
    Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    hq.hq_dense(d, X, W, b, hq.Epilogue(GELU, R), Y)
    Z = R.clone()
    hq.hq_dense(d, X, W, b, hq.Epilogue(GELU, Z), Z)
    assert torch.equal(Y, Z)
    for _ in range(3):
        Z = R.clone()
        hq.hq_dense(d, X, W, b, hq.Epilogue(GELU, Z), Z)
        assert torch.equal(Y, Z)
    assert hq.hq_check_device_error() == 0


@pytest.mark.parametrize("T", [1, 4, 40, 130, 1500])
def test_linear_ep_in_place_residual(hq, T):
    """Added in place, on every code format, again and again the same bits."""
    K, N = 544, 720
    g = _gen(T)
    A, W = _codes(g, T, K, 4), _codes(g, N, K, 4)
    sx, sw, b = torch.rand(T, generator=g, device="cuda"), torch.rand(
        N, generator=g, device="cuda") * 0.01, _randn(g, N)
    R = _bf(_randn(g, T, N))
    for fmt, codes in ((hq.HQ_CODES_I8, A), (hq.HQ_CODES_I4_PACKED, pack_i4(A))):
        desc = hq.LayerDesc(K, N, 16, code_format=fmt)
        Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        hq.hq_linear_ep(desc, codes, sx, None, W, sw, None, b, hq.Epilogue(SILU, R), Y)
        for _ in range(3):
            Z = R.clone()
            hq.hq_linear_ep(desc, codes, sx, None, W, sw, None, b, hq.Epilogue(SILU, Z), Z)
            assert torch.equal(Y, Z)
    assert hq.hq_check_device_error() == 0


def test_products_on_two_streams_at_once(hq):
    """Many calls of every kernel kind in flight on two streams."""
    g = _gen(12)
    cases = []
    for T, K, N in ((1, 1152, 1152), (8, 512, 640), (30, 2304, 1152), (200, 1152, 1152),
                    (3000, 1152, 1152)):
        X, W = _bf(_randn(g, T, K)), _bf(_randn(g, N, K) * 0.03)
        layer = hq.DenseLinear(W, None, GELU)
        cases.append((layer, X, layer(X)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):
        for layer, X, want in cases:
            for st in streams:
                with torch.cuda.stream(st):
                    outs.append((layer(X), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)
    assert hq.hq_check_device_error() == 0


def test_dense_gate_rows_cross_tiles(hq):
    """Gate rows of every length against tiles of 128 rows."""
    K, N, T = 64, 96, 515
    g = _gen(3)
    X, W = _bf(_randn(g, T, K)), _bf(_randn(g, N, K) * 0.1)
    z, ztol = dense64(X, W, None)
    for rows in (1, 2, 31, 32, 33, 127, 128, 129, 500, 514, 515, 516, 10 ** 12):
        G = _bf(_randn(g, -(-T // rows), N))
        Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        hq.hq_dense(hq.DenseDesc(K, N), X, W, None, hq.Epilogue(SILU, None, G, rows), Y)
        y, tol = epilogue64(z, ztol, SILU, None, G, rows)
        check_rounded(Y, y, tol, f"gate_rows {rows}")


def test_dense_zero_rows(hq):
    d = hq.DenseDesc(64, 64)
    W = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    E = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    hq.hq_dense(d, E, W, None, None, E.clone())
    assert hq.DenseLinear(W, None, GELU)(E).shape == (0, 64)


def test_dense_side_stream_and_graph(hq):
    """On a stream of its own, and captured twice and replayed with new inputs."""
    K, N = 1152, 1152
    g = _gen(9)
    W, b = _bf(_randn(g, N, K) * 0.03), _bf(_randn(g, N))
    layer = hq.DenseLinear(W, b, SILU)
    for T in (2, 50, 700):
        X = _bf(_randn(g, T, K))
        want = layer(X)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = layer(X)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got, want)
        Xs = X.clone()
        graphs, outs = [], []
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                outs.append(layer(Xs, residual=None))
            graphs.append(gr)
        X2 = _bf(_randn(g, T, K))
        Xs.copy_(X2)
        for gr in graphs:
            gr.replay()
        want2 = layer(X2)
        assert torch.equal(outs[0], want2) and torch.equal(outs[1], want2)
    assert hq.hq_check_device_error() == 0


# -------------------------------------------------------------- hq_linear_ep
def _codes(g, rows, K, bits):
    q = 2 ** (bits - 1) - 1
    return torch.randint(-q, q + 1, (rows, K), generator=g, device="cuda").to(torch.int8)


def _linear_case(hq, T, K, N, a_bits, w_bits, act, per_token=True, mean=True, packed=False,
                 out_order=0, residual=False, rows=0, bias=True, acc=False, seed=0):
    g = _gen(seed + T + 3 * K + 5 * N)
    A, Wc = _codes(g, T, K, a_bits), _codes(g, N, K, w_bits)
    sx = torch.rand(T if per_token else 1, generator=g, device="cuda") + 0.5
    sw = (torch.rand(N, generator=g, device="cuda") + 0.5) / (2 ** (a_bits + w_bits - 2) * K ** 0.5)
    m = _randn(g, T) if mean else None
    cs = _randn(g, N)
    b = _randn(g, N) if bias else None
    R = _bf(_randn(g, T, N)) if residual else None
    G = _bf(_randn(g, -(-T // rows), N)) if rows else None
    wh = out_order > 1
    desc = hq.LayerDesc(K, N, 1 if wh else 16, a_bits=a_bits, w_bits=w_bits,
                        act_gran=hq.HQ_PER_TOKEN if per_token else hq.HQ_PER_TENSOR_DYNAMIC,
                        centering=hq.HQ_CENTER_TOKEN_MEAN if mean else hq.HQ_CENTER_NONE,
                        code_format=hq.HQ_CODES_I4_PACKED if packed else hq.HQ_CODES_I8,
                        out_order=out_order)
    Y, check = _guarded(T, N)
    dbg = torch.empty(T, N, dtype=torch.int32, device="cuda") if acc else None
    hq.hq_linear_ep(desc, pack_i4(A) if packed else A, sx, m, Wc, sw, cs if not wh else None, b,
                    hq.Epilogue(act, R, G, rows), Y, dbg)
    assert hq.hq_check_device_error() == 0
    if acc:
        assert torch.equal(dbg.double(), A.double() @ Wc.double().t())
    z, ztol = linear64(A, sx if per_token else sx.expand(T), m, Wc, sw, cs, b, out_order)
    y, tol = epilogue64(z, ztol, act, R, G, rows)
    check_rounded(Y, y, tol, f"linear {T}x{K}x{N} A{a_bits}W{w_bits}")
    if T * N > 4000:
        assert rel_frob(Y, y) < ROUND_FROB
    check()


LINEAR_SHAPES = [(1, 16, 16), (1, 1152, 3456), (2, 4608, 1152), (5, 80, 48), (17, 1040, 272),
                 (40, 320, 320), (64, 1152, 1168), (100, 2048, 336), (129, 144, 640),
                 (300, 1024, 1024), (1025, 2560, 512), (2000, 320, 320), (9, 16, 16),
                 (12, 8192, 128), (30, 1040, 3456), (90, 4608, 272), (250, 208, 144),
                 (4100, 640, 1152), (600, 8192, 1536)]


@pytest.mark.parametrize("T,K,N", LINEAR_SHAPES)
@pytest.mark.parametrize("form", range(4))
def test_linear_ep(hq, T, K, N, form):
    kw = [dict(a_bits=4, w_bits=4, act=GELU_TANH, residual=True, rows=max(1, T // 2)),
          dict(a_bits=8, w_bits=8, act=SILU, per_token=False, mean=False, residual=True),
          dict(a_bits=3, w_bits=4, act=NONE, rows=1, residual=True, bias=False),
          dict(a_bits=4, w_bits=8, act=GELU, acc=True)][form]
    _linear_case(hq, T, K, N, **kw)


@pytest.mark.parametrize("T,K,N", [(1, 32, 16), (1, 1152, 3456), (7, 1056, 272), (200, 320, 336),
                                   (1025, 2560, 512), (12, 64, 32), (3000, 1152, 1152)])
@pytest.mark.parametrize("a_bits", [3, 4])
def test_linear_ep_packed(hq, T, K, N, a_bits):
    _linear_case(hq, T, K, N, a_bits, 4, SILU, packed=True, residual=True, rows=max(1, T - 1))
    _linear_case(hq, T, K, N, a_bits, 8, NONE, packed=True, mean=False, residual=True, acc=True)


@pytest.mark.parametrize("m", [16, 32, 64])
@pytest.mark.parametrize("T,K,N", [(1, 64, 64), (9, 1152, 1152), (300, 320, 320), (1000, 2048, 576)])
def test_linear_ep_weight_only(hq, T, K, N, m):
    _linear_case(hq, T, K, N, 4, 4, GELU, mean=False, out_order=m, residual=True, rows=max(1, T // 4))
    _linear_case(hq, T, K, N, 4, 4, SILU, mean=False, out_order=m, packed=True, bias=False)


def test_linear_ep_extreme_codes(hq):
    """Every code at the end of its range: the largest sums."""
    for T, K in ((3, 15360), (200, 10240)):
        N = 128
        A = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
        W = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        W[1::2] = 127
        sx = torch.full((T,), 2.0 ** -20, device="cuda")
        sw = torch.full((N,), 1.0, device="cuda")
        Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        desc = hq.LayerDesc(K, N, 16, a_bits=8, w_bits=8, centering=hq.HQ_CENTER_NONE)
        hq.hq_linear_ep(desc, A, sx, None, W, sw, None, None, hq.Epilogue(RELU), Y)
        z = A.double() @ W.double().t() * 2.0 ** -20
        assert torch.equal(Y, z.clamp(min=0).float().bfloat16())


def test_linear_ep_plain_equals_linear(hq):
    """Without activation, gate and residual the call is hq_linear, bit for bit."""
    K, N = 1152, 1152
    for T in (1, 6, 40, 300, 3000):
        g = _gen(T)
        A, W = _codes(g, T, K, 4), _codes(g, N, K, 4)
        sx, sw, b, m, cs = (_randn(g, n).abs() for n in (T, N, N, T, N))
        desc = hq.LayerDesc(K, N, 128)
        Y = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        hq.hq_linear(desc, A, sx, m, W, sw, cs, b, Y[0])
        hq.hq_linear_ep(desc, A, sx, m, W, sw, cs, b, None, Y[1])
        hq.hq_linear_ep(desc, A, sx, m, W, sw, cs, b, hq.Epilogue(), Y[2])
        assert torch.equal(Y[0], Y[1]) and torch.equal(Y[0], Y[2])


def test_layer_with_epilogue_in_a_graph(hq):
    """quantize + product with epilogue, captured and replayed on new inputs."""
    T, K, N = 260, 512, 512
    g = _gen(2)
    W, b = _bf(_randn(g, N, K) * 0.05), _bf(_randn(g, N))
    layer = hq.HadamardQuantLinear(hq.LayerDesc(K, N, 128), W, b)
    X = _bf(_randn(g, T, K))
    Xs = X.clone()
    ep = hq.Epilogue(GELU, Xs)
    out = layer.forward(Xs, epilogue=ep)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = layer.forward(Xs, epilogue=ep)
    X2 = _bf(_randn(g, T, K))
    Xs.copy_(X2)
    gr.replay()
    got = out.clone()
    want = layer.forward(X2, epilogue=hq.Epilogue(GELU, X2))
    assert torch.equal(got, want)


# ------------------------------------------------------------- hq_group_norm
GN_SHAPES = [  # B, S, C, G
    (1, 1, 8, 1), (1, 1, 7, 7), (2, 1, 6, 3), (1, 2, 2, 1), (3, 5, 10, 5), (2, 33, 320, 32),
    (1, 4096, 320, 32), (4, 1024, 320, 32), (1, 65, 1280, 32), (2, 257, 182, 26), (3, 1000, 77, 11),
    (1, 513, 12, 1), (2, 100, 2560, 32), (1, 31, 8192, 32), (1, 3, 8190, 7), (5, 64, 96, 96),
    (1, 20000, 128, 32), (1, 9000, 64, 1), (300, 16, 64, 8), (1, 7001, 30, 3), (70000, 1, 16, 2),
    (1, 5000, 36, 9), (16, 4096, 320, 32),
    # prime numbers of groups (passes that overlap), one channel a group, wide rows
    (1, 64, 8191, 8191), (2, 40, 1021, 1021), (1, 300, 5160, 1290), (2, 17, 6186, 1031),
    (3, 9, 8184, 8184), (1, 50, 4104, 8), (1, 12, 8192, 1), (1, 700, 8191, 1), (149, 2, 40, 4),
    (5, 1031, 8, 8),
]


@pytest.mark.parametrize("B,S,C,G", GN_SHAPES)
def test_group_norm(hq, B, S, C, G):
    g = _gen(B + S + C + G)
    X = _bf(_randn(g, B, S, C) * torch.exp(0.5 * _randn(g, 1, 1, C)) + _randn(g, B, 1, C))
    ga, be = _bf(1 + 0.3 * _randn(g, C)), _bf(0.5 * _randn(g, C))
    for act, a, b in ((NONE, ga, be), ((SILU, GELU, GELU_TANH, RELU)[(S + C) % 4], ga, be),
                      (SILU, None, None)):
        buf = torch.full((X.numel() + 16,), 77.0, dtype=torch.bfloat16, device="cuda")
        Y = buf[8:8 + X.numel()].view(X.shape)
        d = hq.GroupNormDesc(C, G, act, 1e-5)
        nb = hq.hq_group_norm_workspace_bytes(d, B, S)
        ws = torch.full((nb,), 0x7F, dtype=torch.uint8, device="cuda") if nb else None
        hq.hq_group_norm(d, X, a, b, Y, ws)
        assert hq.hq_check_device_error() == 0
        y, tol = group_norm64(X, G, a, b, 1e-5, act)
        check_rounded(Y, y, tol, f"group norm {B}x{S}x{C} G{G} act {act}")
        if act == NONE and X.numel() > 4000 and S * C // G > 16:
            assert rel_frob(Y, y) < ROUND_FROB
        assert bool((buf[:8] == 77.0).all()) and bool((buf[8 + X.numel():] == 77.0).all())


@pytest.mark.parametrize("B,S,C,G", [(1, 4096, 320, 32), (2, 3000, 66, 6), (1, 40, 128, 32),
                                     (1, 60000, 128, 32)])
def test_group_norm_offset_and_outliers(hq, B, S, C, G):
    """Means far from zero next to the spread, and single values far out, also
    where a thread starts: no cancellation in the variance."""
    g = _gen(5)
    base = _randn(g, B, S, C)
    X1 = _bf(base + 100.0)                      # spread of two bf16 steps
    X2 = base.clone()
    X2[:, 0] = 3000.0                           # every thread's first row is an outlier
    X2 = _bf(X2)
    X3 = base.clone()
    X3[:, S // 2, 0] = -20000.0
    X3 = _bf(X3)
    norm = hq.GroupNorm(C, G)
    for X in (X1, X2, X3):
        Y = norm(X)
        x = X.double().view(B, S, G, -1)
        var, mean = torch.var_mean(x, dim=(1, 3), correction=0, keepdim=True)
        y = ((x - mean) / torch.sqrt(var + 1e-5)).view(X.shape)
        # a variance off by 1 % would show as half a percent
        assert rel_frob(Y, y) < ROUND_FROB
    const = torch.full((B, S, C), 5.0, dtype=torch.bfloat16, device="cuda")
    assert bool((norm(const) == 0).all())       # variance 0: exactly the mean


def test_group_norm_nonfinite_stays_in_its_group(hq):
    for C, G in ((64, 8), (72, 8), (63, 9), (40, 8)):  # groups of 8, 9, 7 and 5 channels
        B, S = 2, 300
        cpg = C // G
        X = _bf(_randn(_gen(1), B, S, C))
        X[0, 17, 3] = float("nan")
        X[1, 200, 2 * cpg + 4] = float("inf")
        for act in (SILU, GELU, GELU_TANH, RELU, NONE):
            Y = hq.GroupNorm(C, G, act=act)(X)
            bad = Y.isnan().view(B, S, G, -1).any(dim=3).any(dim=1)
            want = torch.zeros(B, G, dtype=torch.bool, device="cuda")
            want[0, 0] = want[1, 2] = True
            assert torch.equal(bad, want)
            assert bool(Y.view(B, S, G, -1)[0, :, 0].isnan().all())


@pytest.mark.parametrize("B,S,C,G", [(2, 4096, 320, 32), (1, 1000, 77, 11), (1, 30000, 128, 32)])
def test_group_norm_in_place_streams_and_graphs(hq, B, S, C, G):
    g = _gen(6)
    X = _bf(_randn(g, B, S, C))
    norm = hq.GroupNorm(C, G, _bf(_randn(g, C)), _bf(_randn(g, C)), act=SILU)
    want = norm(X)
    Z = X.clone()
    norm(Z, Z)
    assert torch.equal(Z, want)
    s = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in s:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs += [norm(X) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    Xs = X.clone()
    norm(Xs)
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(norm(Xs))
        graphs.append(gr)
    X2 = _bf(_randn(g, B, S, C))
    Xs.copy_(X2)
    for gr in graphs:
        gr.replay()
    want2 = norm(X2)
    assert torch.equal(outs[0], want2) and torch.equal(outs[1], want2)
    assert hq.hq_check_device_error() == 0


def test_group_norm_empty(hq):
    norm = hq.GroupNorm(64, 8)
    for shape in ((0, 5, 64), (3, 0, 64)):
        X = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        assert norm(X).shape == X.shape


# ------------------------------------------------------------- used together
@pytest.mark.parametrize("per_tensor", [False, True])
def test_pointwise_block(hq, per_tensor):
    """group norm -> quantizer -> 1x1 convolution with the block's input added,
    against the 64-bit forms fed with the codes the quantizer left."""
    B, H, Wd, C, G = 2, 20, 25, 320, 32
    g = _gen(8)
    X = _bf(_randn(g, B, H, Wd, C))
    W, b = _bf(_randn(g, C, C) * C ** -0.5), _bf(0.1 * _randn(g, C))
    ga, be = _bf(1 + 0.2 * _randn(g, C)), _bf(0.2 * _randn(g, C))
    desc = hq.LayerDesc(C, C, 64, a_bits=8, w_bits=8, centering=hq.HQ_CENTER_NONE,
                        act_gran=hq.HQ_PER_TENSOR_DYNAMIC if per_tensor else hq.HQ_PER_TOKEN)
    layer = hq.HadamardQuantLinear(desc, W, b)
    norm = hq.GroupNorm(C, G, ga, be, act=SILU)
    Y = hq.PointwiseBlock(norm, layer, residual=True)(X)
    assert Y.shape == X.shape and hq.hq_check_device_error() == 0
    h = norm(X)
    y, tol = group_norm64(X.view(B, -1, C), G, ga, be, 1e-5, SILU)
    check_rounded(h.view(B, -1, C), y, tol, "norm")
    T = B * H * Wd
    bufs = layer.quantize(h.view(T, C))
    sx = bufs["a_scale"] if not per_tensor else bufs["a_scale"].expand(T)
    z, ztol = linear64(bufs["a_codes"], sx, None, layer.w_codes, layer.w_scale, layer.colsum,
                       layer.bias_f32)
    y, tol = epilogue64(z, ztol, NONE, X.view(T, C))
    check_rounded(Y.view(T, C), y, tol, "block")
    # and near the block in full precision (8-bit codes)
    full = X.view(T, C).double() + h.view(T, C).double() @ W.double().t() + b.double()
    assert rel_frob(Y.view(T, C), full) < 0.02


def test_modulated_mlp(hq):
    """A transformer MLP: modulation rows by hq_dense, fc1 with GELU and fc2
    with gate and residual on 8-bit codes."""
    B, S, D, M = 3, 210, 256, 1024
    g = _gen(10)
    X, temb = _bf(_randn(g, B * S, D)), _bf(_randn(g, B, D))
    W1, b1 = _bf(_randn(g, M, D) * D ** -0.5), _bf(0.1 * _randn(g, M))
    W2, b2 = _bf(_randn(g, D, M) * M ** -0.5), _bf(0.1 * _randn(g, D))
    Wm, bm = _bf(_randn(g, D, D) * D ** -0.5), _bf(0.1 * _randn(g, D))
    kw = dict(a_bits=8, w_bits=8)
    fc1 = hq.HadamardQuantLinear(hq.LayerDesc(D, M, 128, **kw), W1, b1)
    fc2 = hq.HadamardQuantLinear(hq.LayerDesc(M, D, 128, **kw), W2, b2)
    gate = hq.DenseLinear(Wm, bm)(temb)
    h = fc1.forward(X, epilogue=hq.Epilogue(GELU_TANH))
    Y = fc2.forward(h, epilogue=hq.Epilogue(residual=X, gate=gate, gate_rows=S))
    assert hq.hq_check_device_error() == 0
    gd = temb.double() @ Wm.double().t() + bm.double()
    hd = epilogue64(X.double() @ W1.double().t() + b1.double(), torch.zeros((), device="cuda"),
                    GELU_TANH)[0]
    yd = X.double() + gd.repeat_interleave(S, 0) * (hd @ W2.double().t() + b2.double())
    assert rel_frob(Y, yd) < 0.02


# ------------------------------------------------- tensors past 2^31 elements
def _windows(T, at, n=300):
    """Row ranges: the first, those around `at` and the last."""
    return [slice(0, n), slice(at - n // 2, at + n // 2), slice(T - n, T)]


def test_dense_past_31_bits(hq):
    g = _gen(41)
    T, K, N = (1 << 20) + 5, 8, 2056
    assert T * N > 2 ** 31
    X, W = _bf(_randn(g, T, K)), _bf(_randn(g, N, K) * K ** -0.5)
    G = _bf(_randn(g, -(-T // 1000), N))
    Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    wins = _windows(T, 2 ** 31 // N)
    R = [Y[w].clone() for w in wins]
    hq.hq_dense(hq.DenseDesc(K, N), X, W, None, hq.Epilogue(SILU, Y, G, 1000), Y)
    assert hq.hq_check_device_error() == 0
    for w, r in zip(wins, R):
        z, ztol = dense64(X[w], W, None)
        rows = torch.arange(w.start, w.stop, device="cuda") // 1000
        y, tol = epilogue64(z, ztol, SILU, r, G[rows], 1)
        check_rounded(Y[w], y, tol, f"rows {w}")


def test_linear_ep_past_31_bits(hq):
    g = _gen(42)
    T, K, N = (1 << 20) + 5, 16, 2064
    assert T * N > 2 ** 31
    A, W = _codes(g, T, K, 4), _codes(g, N, K, 4)
    sx = torch.rand(T, generator=g, device="cuda") + 0.5
    sw = (torch.rand(N, generator=g, device="cuda") + 0.5) / 256
    Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    wins = _windows(T, 2 ** 31 // N)
    R = [Y[w].clone() for w in wins]
    desc = hq.LayerDesc(K, N, 16, a_bits=4, w_bits=4, centering=hq.HQ_CENTER_NONE)
    hq.hq_linear_ep(desc, A, sx, None, W, sw, None, None, hq.Epilogue(GELU_TANH, Y), Y)
    assert hq.hq_check_device_error() == 0
    for w, r in zip(wins, R):
        z, ztol = linear64(A[w], sx[w], None, W, sw, None, None)
        y, tol = epilogue64(z, ztol, GELU_TANH, r)
        check_rounded(Y[w], y, tol, f"rows {w}")


@pytest.mark.parametrize("B,S,C,G", [(1, (1 << 25) + 3, 72, 8), (3, (1 << 23) + 1, 96, 8)])
def test_group_norm_past_31_bits(hq, B, S, C, G):
    assert B * S * C > 2 ** 31
    g = _gen(43)
    X = torch.empty(B, S, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    X[:, S // 2:] += 2                     # the halves differ: a part that is missed shows
    ga, be = _bf(1 + 0.3 * _randn(g, C)), _bf(0.5 * _randn(g, C))
    Y = hq.GroupNorm(C, G, ga, be, act=SILU)(X)
    assert hq.hq_check_device_error() == 0
    for b in range(B):
        chunks = X[b].split(1 << 21)
        n = S * (C // G)
        mean = sum(c.double().view(-1, G, C // G).sum(dim=(0, 2)) for c in chunks) / n
        m = mean.repeat_interleave(C // G)
        var = sum(((c.double() - m) ** 2).view(-1, G, C // G).sum(dim=(0, 2)) for c in chunks) / n
        rstd = (1 / torch.sqrt(var + 1e-5)).repeat_interleave(C // G)
        for w in _windows(S, min(2 ** 31 // C, S // 2)):
            z = (X[b, w].double() - m) * rstd * ga.double() + be.double()
            assert rel_frob(Y[b, w], z / (1 + torch.exp(-z))) < ROUND_FROB


# small tensors: slices of whole groups held by clusters of one to eight blocks,
# the last chunk of rows shorter, sizes on both sides of what they can hold
@pytest.mark.parametrize("B,S,C,G", [
    (1, 4095, 320, 32), (1, 127, 64, 8), (1, 128, 64, 8), (1, 257, 1280, 32), (4, 1023, 320, 32),
    (2, 4096, 320, 32), (30, 255, 320, 32), (148, 3, 16, 2), (149, 3, 16, 2), (1, 4096, 36, 9),
    (1, 4097, 640, 32), (2, 1000, 100, 5), (1, 513, 512, 512), (7, 65, 24, 1), (1, 3277, 320, 32),
    (1, 6553, 320, 32), (1, 2049, 1280, 32)])
def test_group_norm_small(hq, B, S, C, G):
    g = _gen(B + S + C + G)
    X = _bf(_randn(g, B, S, C) * torch.exp(0.5 * _randn(g, 1, 1, C)) + _randn(g, B, 1, C))
    ga, be = _bf(1 + 0.3 * _randn(g, C)), _bf(0.5 * _randn(g, C))
    norm = hq.GroupNorm(C, G, ga, be, act=SILU)
    Y = norm(X)
    y, tol = group_norm64(X, G, ga, be, 1e-5, SILU)
    check_rounded(Y, y, tol, f"group norm {B}x{S}x{C} G{G}")
    assert rel_frob(Y, y) < ROUND_FROB
    Z = X.clone()
    norm(Z, Z)                              # in place
    assert torch.equal(Z, Y)
    poisoned = X.clone()                    # an infinity stays in its image and group
    poisoned[0, S // 2, 0] = float("inf")
    P = norm(poisoned)
    n = C // G
    assert bool(P[0, :, :n].isnan().all())
    assert torch.equal(P[0, :, n:], Y[0, :, n:]) and torch.equal(P[1:], Y[1:])
    assert hq.hq_check_device_error() == 0
