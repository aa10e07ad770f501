"""GPU tests of every kernel behind hq_dense and hq_linear_ep, each set by
hq_debug_set_product_plan, so that none depends on the sizes at which it is
chosen: partial tiles on every side, several tiles a CTA, one to many K blocks,
gates that cross rows, residuals in place.  Needs a B200."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from ops_ref import (GELU, GELU_TANH, NONE, RELU, SILU, check_rounded, dense64,  # noqa: E402
                     epilogue64, linear64, pack_i4)

pytestmark = pytest.mark.gpu

ROWS, SPLIT, TILES, PAIR = 1, 2, 3, 4
SPLITS = [(SPLIT, nt, k) for nt in (16, 32, 64, 128) for k in (1, 2, 4, 8)]
TILED = [(TILES, w, 1) for w in (64, 128, 192, 256)]
PAIRS = [(PAIR, w, 1) for w in (128, 192, 256)]


@pytest.fixture(scope="module")
def hq():
    import hadamard_rotated_bit_token_b200 as hq_mod
    from hadamard_rotated_bit_token_b200 import build as hq_build
    hq_build.build()
    hq_mod.load_library()
    return hq_mod


@contextlib.contextmanager
def _plan(hq, plan):
    hq.hq_debug_set_product_plan(hq.ProductPlan(*plan))
    try:
        yield
    finally:
        hq.hq_debug_set_product_plan(None)


def _id(plan):
    return "-".join((("", "rows", "split", "tiles", "pair")[plan[0]],) + tuple(map(str, plan[1:])))


def _gen(*seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(s * p for s, p in zip(seed, (1, 31, 977, 7919, 104729))))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _bf(t):
    return t.to(torch.bfloat16)


def _guarded(T, N, fill=None):
    """Y [T, N] (a copy of `fill`, or poison) between rows of poison: (Y, check)."""
    buf = torch.full((T + 16, N), 123.0, dtype=torch.bfloat16, device="cuda")
    Y = buf[8:T + 8]           # 8 rows of a multiple of 8 columns: 16-byte aligned
    if fill is not None:
        Y.copy_(fill)

    def check():
        assert bool((buf[:8] == 123.0).all()) and bool((buf[T + 8:] == 123.0).all()), \
            "rows outside Y were written"
    return Y, check


def _epilogues(hq, g, T, N):
    """(act, residual, gate, gate_rows): every part alone and all together, gate
    rows shorter and longer than tiles and one for all."""
    R = _bf(_randn(g, T, N))
    gate = lambda rows: _bf(_randn(g, -(-T // rows), N))
    few = max(1, T // 3)
    return [(NONE, None, None, 0), (SILU, None, None, 0), (RELU, R, None, 0),
            (NONE, None, gate(37), 37), (GELU, R, gate(few), few),
            (GELU_TANH, R, gate(10 ** 9), 10 ** 9), (NONE, R, gate(1), 1)]


def _run_both(hq, call, T, N, act, R, G, rows):
    """The call into a poisoned Y and, with a residual, once more in place: the
    same bits both times, and nothing outside Y."""
    Y, check = _guarded(T, N)
    call(hq.Epilogue(act, R, G, rows), Y)
    check()
    if R is not None:
        Z, check = _guarded(T, N, R)
        call(hq.Epilogue(act, Z, G, rows), Z)
        check()
        assert torch.equal(Y, Z), "in place differs"
    assert hq.hq_check_device_error() == 0
    return Y


def _dense(hq, plan, T, K, N):
    g = _gen(T, K, N, *plan[:2])
    d = hq.DenseDesc(K, N)
    with _plan(hq, plan):
        chosen = tuple(hq.hq_debug_dense_plan(d, T))
        assert chosen == plan if plan[0] != ROWS else chosen[0] == ROWS
        # integers whose sums fp32 holds exactly: a wrong, missing or doubled product shows
        X, W, R = (_bf(torch.randint(-3, 4, s, generator=g, device="cuda").float())
                   for s in ((T, K), (N, K), (T, N)))
        b = _bf(torch.randint(-8, 9, (N,), generator=g, device="cuda").float())
        want = (X.double() @ W.double().t() + b.double() + R.double()).float().bfloat16()
        call = lambda ep, Y: hq.hq_dense(d, X, W, b, ep, Y)
        assert torch.equal(_run_both(hq, call, T, N, NONE, R, None, 0), want)
        X, W = _bf(_randn(g, T, K)), _bf(_randn(g, N, K) * K ** -0.5)
        for i, (act, R, G, rows) in enumerate(_epilogues(hq, g, T, N)):
            b = _bf(_randn(g, N)) if i % 2 else None
            call = lambda ep, Y: hq.hq_dense(d, X, W, b, ep, Y)
            Y = _run_both(hq, call, T, N, act, R, G, rows)
            z, ztol = dense64(X, W, b)
            y, tol = epilogue64(z, ztol, act, R, G, rows)
            check_rounded(Y, y, tol, f"dense {T}x{K}x{N} epilogue {i}")
    return chosen


def _linear(hq, plan, T, K, N, packed=False, m=0, acc=False):
    g = _gen(T, K, N, *plan[:2])
    code = lambda rows, bits: torch.randint(-2 ** (bits - 1), 2 ** (bits - 1), (rows, K),
                                            generator=g, device="cuda").to(torch.int8)
    for bits in ((4, 4), (8, 8)):
        if packed and bits[0] > 4:
            bits = (3, 8)
        A, Wc = code(T, bits[0]), code(N, bits[1])
        a = pack_i4(A) if packed else A
        per_token = bits[1] == 4
        sx = torch.rand(T if per_token else 1, generator=g, device="cuda") + 0.5
        sw = (torch.rand(N, generator=g, device="cuda") + 0.5) / (
            2 ** (sum(bits) - 2) * K ** 0.5)
        mean = _randn(g, T) if per_token and not m else None
        cs, b = _randn(g, N) if not m else None, _randn(g, N)
        desc = hq.LayerDesc(K, N, 1 if m else 16, a_bits=bits[0], w_bits=bits[1],
                            act_gran=hq.HQ_PER_TOKEN if per_token else hq.HQ_PER_TENSOR_DYNAMIC,
                            centering=hq.HQ_CENTER_TOKEN_MEAN if mean is not None
                            else hq.HQ_CENTER_NONE,
                            code_format=hq.HQ_CODES_I4_PACKED if packed else hq.HQ_CODES_I8,
                            out_order=m)
        plain = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        hq.hq_linear(desc, a, sx, mean, Wc, sw, cs, b, plain)
        dbg = torch.empty(T, N, dtype=torch.int32, device="cuda") if acc else None
        with _plan(hq, plan):
            chosen = tuple(hq.hq_debug_linear_ep_plan(desc, T))
            assert chosen == plan if plan[0] != ROWS else chosen[0] == ROWS
            for i, (act, R, G, rows) in enumerate(_epilogues(hq, g, T, N)):
                call = lambda ep, Y: hq.hq_linear_ep(desc, a, sx, mean, Wc, sw, cs, b, ep, Y, dbg)
                Y = _run_both(hq, call, T, N, act, R, G, rows)
                if i == 0:  # sums are exact and the epilogue is the same arithmetic
                    assert torch.equal(Y, plain), "not hq_linear's result"
                if acc:
                    assert torch.equal(dbg.double(), A.double() @ Wc.double().t())
                z, ztol = linear64(A, sx if per_token else sx.expand(T), mean, Wc, sw, cs, b, m)
                y, tol = epilogue64(z, ztol, act, R, G, rows)
                check_rounded(Y, y, tol, f"linear {T}x{K}x{N} {bits} epilogue {i}")
    return chosen


# tiles: one corner of a tile, partial tiles with 19 K blocks, and more tiles
# than CTAs (or pairs) with partial ones at both ends
@pytest.mark.parametrize("plan", TILED + PAIRS, ids=_id)
@pytest.mark.parametrize("T,K,N", [(1, 8, 8), (131, 1160, 264), (300, 2056, 72), (5117, 200, 1160),
                                   (2100, 64, 2824)])
def test_dense_tiles(hq, plan, T, K, N):
    _dense(hq, plan, T, K, N)


@pytest.mark.parametrize("plan", TILED + PAIRS, ids=_id)
@pytest.mark.parametrize("T,K,N", [(1, 16, 16), (131, 2320, 272), (300, 1040, 80),
                                   (5117, 400, 1168), (2100, 144, 2832)])
def test_linear_tiles(hq, plan, T, K, N):
    _linear(hq, plan, T, K, N, acc=T < 200)


@pytest.mark.parametrize("plan", TILED[:3], ids=_id)
@pytest.mark.parametrize("T,K,N", [(1, 32, 16), (131, 2336, 272), (5117, 416, 1168)])
def test_linear_packed_tiles(hq, plan, T, K, N):
    _linear(hq, plan, T, K, N, packed=True, acc=T < 200)


@pytest.mark.parametrize("plan,packed", [(p, False) for p in TILED] + [(p, True) for p in TILED[:3]],
                         ids=lambda v: _id(v) if isinstance(v, tuple) else ("packed" if v else "i8"))
@pytest.mark.parametrize("m", [16, 32, 64])
@pytest.mark.parametrize("T,K,N", [(1, 32, 64), (131, 1184, 320), (5117, 160, 1216)])
def test_linear_weight_only_tiles(hq, plan, packed, m, T, K, N):
    _linear(hq, plan, T, K, N, packed=packed, m=m)


# K split: fewer tokens than a tile, one more than one, several; as many K blocks
# as CTAs (the last one partial), numbers that do not divide, rings that wrap
@pytest.mark.parametrize("plan", SPLITS, ids=_id)
def test_dense_split(hq, plan):
    _, nt, k = plan
    blocks = lambda n: n * 64 - 24           # n K blocks of 128 bytes, the last partial
    for T, K, N in ((1, blocks(k), 8), (nt - 1, blocks(2 * k + 1), 136),
                    (nt + 1, blocks(37), 264), (2 * nt + 3, blocks(90), 72)):
        _dense(hq, plan, T, K, N)


@pytest.mark.parametrize("plan", SPLITS, ids=_id)
def test_linear_split(hq, plan):
    _, nt, k = plan
    blocks = lambda n: n * 128 - 48
    for T, K, N in ((1, blocks(k), 16), (nt - 1, blocks(2 * k + 1), 144),
                    (nt + 1, blocks(37), 272), (2 * nt + 3, blocks(90), 80)):
        _linear(hq, plan, T, K, N)


# one pass over the weights: K shared by one, two and four warps, steps left over
ROWS_KN = [(8, 8), (520, 264), (1000, 9480), (1096, 5000), (632, 72), (3704, 40)]
ROWS_I8 = [(16, 16), (1040, 272), (2000, 9488), (4112, 2400), (1264, 80), (7424, 48)]
ROWS_T = [1, 2, 3, 4, 5, 7, 8]


def test_dense_rows(hq):
    seen = {_dense(hq, (ROWS, 1, 1), T, K, N) for T in ROWS_T for K, N in ROWS_KN}
    assert seen == {(ROWS, t, w) for t in (1, 2, 4, 8) for w in (1, 2, 4)}


@pytest.mark.parametrize("packed", [False, True])
def test_linear_rows(hq, packed):
    shapes = [(-(-K // 32) * 32, N) if packed else (K, N) for K, N in ROWS_I8]
    seen = {_linear(hq, (ROWS, 1, 1), T, K, N, packed=packed) for T in ROWS_T for K, N in shapes}
    assert seen == {(ROWS, t, w) for t in (1, 2, 4, 8) for w in (1, 2, 4)}
