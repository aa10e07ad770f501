"""The kernels that hq_dense and hq_linear_ep choose (hq_debug_dense_plan,
hq_debug_linear_ep_plan: host logic, no GPU) on a 148-SM B200 that holds 74
CTA-pair clusters: every kernel that is built is chosen at some size, and a plan
that is set is taken or refused."""
import itertools

import pytest

ROWS, SPLIT, TILES, PAIR, LINEAR = 1, 2, 3, 4, 5
OK, INVALID, UNSUPPORTED = 0, 1, 2

# kind -> plan (kernel, width, split) -> a size (T, K, N, act) at which it is chosen
CHOSEN = {
    "bf16": {
        (1, 1, 1): (1, 8, 8, 0), (1, 1, 2): (1, 632, 8, 0), (1, 1, 4): (1, 1072, 8, 4),
        (1, 2, 1): (2, 8, 8, 0), (1, 2, 2): (2, 512, 8, 4), (1, 2, 4): (2, 1136, 8, 0),
        (1, 4, 1): (3, 8, 8, 4), (1, 4, 2): (3, 528, 8, 0), (1, 4, 4): (3, 1200, 8, 0),
        (1, 8, 1): (5, 8, 8, 0), (1, 8, 2): (5, 704, 8, 4), (1, 8, 4): (5, 1048, 8, 0),
        (2, 16, 1): (16, 8, 19488, 0), (2, 16, 2): (1016, 272, 8, 4), (2, 16, 4): (11, 200, 8, 0),
        (2, 16, 8): (9, 512, 8, 0), (2, 32, 1): (19, 16, 30432, 4), (2, 32, 2): (2046, 1040, 8, 4),
        (2, 32, 4): (904, 664, 8, 0), (2, 32, 8): (424, 1600, 8, 4),
        (2, 64, 1): (37, 4176, 15680, 4), (2, 64, 2): (3986, 2648, 8, 0),
        (2, 64, 4): (1807, 1304, 8, 4), (2, 64, 8): (1043, 2472, 8, 4),
        (2, 128, 1): (72, 7392, 17960, 4), (2, 128, 2): (6340, 5088, 8, 0),
        (2, 128, 4): (3503, 3856, 8, 0), (2, 128, 8): (1843, 9728, 8, 4),
        (3, 64, 1): (15, 8, 8, 0), (3, 128, 1): (9, 8, 9768, 4), (3, 192, 1): (9, 8, 20648, 4),
        (3, 256, 1): (29, 8, 32560, 0), (4, 128, 1): (10188, 4416, 80, 0),
        (4, 192, 1): (150, 1728, 10600, 4), (4, 256, 1): (9807, 1032, 256, 0)},
    "i8": {
        (1, 1, 1): (1, 16, 16, 0), (1, 1, 2): (1, 1088, 16, 4), (1, 1, 4): (1, 2272, 16, 0),
        (1, 2, 1): (2, 16, 16, 0), (1, 2, 2): (2, 1360, 16, 4), (1, 2, 4): (2, 2064, 16, 0),
        (1, 4, 1): (3, 16, 16, 4), (1, 4, 2): (3, 1040, 16, 0), (1, 4, 4): (3, 2112, 16, 0),
        (1, 8, 1): (5, 16, 16, 0), (1, 8, 2): (6, 1136, 16, 4), (1, 8, 4): (6, 2112, 16, 0),
        (2, 16, 1): (10, 16, 20480, 4), (2, 16, 2): (934, 560, 16, 0),
        (2, 16, 4): (10, 448, 16, 0), (2, 16, 8): (10, 928, 16, 4), (2, 32, 1): (27, 16, 30080, 4),
        (2, 32, 2): (2354, 2096, 16, 0), (2, 32, 4): (985, 1360, 16, 0),
        (2, 32, 8): (468, 2784, 16, 0), (2, 64, 1): (37, 6864, 19536, 0),
        (2, 64, 2): (4502, 4816, 16, 4), (2, 64, 4): (2350, 2224, 16, 4),
        (2, 64, 8): (996, 5504, 16, 0), (2, 128, 1): (71, 13712, 17360, 0),
        (2, 128, 2): (6493, 10496, 16, 0), (2, 128, 4): (3484, 11520, 16, 0),
        (2, 128, 8): (1890, 10688, 32, 0), (3, 64, 1): (9, 16, 16, 0),
        (3, 128, 1): (10, 16, 11024, 0), (3, 192, 1): (11, 16, 23760, 4),
        (3, 256, 1): (17, 32, 32288, 4), (4, 128, 1): (11443, 9008, 80, 4),
        (4, 192, 1): (132, 3792, 9840, 0), (4, 256, 1): (146, 2096, 18752, 0)},
    "pk": {
        (1, 1, 1): (1, 32, 16, 4), (1, 1, 2): (1, 1024, 16, 4), (1, 1, 4): (1, 2240, 16, 4),
        (1, 2, 1): (2, 32, 16, 4), (1, 2, 2): (2, 1056, 16, 0), (1, 2, 4): (2, 2080, 16, 4),
        (1, 4, 1): (3, 32, 16, 4), (1, 4, 2): (3, 1184, 16, 4), (1, 4, 4): (3, 2304, 16, 4),
        (1, 8, 1): (5, 32, 16, 0), (1, 8, 2): (5, 1312, 16, 0), (1, 8, 4): (5, 2144, 16, 0),
        (3, 64, 1): (9, 32, 16, 0), (3, 128, 1): (9, 32, 10320, 4), (3, 192, 1): (9, 32, 21056, 0)},
    "w16": {
        (3, 64, 1): (1, 16, 16, 4), (3, 128, 1): (1, 16, 9648, 0), (3, 192, 1): (1, 16, 19536, 0),
        (3, 256, 1): (1, 16, 30576, 4)},
    "w32": {
        (3, 64, 1): (1, 16, 32, 4), (3, 128, 1): (1, 16, 9536, 4), (3, 192, 1): (1, 16, 19424, 4),
        (3, 256, 1): (1, 16, 30464, 4)},
    "w64": {
        (3, 64, 1): (1, 16, 64, 4), (3, 128, 1): (1, 16, 10496, 4), (3, 192, 1): (1, 16, 25216, 4),
        (3, 256, 1): (1, 16, 29504, 4)},
    "pk16": {
        (3, 64, 1): (1, 32, 16, 0), (3, 128, 1): (1, 32, 9504, 4), (3, 192, 1): (1, 32, 22112, 0)},
    "pk32": {
        (3, 64, 1): (1, 32, 32, 4), (3, 128, 1): (1, 32, 9536, 4), (3, 192, 1): (1, 32, 19328, 4)},
    "pk64": {
        (3, 64, 1): (1, 32, 64, 4), (3, 128, 1): (1, 32, 10112, 0), (3, 192, 1): (1, 32, 19712, 4)},
}


@pytest.fixture(scope="module")
def hq():
    import hadamard_rotated_bit_token_b200 as hq_mod
    from hadamard_rotated_bit_token_b200 import build as hq_build
    hq_build.build()
    hq_mod.load_library()
    return hq_mod


def _built(kind):
    """Every plan that has a kernel for operands of this kind."""
    rows = set(itertools.product((ROWS,), (1, 2, 4, 8), (1, 2, 4)))
    split = set(itertools.product((SPLIT,), (16, 32, 64, 128), (1, 2, 4, 8)))
    tiles = {(TILES, w, 1) for w in (64, 128, 192, 256)}
    pair = {(PAIR, w, 1) for w in (128, 192, 256)}
    if kind in ("bf16", "i8"):
        return rows | split | tiles | pair
    if kind.startswith("pk"):
        tiles -= {(TILES, 256, 1)}
    return (rows if kind == "pk" else set()) | tiles


def _desc(hq, kind, K, N):
    if kind == "bf16":
        return hq.DenseDesc(K, N)
    m = int(kind[-2:]) if kind != "i8" and kind[-1].isdigit() else 0
    return hq.LayerDesc(K, N, 1 if m else 16, out_order=m, centering=0,
                        code_format=1 if kind.startswith("pk") else 0)


def _plan(hq, kind, K, N, T, act=0, **kw):
    f = hq.hq_debug_dense_plan if kind == "bf16" else hq.hq_debug_linear_ep_plan
    return tuple(f(_desc(hq, kind, K, N), T, act, **kw))


@pytest.mark.parametrize("kind", sorted(CHOSEN))
def test_every_kernel_is_chosen_somewhere(hq, kind):
    assert set(CHOSEN[kind]) == _built(kind)
    for plan, (T, K, N, act) in CHOSEN[kind].items():
        assert _plan(hq, kind, K, N, T, act) == plan, (plan, T, K, N)


def test_plain_products_on_codes_keep_their_own_kernels(hq):
    """Without an epilogue, what is neither a few tokens nor a K split runs
    hq_linear's kernel, with hq_linear's tile."""
    for T, K, N in ((8192, 1152, 3456), (16384, 4096, 8192), (300, 1024, 4096)):
        p = _plan(hq, "i8", K, N, T, plain=True)
        q = hq.hq_debug_plan(hq.LayerDesc(K, N, 16), T, 148, 74)
        assert p == (LINEAR, q["gemm_bn"], 2 if q["gemm_pair"] else 1)
    assert _plan(hq, "i8", 1152, 3456, 1, plain=True)[0] == ROWS
    assert _plan(hq, "i8", 4608, 1152, 16, plain=True)[0] == SPLIT


def test_a_plan_that_is_set_is_taken_or_refused(hq):
    try:
        for plan in sorted(_built("bf16")):
            hq.hq_debug_set_product_plan(hq.ProductPlan(*plan))
            T = 2 if plan[0] == ROWS else 500
            for kind in ("bf16", "i8"):
                got = _plan(hq, kind, 2048, 272, T)
                assert got == plan if plan[0] != ROWS else got[0] == ROWS
        refused = [((ROWS, 1, 1), "bf16", 9, 2048), ((ROWS, 1, 1), "w32", 2, 2048),
                   ((SPLIT, 16, 8), "i8", 9, 7 * 128), ((SPLIT, 16, 1), "pk", 9, 2048),
                   ((SPLIT, 16, 1), "w16", 9, 2048), ((TILES, 256, 1), "pk", 9, 2048),
                   ((TILES, 256, 1), "pk32", 9, 2048), ((PAIR, 256, 1), "w64", 500, 2048),
                   ((PAIR, 128, 1), "pk", 500, 2048)]
        for plan, kind, T, K in refused:
            hq.hq_debug_set_product_plan(hq.ProductPlan(*plan))
            with pytest.raises(hq.HQError) as e:
                _plan(hq, kind, K, 256, T)
            assert e.value.status == UNSUPPORTED
        hq.hq_debug_set_product_plan(hq.ProductPlan(PAIR, 128))
        with pytest.raises(hq.HQError):
            _plan(hq, "bf16", 2048, 256, 500, pair_clusters=0)
        for bad in ((SPLIT, 48, 1), (SPLIT, 16, 3), (TILES, 96, 1), (PAIR, 64, 1), (LINEAR, 64, 1),
                    (6, 64, 1), (-1, 64, 1)):
            with pytest.raises(hq.HQError) as e:
                hq.hq_debug_set_product_plan(hq.ProductPlan(*bad))
            assert e.value.status == INVALID
    finally:
        hq.hq_debug_set_product_plan(None)
    assert _plan(hq, "bf16", 4096, 8192, 16384) == (PAIR, 256, 1)


def test_plan_queries_refuse_what_is_no_product(hq):
    for call in (lambda: hq.hq_debug_dense_plan(hq.DenseDesc(0, 8), 1),
                 lambda: hq.hq_debug_dense_plan(hq.DenseDesc(8, 8), 0),
                 lambda: hq.hq_debug_dense_plan(hq.DenseDesc(8, 8), 1, sms=0),
                 lambda: hq.hq_debug_linear_ep_plan(hq.LayerDesc(64, 0, 16), 1),
                 lambda: hq.hq_debug_linear_ep_plan(hq.LayerDesc(64, 64, 16), 1, pair_clusters=-1)):
        with pytest.raises(hq.HQError) as e:
            call()
        assert e.value.status == INVALID
