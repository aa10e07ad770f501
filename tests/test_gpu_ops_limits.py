"""GPU tests of the products' bounded waits: a wait that runs out (a test hook
withholds an arrival; nothing faults) is reported, the kernel ends by itself, and
the next call is right.  Needs a B200."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TIMEOUT = 5  # HQ_ERR_TIMEOUT


@pytest.fixture(scope="module")
def hq():
    import hadamard_rotated_bit_token_b200 as hq_mod
    from hadamard_rotated_bit_token_b200 import build as hq_build
    hq_build.build()
    hq_mod.load_library()
    return hq_mod


@contextlib.contextmanager
def _fault(hq, kind):
    hq.hq_debug_set_wait_limit(2_000_000)  # 2 ms
    hq.hq_debug_inject_fault(kind)
    try:
        yield
    finally:
        hq.hq_debug_inject_fault(hq.HQ_FAULT_NONE)
        hq.hq_debug_set_wait_limit(0)


def _dense(hq, T, K, N, seed=0):
    """(call, result): integer operands, whose sums are exact."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + T + K + N)
    X, W, R = (torch.randint(-3, 4, s, generator=g, device="cuda").to(torch.bfloat16)
               for s in ((T, K), (N, K), (T, N)))
    want = (X.double() @ W.double().t() + R.double()).float().bfloat16()

    def call():
        Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        hq.hq_dense(hq.DenseDesc(K, N), X, W, None, hq.Epilogue(residual=R), Y)
        return Y
    return call, want


def _linear(hq, T, K, N, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + T + K + N)
    A, W = (torch.randint(-7, 8, s, generator=g, device="cuda").to(torch.int8)
            for s in ((T, K), (N, K)))
    R = torch.randint(-3, 4, (T, N), generator=g, device="cuda").to(torch.bfloat16)
    one = lambda n: torch.ones(n, device="cuda")
    want = (A.double() @ W.double().t() + R.double()).float().bfloat16()
    desc = hq.LayerDesc(K, N, 16, centering=hq.HQ_CENTER_NONE)

    def call():
        Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        hq.hq_linear_ep(desc, A, one(T), None, W, one(N), None, None, hq.Epilogue(residual=R), Y)
        return Y
    return call, want


def _times_out_and_recovers(hq, call, want, kind):
    assert torch.equal(call(), want) and hq.hq_check_device_error() == 0
    with _fault(hq, kind):
        call()
        assert hq.hq_check_device_error() == TIMEOUT
    assert hq.hq_check_device_error() == 0
    for _ in range(3):
        assert torch.equal(call(), want)
    assert hq.hq_check_device_error() == 0


@pytest.mark.parametrize("make", [_dense, _linear])
@pytest.mark.parametrize("T,K,N", [(16, 512, 1152), (64, 1152, 1152), (64, 9216, 1152)])
def test_split_k_gives_up_and_recovers(hq, make, T, K, N):
    """A stage of the K split that never comes, where the producer has issued all
    its copies and left (few K blocks a CTA) and where it waits for a free stage."""
    _times_out_and_recovers(hq, *make(hq, T, K, N), hq.HQ_FAULT_SPLITK_WITHHOLD_STAGE)


# one output tile a CTA and several, one CTA a tile and pairs of them, few K
# blocks (the producer has left) and many
TILES = [(_dense, 600, 1152, 1152), (_dense, 4100, 512, 1152), (_dense, 7000, 4608, 1152),
         (_dense, 4096, 4608, 4608), (_linear, 2000, 320, 320), (_linear, 8192, 4608, 1152),
         (_linear, 4096, 4608, 4608)]


@pytest.mark.parametrize("make,T,K,N", TILES)
def test_tiles_give_up_and_recover(hq, make, T, K, N):
    """A stage of a tile kernel's main loop that never comes."""
    _times_out_and_recovers(hq, *make(hq, T, K, N), hq.HQ_FAULT_TILE_WITHHOLD_STAGE)


# tiles of 256 columns read the residual without a wait
@pytest.mark.parametrize("make,T,K,N", [(_dense, 600, 1152, 1152), (_dense, 4100, 512, 1152),
                                        (_linear, 2000, 320, 320), (_linear, 8192, 4608, 1152)])
def test_residual_box_gives_up_and_recovers(hq, make, T, K, N):
    """A box of the residual that never comes."""
    _times_out_and_recovers(hq, *make(hq, T, K, N), hq.HQ_FAULT_TILE_WITHHOLD_RESIDUAL)


# every tile kernel (kernel, columns, fault it knows), set by the plan hook
SET = [(k, w, f) for k, ws in ((3, (64, 128, 192, 256)), (4, (128, 192, 256))) for w in ws
       for f in ("STAGE", "RESIDUAL") if f == "STAGE" or w <= 192]


@pytest.mark.parametrize("make", [_dense, _linear])
@pytest.mark.parametrize("kernel,width,fault", SET)
@pytest.mark.parametrize("T,K,N", [(131, 272, 208), (5117, 1168, 1168)])
def test_every_tile_kernel_gives_up_and_recovers(hq, make, kernel, width, fault, T, K, N):
    call, want = make(hq, T, K, N)
    hq.hq_debug_set_product_plan(hq.ProductPlan(kernel, width))
    try:
        _times_out_and_recovers(hq, call, want, getattr(hq, f"HQ_FAULT_TILE_WITHHOLD_{fault}"))
    finally:
        hq.hq_debug_set_product_plan(None)
