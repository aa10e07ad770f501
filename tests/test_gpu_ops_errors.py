"""GPU test of what a refused launch leaves behind.  Needs a B200."""
import ctypes

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


class _InvalidatedCapture:
    """A stream whose capture was spoiled by a synchronization: every launch on it
    is refused on the host, until the capture ends."""

    def __enter__(self):
        torch.zeros(1, device="cuda")
        self.cu = ctypes.CDLL("libcuda.so.1")
        self.stream = ctypes.c_void_p()
        assert self.cu.cuStreamCreate(ctypes.byref(self.stream), 1) == 0
        assert self.cu.cuStreamBeginCapture_v2(self.stream, 1) == 0
        assert self.cu.cuStreamSynchronize(self.stream) != 0
        return self.stream.value

    def __exit__(self, *exc):
        graph = ctypes.c_void_p()
        assert self.cu.cuStreamEndCapture(self.stream, ctypes.byref(graph)) != 0
        assert self.cu.cuStreamDestroy_v2(self.stream) == 0


def test_a_refused_launch_is_reported_once(hq):
    """The call that was refused says so; the next ones, whatever kernel they run,
    succeed and give their results."""
    X = torch.ones(40, 1152, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(64, 1152, dtype=torch.bfloat16, device="cuda")
    d = hq.DenseDesc(1152, 64)
    norms = [torch.randn(1, S, 64, device="cuda").to(torch.bfloat16) for S in (100, 30000)]
    out = lambda n: torch.empty(n, 64, dtype=torch.bfloat16, device="cuda")
    nd = hq.GroupNormDesc(64, 8)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    kernels = [hq.ProductPlan(*p) for p in ((1, 1, 1), (2, 16, 4), (3, 64, 1), (4, 128, 1))]
    Y, Yn = [out(8) for _ in kernels], [torch.empty_like(X) for X in norms]
    calls = []
    for plan, y in zip(kernels, Y):
        def dense(stream, plan=plan, y=y):
            hq.hq_debug_set_product_plan(plan)
            try:
                hq.hq_dense(d, X[:8], W, None, None, y, stream=stream)
            finally:
                hq.hq_debug_set_product_plan(None)
        calls.append(dense)
    for x, y in zip(norms, Yn):
        calls.append(lambda stream, x=x, y=y: hq.hq_group_norm(nd, x, None, None, y, ws, stream))
    for call in calls:
        call(None)                              # attributes are set, nothing left to do but launch
    torch.cuda.synchronize()
    for refused in calls:
        for y in Y:
            y.zero_()
        with _InvalidatedCapture() as stream:
            with pytest.raises(hq.HQError) as e:
                refused(stream)
            assert e.value.status == 4          # HQ_ERR_CUDA
        for call in calls:
            call(None)
        torch.cuda.synchronize()
        assert all(bool((y == 1152).all()) for y in Y)
    assert hq.hq_check_device_error() == 0
