"""GPU test of the activations' fp32 values against the bounds that
include/hq_ops.h states, finer than a bf16 output shows.  Needs a B200.

The epilogue stores bf16(R + act(z)).  With z a bias (all codes zero) that is
known to fp32, and R = -bf16(act(z)), the sum is act's fp32 value less a bf16 one:
exact in fp32, as the two are within a factor of two.  Its rounding to bf16 is off
by at most 2^-8 of the difference; with inputs whose act(z) lies within 2^-13 of a
bf16 value that is 2^-21 of act(z).

The absolute 7e-18: two values share the reciprocal of d1 d2, d = 1 + e^-u, whose
result below 2^-126 is flushed to 0.  e^-u is at most 2^63.48 (u = -44), so that
takes d >= 2^62.52 of both, u <= -43.34, and silu is 43.34 2^-62.52 = 6.6e-18 there
and less below."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

SILU, GELU, GELU_TANH = 2, 3, 4
# tokens and the kernel (hq_debug_set_product_plan): few tokens, K split, tiles with
# either epilogue, a pair
KERNELS = [(1, (1, 1, 1)), (5, (2, 16, 2)), (40, (3, 64, 1)), (40, (3, 256, 1)), (300, (4, 192, 1))]
LOW = {SILU: -44.0, GELU: -13.5, GELU_TANH: -7.6}


@pytest.fixture(scope="module")
def hq():
    import hadamard_rotated_bit_token_b200 as hq_mod
    from hadamard_rotated_bit_token_b200 import build as hq_build
    hq_build.build()
    hq_mod.load_library()
    yield hq_mod
    hq_mod.hq_debug_set_product_plan(None)


def _exponent(z, act):
    return z if act == SILU else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)


def _exact(z, act):
    if act == GELU:
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    # sigmoid(u) = 1 / (1 + e^-u), e^u / (1 + e^u): no cancellation on either side
    u = _exponent(z, act)
    e = torch.exp(-u.abs())
    return z * torch.where(u < 0, e, torch.ones_like(e)) / (1 + e)


def _bound(z, act):
    """The error that the header allows."""
    a = _exact(z, act).abs()
    if act == GELU:
        return 2.0 ** -16 * a + 1.1e-7
    return 2.0 ** -20 * (1 + _exponent(z, act).abs().clamp(max=44.0) / 4) * a + 7e-18


@pytest.mark.parametrize("act", [SILU, GELU, GELU_TANH])
@pytest.mark.parametrize("T,plan", KERNELS)
def test_activation_within_its_stated_error(hq, act, T, plan):
    hq.hq_debug_set_product_plan(hq.ProductPlan(*plan))
    g = torch.Generator(device="cuda")
    g.manual_seed(act * 10 + T)
    K, N = 256, 4096
    total = 1 << 19                                  # values looked at
    A = torch.zeros(T, K, dtype=torch.int8, device="cuda")
    W = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    one = lambda n: torch.ones(n, device="cuda")
    desc = hq.LayerDesc(K, N, 16, centering=hq.HQ_CENTER_NONE)
    seen, worst = 0, 0.0
    while seen < total:
        z = torch.rand(1 << 20, generator=g, device="cuda") * (-LOW[act] + 6.0) + LOW[act]
        y = _exact(z.double(), act)
        yb = y.float().bfloat16().double()
        z = z[((y - yb).abs() <= 2.0 ** -13 * y.abs()) & (y.abs() > 1e-30)]
        z = z[: z.numel() // N * N].view(-1, N)
        assert z.shape[0] > 0
        for bias in z:
            y = _exact(bias.double(), act)
            R = -y.float().bfloat16().expand(T, N).contiguous()
            Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
            hq.hq_linear_ep(desc, A, one(T), None, W, one(N), None, bias.contiguous(),
                            hq.Epilogue(act, R), Y)
            exact = y + R[0].double()
            # the stored rounding, of a difference that is off by the bound itself
            tol = _bound(bias.double(), act) + 2.0 ** -8 * exact.abs()
            tol = tol * (1 + 2.0 ** -8)
            off = (Y.double() - exact).abs()
            assert bool((off <= tol).all()), [
                (float(bias[i]), float(exact[i]), float(Y[t, i]))
                for t, i in (off > tol).nonzero().tolist()[:5]]
            worst = max(worst, float((off / tol).max()))
        seen += z.numel()
    assert worst > 1e-3  # the comparison sees something
    assert hq.hq_check_device_error() == 0


@pytest.mark.parametrize("act", [SILU, GELU, GELU_TANH])
@pytest.mark.parametrize("T,plan", KERNELS)
def test_activation_far_below(hq, act, T, plan):
    """Below the lowest argument the value is 0 to the absolute part of the bound,
    down to -infinity."""
    hq.hq_debug_set_product_plan(hq.ProductPlan(*plan))
    K, N = 256, 64
    z = torch.cat((torch.linspace(LOW[act], 40 * LOW[act], N - 4),
                   torch.tensor([-1e10, -1e30, -3e38, float("-inf")]))).cuda()
    A = torch.zeros(T, K, dtype=torch.int8, device="cuda")
    W = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    one = lambda n: torch.ones(n, device="cuda")
    hq.hq_linear_ep(hq.LayerDesc(K, N, 16, centering=hq.HQ_CENTER_NONE), A, one(T), None, W, one(N),
                    None, z, hq.Epilogue(act), Y)
    limit = 1.1e-7 if act == GELU else 7e-18
    # at the lowest argument itself the value is not yet 0
    y = torch.where(torch.isfinite(z), _exact(z.double().clamp(min=-1e4), act), 0.0)
    assert bool(((Y.double() - y).abs() <= limit * (1 + 2.0 ** -8)).all())
    assert bool((Y <= 0).all())
