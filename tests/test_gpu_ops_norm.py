"""GPU tests of the group norm at the ends of its number range.  Needs a B200."""
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


# small tensors (one launch) and others, vectors of 8, 4, 2 and 1 channels, and
# rows wider than a block
SHAPES = [(2, 300, 64, 8), (1, 4096, 320, 32), (2, 500, 36, 3), (3, 1000, 66, 6), (2, 700, 77, 11),
          (1, 30000, 128, 32), (1, 600, 8192, 1), (160, 9, 64, 8)]


@pytest.mark.parametrize("B,S,C,G", SHAPES)
def test_squares_past_fp32_are_no_silent_zero(hq, B, S, C, G):
    """Finite values whose squared deviations overflow fp32: the group is NaN, as
    with an infinity, and not beta; its neighbours are as without it."""
    X = torch.randn(B, S, C, generator=_gen(C), device="cuda").to(torch.bfloat16)
    norm = hq.GroupNorm(C, G, act=hq.HQ_ACT_SILU)
    n = C // G
    calm = norm(X)
    for big in (1e20, -3e38):
        for where in ("one", "all"):
            Z = X.clone()
            if where == "one":
                Z[0, S // 2, 0] = big
            else:
                Z[0, :, :n] *= abs(big) / 4
            Y = norm(Z)
            assert bool(Y[0, :, :n].isnan().all()), (big, where)
            assert torch.equal(Y[0, :, n:], calm[0, :, n:]) and torch.equal(Y[1:], calm[1:])
    assert hq.hq_check_device_error() == 0


@pytest.mark.parametrize("B,S,C,G", SHAPES)
def test_large_values_whose_squares_fit(hq, B, S, C, G):
    """The largest scale that is sure to fit (sums of squares below 2^127): the
    result does not depend on the scale, a power of two."""
    X = torch.randn(B, S, C, generator=_gen(C + 1), device="cuda").to(torch.bfloat16)
    norm = hq.GroupNorm(C, G, eps=0.0)
    want = norm(X)
    assert bool(want.isfinite().all())
    # |x| < 8, S C values a group at most 2^23: 2^k with 2 k + 6 + 23 < 127
    assert torch.equal(norm(X * 2.0 ** 48), want)
    assert torch.equal(norm(X * 2.0 ** -30), want)
    assert hq.hq_check_device_error() == 0


# rows: those that a block's threads start with, one or a few rows a thread
@pytest.mark.parametrize("B,S,C,G,rows,v", [
    (1, 1 << 27, 8, 1, 512, 139.0), (1, (1 << 24) + 9, 128, 8, 32, 182.0),
    (1, 300000, 8192, 1, 1, 182.0), (1, (1 << 26) + 1, 7, 7, 73, 139.0),
    (2, (1 << 23) + 3, 66, 6, 15, 182.0), (1, (1 << 24) + 9, 128, 8, 3200, 182.0)])
def test_a_first_value_far_from_thousands_of_equal_ones(hq, B, S, C, G, rows, v):
    """One value in the threads' first rows of the first chunk, zeros behind: the
    variance is all that value's, and the squares of the others' distance from it
    must not swamp it.  Tensors of up to 5 GB, whose statistics are known exactly."""
    X = torch.zeros(B, S, C, dtype=torch.bfloat16, device="cuda")
    X[:, :rows] = v
    Y = hq.GroupNorm(C, G)(X)
    mean = v * rows / S
    var = v * v * (rows / S) * (1 - rows / S)
    for got, x in ((Y[:, :rows], v), (Y[:, rows:rows + 5000], 0.0), (Y[:, -5000:], 0.0)):
        want = (x - mean) / (var + 1e-5) ** 0.5
        # one rounding to bf16, and 2^-11 for the statistics
        assert bool(((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * abs(want)).all()), (
            x, want, float(got.double().min()), float(got.double().max()))
    assert hq.hq_check_device_error() == 0
