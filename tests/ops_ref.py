"""Plain 64-bit forms of the operators beside the quantized layer, and the
bounds their fp32 evaluations are held to (test-side only).

Bounds.  u = 2^-24 is half a step of fp32 relative to a value.
  products   bf16 products are exact in fp32; a sum of K of them and a bias is
             off by at most K 2^-23 (sum |x w| + |b|), one truncated addition
             a product.  Integer-valued operands sum exactly.
  act        silu / gelu_tanh: exponential and reciprocal instructions of 2^-22
             each, the argument's rounding 3 u |u_arg|: relative error at most
             2^-20 (1 + |u_arg|), u_arg capped where the result vanishes;
             gelu adds 1.4e-5 relative and 1.1e-7 absolute (its fit).  All
             three enter no lower than z = -44 (-7.6, -13.5), where z sigmoid(u)
             is -44 / (1 + e^44) = -3.5e-18 (less for the others): below, the
             result is off by at most 4e-18.
  slopes     |act'| <= 1.13 for all of them.
The stored value is the rounding of an fp32 value within tol of the exact one;
rounding is monotone, so it lies between the roundings of exact - tol and
exact + tol."""
import math

import numpy as np
import torch

NONE, RELU, SILU, GELU, GELU_TANH = range(5)
ACTS = {"none": NONE, "relu": RELU, "silu": SILU, "gelu": GELU, "gelu_tanh": GELU_TANH}
U = 2.0 ** -24


def act64(z, act):
    if act == RELU:
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == SILU:
        return z / (1 + torch.exp(-z))
    if act == GELU:
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if act == GELU_TANH:
        v = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
        return z / (1 + torch.exp(-2 * v))
    return z


def act_tol(z, act):
    """Bound of the fp32 activation's error at z (its own, not z's)."""
    a = act64(z, act).abs()
    if act in (NONE, RELU):
        return torch.zeros_like(a)
    arg = z.abs()
    if act == GELU_TANH:
        arg = 1.6 * (z.abs() + 0.045 * z.abs() ** 3)
    if act == GELU:
        arg = z.abs() * (1.6 + 0.075 * z.abs() ** 2)
    tol = 2.0 ** -20 * (1 + arg.clamp(max=128.0)) * a + 4e-18
    if act == GELU:
        tol = tol + 1.4e-5 * a + 1.1e-7
    return tol


def epilogue64(z, ztol, act, residual=None, gate=None, gate_rows=0):
    """(exact, tol) of residual + gate * act(z)."""
    y = act64(z, act)
    tol = 1.13 * ztol + act_tol(z, act)
    T = z.shape[0]
    if gate is not None:
        g = gate.double()[torch.arange(T, device=z.device) // gate_rows]
        y, tol = y * g, tol * g.abs()
    mag = y.abs()
    if residual is not None:
        y = y + residual.double()
        mag = mag + residual.double().abs()
    return y, tol + 4 * U * mag


def check_rounded(got, exact, tol, what):
    """got (bf16) lies between the roundings of exact -+ tol."""
    lo = (exact - tol).float().bfloat16().double()
    hi = (exact + tol).float().bfloat16().double()
    # exact -> float -> bf16 rounds twice: at most one fp32 step, within tol's slack
    lo = torch.minimum(lo, (exact - tol - 2 * U * exact.abs()).float().bfloat16().double())
    hi = torch.maximum(hi, (exact + tol + 2 * U * exact.abs()).float().bfloat16().double())
    g = got.double()
    bad = ~((g >= lo) & (g <= hi))
    n = int(bad.sum())
    if n:
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {n} of {bad.numel()} outside their bounds, first at {i}: "
                             f"got {float(g[i])}, exact {float(exact[i])}, tol {float(tol[i])}")


def rel_frob(got, exact):
    return float((got.double() - exact).norm() / exact.norm())


def dense64(X, W, bias):
    """(z, bound of the fp32 sum's error)."""
    x, w = X.double(), W.double()
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    return z, (X.shape[1] + 1) * 2.0 ** -23 * mag


def linear64(a_codes, a_scale, a_mean, w_codes, w_scale, colsum, bias, out_order=0):
    """(z, bound): integer sums are exact; the fp32 epilogue rounds four times,
    the weight-only form's transform log2(m) + 2 times more, each relative to
    the magnitudes it adds."""
    acc = a_codes.double() @ w_codes.double().t()
    z = acc * a_scale.double()[:, None] * w_scale.double()
    mag = z.abs()
    n = 4
    if out_order > 1:
        N = z.shape[1]
        h = torch.tensor([[1.0]], dtype=torch.float64, device=z.device)
        while h.shape[0] < out_order:
            h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
        s = 1.0 / math.sqrt(out_order)
        z = (z.view(-1, N // out_order, out_order) @ h * s).reshape(-1, N)
        mag = (mag.view(-1, N // out_order, out_order) @ h.abs() * s).reshape(-1, N)
        n = 8 + int(math.log2(out_order))
    if a_mean is not None:
        t = a_mean.double()[:, None] * colsum.double()
        z, mag = z + t, mag + t.abs()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    return z, n * U * mag


def unpack_i4(b, K):
    """[T, K/2] bytes -> [T, K] codes, even element in the low nibble."""
    v = b.view(torch.int8)
    return torch.stack(((v << 4) >> 4, v >> 4), dim=2).reshape(-1, K)


def pack_i4(codes):
    c = codes.to(torch.int16)
    return ((c[:, 0::2] & 15) | ((c[:, 1::2] & 15) << 4)).to(torch.uint8)


def group_norm64(X, G, gamma, beta, eps, act, n_sum=700):
    """(exact, tol).  The statistics are sums of at most n_sum parts one
    after the other (rows of a thread, threads, channels, chunks); with D the
    group's largest distance between values:
      mean off by <= n_sum u D;  variance, relative: n_sum u (1 + 4 D^2 / var),
    capped at what the tests' own inputs allow, and the rest is four roundings."""
    B, C = X.shape[0], X.shape[-1]
    x = X.double().reshape(B, -1, G, C // G)
    mean = x.mean(dim=(1, 3), keepdim=True)
    var = ((x - mean) ** 2).mean(dim=(1, 3), keepdim=True)
    D = x.amax(dim=(1, 3), keepdim=True) - x.amin(dim=(1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    n = (x - mean) * rstd
    dn = n_sum * U * (D * rstd + n.abs() * 0.5 * (1 + 4 * D ** 2 / (var + eps))) + 8 * U * n.abs()
    dn = dn + 2 * U * x.abs() * rstd
    ga = (torch.ones(C, device=X.device) if gamma is None else gamma).double().view(G, -1)
    be = (torch.zeros(C, device=X.device) if beta is None else beta).double().view(G, -1)
    z = n * ga + be
    tol = dn * ga.abs() + 4 * U * ((n * ga).abs() + be.abs())
    y = act64(z, act)
    return y.reshape(X.shape), (1.13 * tol + act_tol(z, act) + 4 * U * y.abs()).reshape(X.shape)
