"""Plain 64-bit forms of the linear-layer operators, and the error bounds their tests use.

Bounds (u = 2^-24, the fp32 unit roundoff):
  * a sum of K products in fp32, in any order, is within (K + 16) u S of the exact one, S the sum of the
    products' magnitudes (16 covers alpha, bias and the joins of partial sums);
  * the activations' slopes are at most 1.13 in magnitude, their values are evaluated within 2^-19 (|z| + 1) and
    their slopes within 2^-17 (the fast exponential's error at the clamped arguments);
  * the result is rounded once to its type: half the spacing of the type's numbers, which is at most eps / 2 of
    the value (2^-11 for float16, 2^-8 for bfloat16, 2^-24 for float32), plus the type's smallest subnormal.
"""
import math

import torch

U = 2.0 ** -24
ROUND = {t: torch.finfo(t).eps / 2 for t in (torch.float16, torch.bfloat16, torch.float32)}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}
SLOPE = 1.13
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def phi(z):
    return torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def act_value(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, act):
    if act == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), torch.ones_like(z) + 0 * z)
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * phi(z)
    if act == "gelu_tanh":
        s = torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
        return s + z * s * (1 - s) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def rounded(bound, value, dtype):
    """The bound on a value that is computed within `bound` and then rounded to `dtype`."""
    return bound * (1 + ROUND[dtype]) + ROUND[dtype] * value.abs() + TINY[dtype]


def product(A, B, alpha=1.0):
    """(alpha A·B in fp64, the bound on its fp32 sum) for A (M x K) and B (K x N)."""
    a, b = A.double(), B.double()
    K = a.shape[1]
    return alpha * (a @ b), (K + 16) * U * abs(alpha) * (a.abs() @ b.abs())


def linear(X, W, bias, act, residual, out_dtype, alpha=1.0):
    """((Y, its bound), (Z, its bound))."""
    z, ez = product(X, W.t(), alpha)
    if bias is not None:
        z = z + bias.double()
        ez = ez + 16 * U * (z.abs() + bias.double().abs())
    y = act_value(z, act)
    ey = SLOPE * ez + (0 if act in ("none", "relu") else 2.0 ** -19 * (z.abs() + 1))
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2 * U * (y.abs() + residual.double().abs())
    return (y, rounded(ey, y, out_dtype)), (z, rounded(ez, z, out_dtype))


def through_act(g, eg, Z, act, out_dtype, dbias_dtype, dbias0=None, beta=0.0):
    """((d, its bound), (dbias, its bound)) for d = g * act'(Z)."""
    s = torch.ones_like(g) if Z is None else act_slope(Z.double(), act)
    d = g * s
    ed = eg * SLOPE + g.abs() * (2.0 ** -17 if act not in ("none", "relu") else 0) + 4 * U * d.abs()
    M = g.shape[0]
    b = d.sum(0)
    eb = ed.sum(0) + (M + 16) * U * d.abs().sum(0)
    if beta:
        b = b + beta * dbias0.double()
        eb = eb + 4 * U * (b.abs() + abs(beta) * dbias0.double().abs())
    return (d, rounded(ed, d, out_dtype)), (b, rounded(eb, b, dbias_dtype))


def wgrad(dY, X, out_dtype, alpha=1.0, beta=0.0, dW0=None):
    d, e = product(dY.t(), X, alpha)
    if beta:
        d = d + beta * dW0.double()
        e = e + 4 * U * (d.abs() + abs(beta) * dW0.double().abs())
    return d, rounded(e, d, out_dtype)


def assert_within(got, ref_and_bound, what=""):
    ref, bound = ref_and_bound
    assert tuple(got.shape) == tuple(ref.shape), what
    bad = ~((got.double() - ref).abs() <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first at {i}: "
                             f"{got[i].item()} for {ref[i].item()}, bound {bound[i].item()}")
