"""Plain 64-bit forms of the gated feed-forward block's operators, and the error bounds their tests use; the roundings are
those of linear_reference (u = 2^-24).

  * A block-scaled product is a sum of K terms x w scaled by xs ws: the scales' product and the step that scales a block's sum
    and adds it are two roundings more, so (K + 32) u S bounds it, S the sum of the scaled terms' magnitudes.
  * A sum over a row in the norm's kernels is at most 128 additions by one lane (8 elements a step, 16 steps at the longest
    row tested), then a tree of 5 + 32: 165 u times the magnitudes' sum, SUM below.
"""
import torch

import linear_reference as ref
from linear_reference import SLOPE, U, act_slope, act_value, product, rounded

SUM = 165 * U


def assert_within(got, ref_and_bound, what=""):
    """linear_reference's, knowing that fp16 rounds magnitudes from 65520 (its largest number, 65504, and half a step of 32)
    on to infinity: beyond that an infinity of the value's sign is the rounded value, within the bound of it either."""
    value, bound = ref_and_bound
    if got.dtype is torch.float16:
        must, may = value.abs() - bound >= 65520, value.abs() + bound >= 65520
        right = got.double() == torch.copysign(torch.full_like(value, float("inf")), value)
        assert bool(right[must].all()), f"{what}: a finite number beyond fp16's range"
        got = torch.where(may & right, value, got.double())
    ref.assert_within(got, (value, bound), what)


def value_bound(e, z, act):
    """The bound on act(z) for z within e."""
    return SLOPE * e + (0 if act in ("none", "relu") else 2.0 ** -19 * (z.abs() + 1))


def spread(s, rows, M, K):
    """The scale of every element of an M x K matrix with a scale for every `rows` x 128."""
    return s.double().repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :K]


def scaled(q, s, rows):
    """The matrix that 8-bit values and their scales stand for (None: scales of 1)."""
    return q.double() if s is None else q.double() * spread(s, rows, *q.shape)


def scaled_product(x, w, alpha=1.0):
    """(alpha x·w^T, the bound on its block-scaled fp32 sum) for matrices that `scaled` gave."""
    return alpha * (x @ w.t()), (x.shape[1] + 32) * U * abs(alpha) * (x.abs() @ w.abs().t())


def with_bias(z, e, bias):
    if bias is None:
        return z, e
    z = z + bias.double()
    return z, e + 16 * U * (z.abs() + bias.double().abs())


def glu(z, ez, act, out_dtype):
    """((H, its bound), (Z, its bound)) from Z = [G | U] within ez."""
    N = z.shape[1] // 2
    g, u, eg, eu = z[:, :N], z[:, N:], ez[:, :N], ez[:, N:]
    a, ea = act_value(g, act), value_bound(eg, g, act)
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu + 2 * U * h.abs()
    return (h, rounded(eh, h, out_dtype)), (z, rounded(ez, z, out_dtype))


def glu_dgrad(d, ed, Z, act, out_dtype, dbias_dtype, dbias0=None, beta=0.0):
    """((dZ, its bound), (dbias, its bound)) for d within ed."""
    z = Z.double()
    N = z.shape[1] // 2
    g, u = z[:, :N], z[:, N:]
    a, s = act_value(g, act), act_slope(g, act)
    ea, es = value_bound(torch.zeros_like(g), g, act), (0 if act in ("none", "relu") else 2.0 ** -17)
    dz = torch.cat([d * u * s, d * a], 1)
    e = torch.cat([u.abs() * (s.abs() * ed + (d.abs() + ed) * es), a.abs() * ed + (d.abs() + ed) * ea], 1) + 4 * U * dz.abs()
    M = d.shape[0]
    b, eb = dz.sum(0), e.sum(0) + (M + 16) * U * dz.abs().sum(0)
    if beta:
        b = b + beta * dbias0.double()
        eb = eb + 4 * U * (b.abs() + abs(beta) * dbias0.double().abs())
    return (dz, rounded(e, dz, out_dtype)), (b, rounded(eb, b, dbias_dtype))


def quantize(X, block_rows, dtype):
    """(Q, scales) with the definition's roundings, from fp64 quotients and products."""
    M, K = X.shape
    x, rows, cols = X.double(), -(-M // block_rows), -(-K // 128)
    full = torch.zeros((rows * block_rows, cols * 128), dtype=torch.float64, device=X.device)
    full[:M, :K] = x
    a = full.view(rows, block_rows, cols, 128).abs().amax((1, 3))
    s = torch.maximum((a / torch.full_like(a, torch.finfo(dtype).max)).float(), torch.full_like(a, 2.0 ** -126).float())
    r = (1 / s.double()).float()
    return (x * spread(r, block_rows, M, K)).float().to(dtype), s


def layer_norm(X, w, b, eps, out_dtype):
    """((Y, bound), (mean, bound), (rstd, bound)).  With d the error of the mean, the mean square of x - mean is off by
    2 sqrt(v) d + d^2 and the roundings of its sum; half of that, relative to v + eps, is rstd's relative error (1.5 times the
    half covers the second order while it stays under 1/4)."""
    x = X.double()
    mean = x.mean(1, keepdim=True)
    em = SUM * x.abs().mean(1, keepdim=True) + 2 * U * mean.abs()
    c = x - mean
    v = c.square().mean(1, keepdim=True)
    ev = (SUM + 8 * U) * (v + em * em) + 2 * v.sqrt() * em + em * em
    rstd = (v + eps).rsqrt()
    er = rstd * (0.75 * ev / (v + eps) + 8 * U)
    ww = torch.ones_like(x[0]) if w is None else w.double()
    y = c * rstd * ww + (0 if b is None else b.double())
    ec = em + 2 * U * (c.abs() + em)
    ey = ww.abs() * ((rstd + er) * ec + c.abs() * er) + 6 * U * ((c * rstd * ww).abs() + y.abs())
    f32 = torch.float32
    return (y, rounded(ey, y, out_dtype)), (mean[:, 0], rounded(em, mean, f32)[:, 0]), (rstd[:, 0], rounded(er, rstd, f32)[:, 0])


def layer_norm_grad(dY, X, mean, rstd, w, residual, out_dtype, dtypes, beta=0.0, dw0=None, db0=None):
    """((dX, bound), (dw, bound), (db, bound)) for the given statistics."""
    dy, x, mu, r = dY.double(), X.double(), mean.double()[:, None], rstd.double()[:, None]
    ww = torch.ones_like(x[0]) if w is None else w.double()
    h = (x - mu) * r
    eh = 3 * U * h.abs()
    g = dy * ww
    eg = U * g.abs()
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    ec1 = eg.mean(1, keepdim=True) + SUM * g.abs().mean(1, keepdim=True) + 2 * U * c1.abs()
    ec2 = (g.abs() * eh + h.abs() * eg).mean(1, keepdim=True) + SUM * (g * h).abs().mean(1, keepdim=True) + 2 * U * c2.abs()
    dx = r * (g - c1 - h * c2)
    edx = r * (eg + ec1 + h.abs() * ec2 + c2.abs() * eh + 4 * U * (g.abs() + c1.abs() + (h * c2).abs()))
    if residual is not None:
        dx = dx + residual.double()
        edx = edx + 2 * U * (dx.abs() + residual.double().abs())
    M = dy.shape[0]
    sums = []
    for v, e, v0, t in ((dy * h, dy.abs() * eh, dw0, dtypes[0]), (dy, torch.zeros_like(dy), db0, dtypes[1])):
        s, es = v.sum(0), e.sum(0) + (M + 16) * U * v.abs().sum(0)
        if beta:
            s = s + beta * v0.double()
            es = es + 4 * U * (s.abs() + abs(beta) * v0.double().abs())
        sums.append((s, rounded(es, s, t)))
    return (dx, rounded(edx, dx, out_dtype)), sums[0], sums[1]
