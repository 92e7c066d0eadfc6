"""The linear-layer operators where their parts meet: staging buffers between ragged and whole boxes, shares that end
inside a warp, calls on several streams at once, contractions longer than one accumulator keeps.

On integer data the sums are exact, so results must match the 64-bit forms bit for bit.
"""
import pytest
import torch

import linear_reference as ref
from dense_tiled_gemm_04_gb300 import native
from test_gpu_linear import BF16, F16, F32, Guarded, clean, g, gen, matrix, same, vector  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

TILES = [native.CONFIG_128x128, native.CONFIG_128x256, native.CONFIG_256x256]


# ------------------------------------------------------------------ staging buffers

# A column count that is no multiple of 8 sends a warp's last box of a tile through masked stores, between boxes that
# leave by TMA from alternating buffers.  Many tiles a CTA and short contractions keep those stores close together.
@pytest.mark.parametrize("config", TILES)
@pytest.mark.parametrize("M,N,K,ctas", [(9000, 8, 1001, 0), (9000, 64, 8191, 0), (1100, 64, 301, 6), (2000, 8, 1003, 6),
                                        (700, 200, 1001, 6)])
def test_dgrad_ragged_columns_without_an_activation(g, config, M, N, K, ctas):  # noqa: F811
    g.set_option(native.OPT_CONFIG, config)
    g.set_option(native.OPT_MAX_CTAS, ctas)
    for dtype in (F16, BF16):
        r = gen(M + K)
        dY, W = matrix(r, M, N, dtype, ints=True), matrix(r, N, K, dtype, ints=True)
        d = dY.double() @ W.double()
        want, sums = d.to(dtype), d.sum(0).float()
        for with_sums in (True, False):
            for _ in range(4):
                dX, db = Guarded(M, K, dtype), Guarded(1, K, F32)
                g.linear_dgrad(dY, W, out=dX.t, dbias=db.t[0] if with_sums else None)
                same(dX.t, want, "dX")
                dX.check("dX")
                if with_sums:
                    same(db.t[0], sums, "dbias")
                    db.check("dbias")


# ------------------------------------------------------------------ shares that end inside a warp

# The lanes of a warp take different paths before the cluster's barriers: features and tokens that end inside a
# warp's units, a bias and a residual whose last groups of four are read one by one, ranks with fewer units than threads.
@pytest.mark.parametrize("M,N,K", [(1, 5, 4096), (3, 131, 2048), (17, 1003, 4100), (61, 130, 1024), (127, 2047, 1000)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_cluster_shares_that_end_inside_a_warp(g, M, N, K, dtype):  # noqa: F811
    r = gen(M + N + K)
    X, W = matrix(r, M, K, dtype, ints=True), matrix(r, N, K, dtype, ints=True)
    z = X.double() @ W.double().t()
    for bias in (vector(r, N, F32, ints=True, offset=1), vector(r, N, dtype, ints=True, offset=3), None):
        res = matrix(r, M, N, dtype, ints=True)
        y = z + (0 if bias is None else bias.double())
        y = ref.act_value(y, "relu") + res.double()
        for _ in range(3):
            Y = Guarded(M, N, dtype)
            g.linear(X, W, bias, act="relu", residual=res, out=Y.t)
            same(Y.t, y.to(dtype), "Y")
            Y.check("Y")
    dY = matrix(r, M, N, dtype, ints=True)
    d = dY.double() @ W.double()
    dX, db = Guarded(M, K, dtype), Guarded(1, K, F32)
    g.linear_dgrad(dY, W, out=dX.t, dbias=db.t[0])
    same(dX.t, d.to(dtype), "dX")
    same(db.t[0], d.sum(0).float(), "dbias")
    dX.check("dX"), db.check("dbias")
