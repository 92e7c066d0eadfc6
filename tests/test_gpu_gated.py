"""The gated feed-forward block's operators on the GPU against plain 64-bit forms: sizes from one element to several tiles,
ragged edges, padded rows, empty dimensions, every activation and type, block scales, in-place forms, streams, graphs,
refusals, and a block of them together, trained and served.

On integer data (scales powers of two) with act none or relu every sum is exact, so results must match bit for bit; elsewhere
they must lie within the bounds that gated_reference derives.  Inputs sit in NaN-padded rows, outputs in sentinel-filled buffers.
"""
import ctypes
import threading

import pytest
import torch

import gated_reference as gref
import linear_reference as ref
from dense_tiled_gemm_04_gb300 import native
from test_gpu_linear import BF16, E4M3, E5M2, F16, F32, SHAPES, Guarded, gen, matrix, pitch, same, vector

pytestmark = pytest.mark.gpu

TYPES8 = [(E4M3, BF16), (E4M3, F16), (E5M2, BF16), (E5M2, F16)]
CONFIGS = [native.CONFIG_AUTO, native.CONFIG_128x128, native.CONFIG_128x256, native.CONFIG_256x256]


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_tiled_gemm_04_gb300 import build

    build.build()
    h = native.Gemm(0)
    yield h
    h.close()


@pytest.fixture(autouse=True)
def clean(request):
    yield
    if "g" in request.fixturenames:
        h = request.getfixturevalue("g")
        assert h.sync_status() == native.OK
        h.set_option(native.OPT_CONFIG, native.CONFIG_AUTO)
        h.set_option(native.OPT_MAX_CTAS, 0)


def scales(r, rows, cols, powers=False, pad=1):
    """rows x cols scales in NaN-padded rows; powers: 1/4 to 4."""
    buf = torch.full((rows + 1, cols + pad), float("nan"), device="cuda")
    s = 2.0 ** torch.randint(-2, 3, (rows, cols), generator=r, device="cuda").float() if powers else \
        torch.exp(torch.randn((rows, cols), generator=r, device="cuda"))
    buf[:rows, :cols] = s
    return buf[:rows, :cols]


def blocks(n):
    return -(-n // 128)


def stacked(W, ws):
    """The 2N x K weights of a gated layer that stacked values and stacked block scales stand for."""
    if ws is None:
        return W.double()
    N, n = W.shape[0] // 2, ws.shape[0] // 2
    return torch.cat([gref.scaled(W[:N], ws[:n], 128), gref.scaled(W[N:], ws[n:], 128)])


# ------------------------------------------------------------------ block scales

@pytest.mark.parametrize("M,N,K", SHAPES + [(40, 260, 3000), (257, 400, 1000)])
def test_scaled_integers_are_exact(g, M, N, K):
    r = gen(M + N + K)
    for dtype, out in ((E4M3, F16), (E5M2, BF16)):
        X, W = matrix(r, M, K, dtype, ints=True), matrix(r, N, K, dtype, ints=True, pad=0)
        xs, ws = scales(r, M, blocks(K), powers=True), scales(r, blocks(N), blocks(K), powers=True, pad=3)
        bias, res = vector(r, N, F32, ints=True, offset=1), matrix(r, M, N, out, ints=True)
        z = gref.scaled(X, xs, 1) @ gref.scaled(W, ws, 128).t() + bias.double()
        Y, Z = Guarded(M, N, out), Guarded(M, N, out)
        g.linear_scaled(X, W, xs, ws, bias, act="relu", residual=res, out=Y.t, preact=Z.t)
        same(Z.t, z.to(out), "Z")
        same(Y.t, (z.clamp_min(0) + res.double()).to(out), "Y")
        Y.check("Y"), Z.check("Z")


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_scaled_against_64_bits(g, M, N, K, act):
    r = gen(3 * M + N + K)
    for (dtype, out), (with_x, with_w) in zip(TYPES8, [(True, True), (True, False), (False, True), (False, False)]):
        X, W = matrix(r, M, K, dtype), matrix(r, N, K, dtype)
        xs, ws = scales(r, M, blocks(K)) if with_x else None, scales(r, blocks(N), blocks(K)) if with_w else None
        bias, res = vector(r, N, out, offset=3), matrix(r, M, N, out)
        alpha = K ** -0.5
        Y, Z = Guarded(M, N, out), Guarded(M, N, out)
        g.linear_scaled(X, W, xs, ws, bias, act=act, residual=res, out=Y.t, preact=Z.t, alpha=alpha)
        z, ez = gref.with_bias(*gref.scaled_product(gref.scaled(X, xs, 1), gref.scaled(W, ws, 128), alpha), bias)
        y = ref.act_value(z, act) + res.double()
        ey = gref.value_bound(ez, z, act) + 2 * ref.U * (y.abs() + res.double().abs())
        gref.assert_within(Z.t, (z, ref.rounded(ez, z, out)), f"Z {dtype} {out}")
        gref.assert_within(Y.t, (y, ref.rounded(ey, y, out)), f"Y {dtype} {out}")
        Y.check(), Z.check()


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("M,N,K", [(300, 520, 1100), (257, 1000, 300), (700, 300, 4100)])
@pytest.mark.parametrize("ctas", [0, 6])
def test_scaled_every_tile(g, config, M, N, K, ctas):
    # Several tiles per CTA: every second one walks its K blocks backwards; and shares of K blocks (few CTAs).
    g.set_option(native.OPT_CONFIG, config)
    g.set_option(native.OPT_MAX_CTAS, ctas)
    r = gen(M)
    for dtype, out in ((E4M3, BF16), (E5M2, F16)):
        X, W, xs, ws = matrix(r, M, K, dtype), matrix(r, N, K, dtype), scales(r, M, blocks(K)), scales(r, blocks(N), blocks(K))
        Y = Guarded(M, N, out)
        g.linear_scaled(X, W, xs, ws, out=Y.t, alpha=K ** -0.5)
        z, ez = gref.scaled_product(gref.scaled(X, xs, 1), gref.scaled(W, ws, 128), K ** -0.5)
        gref.assert_within(Y.t, (z, ref.rounded(ez, z, out)), f"{dtype} {out}")
        Y.check()


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (3, 1024, 20000), (33, 1024, 8192), (64, 520, 9000), (65, 136, 12000),
                                   (128, 2048, 2048), (10, 30000, 640), (200, 128, 3000)])
def test_scaled_split_over_a_cluster(g, M, N, K):
    # More K blocks per CTA than accumulators: their ring comes round.
    r = gen(M + K)
    X, W, xs, ws = matrix(r, M, K, E4M3), matrix(r, N, K, E4M3), scales(r, M, blocks(K)), scales(r, blocks(N), blocks(K))
    res = matrix(r, M, N, BF16)
    Y = Guarded(M, N, BF16)
    g.linear_scaled(X, W, xs, ws, residual=res, out=Y.t, alpha=K ** -0.5)
    z, ez = gref.scaled_product(gref.scaled(X, xs, 1), gref.scaled(W, ws, 128), K ** -0.5)
    y = z + res.double()
    gref.assert_within(Y.t, (y, ref.rounded(ez + 2 * ref.U * (y.abs() + res.double().abs()), y, BF16)))
    Y.check()


@pytest.mark.parametrize("M", [2, 200])
def test_scaled_special_values(g, M):
    # A NaN scale of X reaches its row alone, one of W the 128 outputs of its block alone; infinities likewise.
    X, W = torch.ones((M, 384), device="cuda").to(E4M3), torch.ones((300, 384), device="cuda").to(E4M3)
    xs, ws = torch.ones((M, 3), device="cuda"), torch.ones((3, 3), device="cuda")
    xs[1, 2], ws[1, 0] = float("nan"), float("inf")
    Y = g.linear_scaled(X, W, xs, ws)
    assert bool(Y[1].isnan().all()) and bool((Y[0, 128:256] == float("inf")).all())
    assert bool((Y[0, :128] == 384).all()) and bool((Y[0, 256:] == 384).all())


@pytest.mark.parametrize("M,N,K", [(0, 8, 8), (5, 0, 8), (1, 24, 0), (200, 300, 0)])
def test_scaled_and_gated_empty_dimensions(g, M, N, K):
    r = gen(2)
    X = torch.zeros((M, K), dtype=E4M3, device="cuda")
    xs = torch.ones((M, blocks(K)), device="cuda")
    res, bias = matrix(r, M, N, F16), vector(r, 2 * N, F16)
    Y, H = Guarded(M, N, F16), Guarded(M, N, F16)
    g.linear_scaled(X, torch.zeros((N, K), dtype=E4M3, device="cuda"), xs, torch.ones((blocks(N), blocks(K)), device="cuda"),
                    bias[:N], residual=res, out=Y.t)
    y = bias[:N].double() + res.double()
    same(Y.t, y.to(F16).expand(M, N))
    for dtype in (F16, E4M3):
        g.linear_glu(torch.zeros((M, K), dtype=dtype, device="cuda"), torch.zeros((2 * N, K), dtype=dtype, device="cuda"), bias,
                     act="none", out=H.t)
        same(H.t, (bias[:N].double() * bias[N:].double()).to(F16).expand(M, N))
    Y.check(), H.check()


# ------------------------------------------------------------------ gated forward

def gated_operands(r, M, N, K, dtype, ints=False):
    f8 = dtype in (E4M3, E5M2)
    X, W = matrix(r, M, K, dtype, ints=ints), matrix(r, 2 * N, K, dtype, ints=ints, scale=1.0 if f8 else K ** -0.5)
    xs, ws = (scales(r, M, blocks(K), ints), scales(r, 2 * blocks(N), blocks(K), ints)) if f8 else (None, None)
    return X, W, xs, ws


def gated_form(X, W, xs, ws, bias, act, out, alpha):
    z, e = gref.scaled_product(gref.scaled(X, xs, 1), stacked(W, ws), alpha)
    return gref.glu(*gref.with_bias(z, e, bias), act, out)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype,out", [(F16, F16), (BF16, BF16), (E4M3, BF16), (E5M2, F16)])
def test_glu_integers_are_exact(g, M, N, K, dtype, out):
    r = gen(M + N + K)
    for keep in (False, True):
        N = -(-N // 8) * 8 if keep else N
        X, W, xs, ws = gated_operands(r, M, N, K, dtype, ints=True)
        bias = vector(r, 2 * N, F32, ints=True, offset=1)
        z = gref.scaled(X, xs, 1) @ stacked(W, ws).t() + bias.double()
        H, Z = Guarded(M, N, out), Guarded(M, 2 * N, out)
        g.linear_glu(X, W, bias, act="relu", out=H.t, preact=Z.t if keep else None, x_scales=xs, w_scales=ws)
        same(H.t, (z[:, :N].clamp_min(0) * z[:, N:]).to(out), "H")
        if keep:
            same(Z.t, z.to(out), "Z")
        H.check("H"), Z.check("Z")


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ref.ACTS)
def test_glu_against_64_bits(g, M, N, K, act):
    r = gen(7 * M + N + K)
    for dtype, out in ((F16, F16), (BF16, BF16), (E4M3, F16), (E5M2, BF16)):
        alpha = K ** -0.5 if dtype in (E4M3, E5M2) else 1.5
        for bias_dtype, keep in ((F32, False), (out, True), (None, True), (None, False)):
            n = -(-N // 8) * 8 if keep else N
            X, W, xs, ws = gated_operands(r, M, n, K, dtype)
            bias = None if bias_dtype is None else vector(r, 2 * n, bias_dtype, offset=3)
            H, Z = Guarded(M, n, out), Guarded(M, 2 * n, out)
            g.linear_glu(X, W, bias, act=act, out=H.t, preact=Z.t if keep else None, alpha=alpha, x_scales=xs, w_scales=ws)
            h, z = gated_form(X, W, xs, ws, bias, act, out, alpha)
            what = f"{(M, n, K)} {dtype} {act} bias {bias_dtype}"
            gref.assert_within(H.t, h, "H " + what)
            if keep:
                gref.assert_within(Z.t, z, "Z " + what)
            H.check(what), Z.check(what)


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("dtype,out", [(F16, F16), (BF16, BF16)] + TYPES8)
def test_glu_every_tile(g, config, dtype, out):
    g.set_option(native.OPT_CONFIG, config)
    for M, N, K in ((300, 520, 1100), (257, 1000, 300), (700, 301, 4100), (260, 136, 9000)):
        for ctas in (0, 6):
            g.set_option(native.OPT_MAX_CTAS, ctas)
            r = gen(M)
            X, W, xs, ws = gated_operands(r, M, N, K, dtype)
            bias = vector(r, 2 * N, F32)
            H, Z = Guarded(M, N, out), Guarded(M, 2 * N, out)
            g.linear_glu(X, W, bias, act="gelu", out=H.t, preact=Z.t if N % 8 == 0 else None, alpha=0.5, x_scales=xs, w_scales=ws)
            h, z = gated_form(X, W, xs, ws, bias, "gelu", out, 0.5)
            gref.assert_within(H.t, h, f"{(M, N, K)} {ctas} H")
            if N % 8 == 0:
                gref.assert_within(Z.t, z, f"{(M, N, K)} {ctas} Z")
            H.check(), Z.check()


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (5, 2056, 8192), (20, 1000, 2050), (48, 520, 4104), (90, 300, 8192),
                                   (256, 1032, 4100), (600, 136, 5000)])
@pytest.mark.parametrize("dtype,out", [(F16, F16), (BF16, BF16), (E4M3, BF16), (E5M2, F16)])
def test_glu_split_over_a_cluster(g, M, N, K, dtype, out):
    r = gen(M + K)
    X, W, xs, ws = gated_operands(r, M, N, K, dtype)
    bias = vector(r, 2 * N, out, offset=1)
    alpha = K ** -0.5 if dtype in (E4M3, E5M2) else 1.0
    keep = N % 8 == 0
    H, Z = Guarded(M, N, out), Guarded(M, 2 * N, out)
    g.linear_glu(X, W, bias, out=H.t, preact=Z.t if keep else None, alpha=alpha, x_scales=xs, w_scales=ws)
    h, z = gated_form(X, W, xs, ws, bias, "silu", out, alpha)
    gref.assert_within(H.t, h, "H")
    if keep:
        gref.assert_within(Z.t, z, "Z")
    H.check(), Z.check()


# ------------------------------------------------------------------ gated backward

BACK = [(1, 8, 8), (1, 520, 1000), (7, 40, 129), (65, 136, 97), (128, 192, 256), (300, 200, 257), (1003, 128, 77),
        (513, 1032, 520), (260, 304, 2100)]  # M, N (hidden), K (the contraction)


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_glu_dgrad_integers_are_exact(g, M, N, K, dtype):
    r = gen(M + N)
    dY, W, Z = matrix(r, M, K, dtype, ints=True), matrix(r, K, N, dtype, ints=True), matrix(r, M, 2 * N, dtype, ints=True)
    dZ, db = Guarded(M, 2 * N, dtype), Guarded(1, 2 * N, F32, init=torch.ones((1, 2 * N), device="cuda"))
    g.linear_glu_dgrad(dY, W, Z, act="relu", out=dZ.t, dbias=db.t[0], beta_bias=3.0, alpha=2.0)
    d, z = 2 * (dY.double() @ W.double()), Z.double()
    dz = torch.cat([d * z[:, N:] * (z[:, :N] > 0), d * z[:, :N].clamp_min(0)], 1)
    same(dZ.t, dz.to(dtype), "dZ")
    same(db.t[0], (dz.sum(0) + 3).float(), "dbias")
    dZ.check(), db.check()


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_glu_dgrad_against_64_bits(g, M, N, K, act, dtype):
    r = gen(5 * M + N)
    dY, W, Z = matrix(r, M, K, dtype), matrix(r, K, N, dtype, scale=K ** -0.5), matrix(r, M, 2 * N, dtype, scale=2.0)
    for db_dtype, beta in ((F32, 0.0), (dtype, 0.0), (F32, -0.5), (None, 0.0)):
        b0 = vector(r, 2 * N, F32)
        dZ, db = Guarded(M, 2 * N, dtype), None
        if db_dtype is not None:
            db = Guarded(1, 2 * N, db_dtype, init=b0[None] if beta else None)
        g.linear_glu_dgrad(dY, W, Z, act=act, out=dZ.t, dbias=None if db is None else db.t[0], beta_bias=beta, alpha=0.75)
        z, b = gref.glu_dgrad(*ref.product(dY, W, 0.75), Z, act, dtype, db_dtype or F32, b0, beta)
        gref.assert_within(dZ.t, z, f"dZ {act}")
        dZ.check()
        if db is not None:
            gref.assert_within(db.t[0], b, f"dbias {act} {db_dtype} {beta}")
            db.check()


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("sums", [True, False])
def test_glu_dgrad_every_tile(g, config, dtype, sums):
    g.set_option(native.OPT_CONFIG, config)
    for M, N, K in ((300, 520, 1100), (257, 1000, 300), (700, 304, 4100), (2050, 776, 72)):
        for ctas in (0, 6):
            g.set_option(native.OPT_MAX_CTAS, ctas)
            r = gen(M)
            dY, W, Z = matrix(r, M, K, dtype), matrix(r, K, N, dtype, scale=K ** -0.5), matrix(r, M, 2 * N, dtype)
            dZ, db = Guarded(M, 2 * N, dtype), Guarded(1, 2 * N, F32)
            g.linear_glu_dgrad(dY, W, Z, act="gelu", out=dZ.t, dbias=db.t[0] if sums else None)
            z, b = gref.glu_dgrad(*ref.product(dY, W), Z, "gelu", dtype, F32)
            gref.assert_within(dZ.t, z, f"{(M, N, K)} {ctas}")
            dZ.check()
            if sums:
                gref.assert_within(db.t[0], b, f"{(M, N, K)} {ctas}")
                db.check()


@pytest.mark.parametrize("M,N,K", [(0, 24, 8), (5, 0, 8), (70, 200, 0)])
def test_glu_dgrad_empty_dimensions(g, M, N, K):
    r = gen(4)
    dY, W = torch.zeros((M, K), dtype=F16, device="cuda"), torch.zeros((K, N), dtype=F16, device="cuda")
    Z, b0 = matrix(r, M, 2 * N, F16), vector(r, 2 * N, F32)
    dZ, db = Guarded(M, 2 * N, F16), b0.clone()
    g.linear_glu_dgrad(dY, W, Z, out=dZ.t, dbias=db, beta_bias=2.0)
    assert bool((dZ.t == 0).all())
    same(db, b0 * 2)
    g.linear_glu_dgrad(dY, W, Z, out=dZ.t, dbias=db)
    assert bool((db == 0).all())


@pytest.mark.parametrize("M", [40, 130, 700])
def test_glu_dgrad_rows_past_the_end_stay_out_of_the_sums(g, M):
    # An infinite weight times the zeros that fill a ragged tile would be NaN: those rows must not count.
    r = gen(5)
    dY, W = matrix(r, M, 64, BF16).abs(), matrix(r, 64, 200, BF16)
    W[3, 7] = float("inf")
    Z, db = matrix(r, M, 400, BF16).abs() + 1, torch.empty(400, device="cuda")
    dZ = g.linear_glu_dgrad(dY, W, Z, act="relu", dbias=db)
    assert bool((dZ[:, 7] == float("inf")).all()) and db[7].item() == float("inf") and db[207].item() == float("inf")
    others = torch.arange(400, device="cuda") % 200 != 7
    assert bool(db[others].isfinite().all())


def test_glu_special_values(g):
    # Gates at their limits: act and its slope keep theirs, forward and backward, in both kinds of kernel.
    inf, nan = float("inf"), float("nan")
    gate = torch.tensor([inf, -inf, nan, 0.0, 3e4, -3e4, 1.0, -1.0], device="cuda")
    for M in (3, 300):
        Z = torch.cat([gate.expand(M, 8), torch.full((M, 8), 2.0, device="cuda")], 1).half()
        one = torch.ones((M, 8), device="cuda").half()
        for act in ("gelu", "gelu_tanh", "silu"):
            dZ = g.linear_glu_dgrad(one, torch.eye(8, device="cuda").half(), Z, act=act)
            want_g = torch.tensor([2, 0, nan, 1, 2, 0], device="cuda").half().expand(M, 6)
            want_u = torch.tensor([inf, 0, nan, 0, 3e4, 0], device="cuda").half().expand(M, 6)
            same(dZ[:, :6], want_g, act)
            same(dZ[:, 8:14], want_u, act)
            X = torch.zeros((M, 16), device="cuda").half()
            X[:, 0] = 1
            W = torch.zeros((16, 16), device="cuda").half()
            W[:6, 0], W[8:, 0] = gate[:6].half(), 2.0
            W[:, 1:] = 0
            H = g.linear_glu(X, W, act=act)
            same(H[:, 3:6], torch.tensor([0, 6e4, 0], device="cuda").half().expand(M, 3), act)
            assert bool(H[:, 2].isnan().all()), act


def test_glu_gradient_against_differences(g):
    # H's slope along d for G and U: (h(z + t v) - h(z - t v)) / 2t in fp64, from which dZ . v differs by t^2 times third
    # derivatives (under 8 |u| + 12 here) and by dZ's rounding.
    r = gen(11)
    M, N = 90, 136
    for act in ref.ACTS[2:]:
        Z = matrix(r, M, 2 * N, F16, scale=1.5)
        dY, eye = matrix(r, M, N, F16), torch.eye(N, device="cuda").half()
        dZ = g.linear_glu_dgrad(dY, eye, Z, act=act).double()
        z, t = Z.double(), 1e-4
        v = torch.randn(z.shape, generator=r, device="cuda", dtype=torch.float64)

        def h(z):
            return dY.double() * ref.act_value(z[:, :N], act) * z[:, N:]

        want = (h(z + t * v) - h(z - t * v)) / (2 * t)
        got = dZ[:, :N] * v[:, :N] + dZ[:, N:] * v[:, N:]
        mags = dZ[:, :N].abs() * v[:, :N].abs() + dZ[:, N:].abs() * v[:, N:].abs()
        bound = mags * 2.0 ** -11 + 2.0 ** -15 * dY.double().abs() * (z[:, N:].abs() + z[:, :N].abs() + 1) * (v.abs()[:, :N] + v.abs()[:, N:]) + 1e-5
        assert bool(((got - want).abs() <= bound).all()), act


# ------------------------------------------------------------------ 8 bits

@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (2, 127), (7, 129), (33, 1000), (65, 520), (128, 256), (300, 2056),
                                 (1003, 77)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q", [E4M3, E5M2])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize(g, M, K, dtype, q, rows):
    r = gen(M + K)
    X = matrix(r, M, K, dtype)
    X *= torch.exp(3 * torch.randn((M, 1), generator=r, device="cuda")).to(dtype)
    if M > 2:
        X[1] = 0
    out, S = Guarded(M, K, q), torch.full((-(-M // rows) + 1, blocks(K) + 2), 5.0, device="cuda")
    s = S[:-1, :-2]
    g.quantize(X, block_rows=rows, out=out.t, scales=s)
    want_q, want_s = gref.quantize(X, rows, q)
    same(s.clone(), want_s, "scales")
    same(out.t.float(), want_q.float(), "values")
    out.check()
    assert bool((S[-1] == 5).all()) and bool((S[:, -2:] == 5).all())
    # What the values stand for is within half a step of X: 2^-4 or 2^-3 of the value, or of the smallest step (2^-10 or
    # 2^-17 times the scale), and the two fp32 roundings of x r.
    step, tiny = (2.0 ** -4, 2.0 ** -10) if q is E4M3 else (2.0 ** -3, 2.0 ** -17)
    err = (gref.scaled(out.t, s, rows) - X.double()).abs()
    assert bool((err <= (step + 2.0 ** -20) * X.double().abs() + tiny * gref.spread(s, rows, M, K)).all())
    new_q, new_s = g.quantize(X, rows, q)
    same(new_q.float(), want_q.float()), same(new_s, want_s)


@pytest.mark.parametrize("M,K", [(1100, 5000), (20000, 264), (9800, 512), (3, 160000), (70, 80001), (2432, 8192)])
def test_quantize_many_boxes(g, M, K):
    # More boxes of 32 x 256 than blocks run at once: a block's boxes lie on one strip of columns, or wander over them.
    r = gen(M + K)
    X = matrix(r, M, K, BF16)
    want_q, want_s = gref.quantize(X, 1, E4M3)
    out, S = Guarded(M, K, E4M3), torch.full((M + 1, want_s.shape[1] + 2), 5.0, device="cuda")
    g.quantize(X, 1, out=out.t, scales=S[:M, :want_s.shape[1]])
    same(S[:M, :want_s.shape[1]], want_s, "scales")
    same(out.t.float(), want_q.float(), "values")
    out.check()
    assert bool((S[-1] == 5).all()) and bool((S[:, -2:] == 5).all())


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("q", [E4M3, E5M2])
def test_quantize_special_values(g, rows, q):
    X = torch.ones((rows * 2, 512), device="cuda", dtype=BF16)
    X[0, 0], X[0, 130], X[0, 260] = float("nan"), float("-inf"), 2.0 ** -133
    X[:rows, 256:260], X[:rows, 261:384] = 0, 0
    X[:rows, 384:] = 3e38
    Q, S = g.quantize(X, rows, q)
    values = Q.float()
    # Beside a NaN everything is NaN; beside an infinity (1 / s = 0) finite values are 0, which stands for 0 times infinity.
    assert bool(values[:rows, :128].isnan().all()) and bool(S[0, 0].isnan()) and S[0, 1].item() == float("inf")
    assert bool(values[0, 130].isnan()) and values[:rows, 128:256].nan_to_num(0).abs().sum().item() == 0
    assert bool(gref.scaled(Q, S, rows)[:rows, :256].isnan().all())
    # (A block of 128 rows has ones in column 260 below the tiny one.)
    largest = torch.tensor(2.0 ** -126 if rows == 1 else 1 / torch.finfo(q).max).float()
    assert S[0, 2].item() == largest.item() and values[0, 256].item() == 0
    Q, S = g.quantize(torch.full((rows, 128), 2.0 ** -133, device="cuda", dtype=BF16), rows, q)
    assert S[0, 0].item() == 2.0 ** -126 and bool((Q.float() == torch.tensor(2.0 ** -7).to(q).float().item()).all())
    assert bool((values[:rows, 384:] == torch.finfo(q).max).all())
    assert bool((values[rows:] == torch.finfo(q).max).all())


# ------------------------------------------------------------------ layer norm

NORMS = [(1, 1), (3, 7), (1, 4096), (33, 64), (65, 1000), (9, 257), (40, 512), (70, 513), (12, 1024), (5, 2047), (300, 2056),
         (31, 4100), (610, 8192), (4, 9001), (6, 16384), (7, 16392), (40, 20001), (1003, 40)]


@pytest.mark.parametrize("M,N", NORMS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_layer_norm(g, M, N, dtype):
    r = gen(M + N)
    for w_dtype, b_dtype, offset in ((F32, F32, 0), (dtype, dtype, 1), (None, F32, 3), (F32, None, 2), (None, None, 0)):
        X = matrix(r, M, N, dtype, scale=2.0)
        X += torch.randn((M, 1), generator=r, device="cuda").to(dtype)
        w = None if w_dtype is None else vector(r, N, w_dtype, offset=offset)
        b = None if b_dtype is None else vector(r, N, b_dtype, offset=offset)
        Y, mean, rstd = Guarded(M, N, dtype), vector(r, M, F32, offset=1), vector(r, M, F32, offset=1)
        g.layer_norm(X, w, b, eps=1e-3, out=Y.t, mean=mean, rstd=rstd)
        y, m, s = gref.layer_norm(X, w, b, 1e-3, dtype)
        gref.assert_within(Y.t, y, f"Y {w_dtype}")
        gref.assert_within(mean, m, "mean")
        gref.assert_within(rstd, s, "rstd")
        Y.check()
    buf = Guarded(M, N, dtype, init=X)
    g.layer_norm(buf.t, w, b, eps=1e-3, out=buf.t)
    same(buf.t, g.layer_norm(X, w, b, eps=1e-3), "in place")
    buf.check()


@pytest.mark.parametrize("M,N", [(1300, 7936), (611, 8000), (9800, 200), (5000, 768), (2600, 1024), (650, 5120), (611, 10240),
                                 (460, 12296)])
def test_layer_norm_rows_ahead(g, M, N):
    # Every warp takes several rows, one to three of them in flight.
    r = gen(M + N)
    X, w, b = matrix(r, M, N, BF16), vector(r, N, F32), vector(r, N, F32)
    Y = Guarded(M, N, BF16)
    g.layer_norm(X, w, b, eps=1e-3, out=Y.t)
    gref.assert_within(Y.t, gref.layer_norm(X, w, b, 1e-3, BF16)[0], "Y")
    Y.check()
    buf = Guarded(M, N, BF16, init=X)
    g.layer_norm(buf.t, w, b, eps=1e-3, out=buf.t)
    same(buf.t, Y.t, "in place")


def test_layer_norm_of_a_large_mean(g):
    # Values 1000 apart from zero, spread of 1: the statistics do not cancel.
    r = gen(1)
    X = (torch.randn((50, 4096), generator=r, device="cuda") + 1000).half()
    y, m, s = gref.layer_norm(X, None, None, 0.0, F16)
    rstd = torch.empty(50, device="cuda")
    gref.assert_within(g.layer_norm(X, eps=0.0, rstd=rstd), y)
    assert float(((rstd.double() - s[0]) / s[0]).abs().max()) < 1e-3


def test_layer_norm_special_rows(g):
    # A NaN or infinity reaches its own row alone; a constant row gives the bias.
    r = gen(2)
    for N in (64, 500, 3000, 20000):
        X, b = matrix(r, 6, N, F16), vector(r, N, F32)
        X[1, 3], X[3, N - 1], X[4] = float("nan"), float("inf"), 7.0
        Y = g.layer_norm(X, None, b)
        assert bool(Y[1].isnan().all()) and bool(Y[3].isnan().all())
        assert bool(Y[[0, 2, 5]].isfinite().all())
        same(Y[4], b.half())


@pytest.mark.parametrize("N", [8, 200, 1024, 3000, 8192, 9000, 20000])
def test_layer_norm_beyond_the_range_of_its_sums(g, N):
    # Finite values whose squares' sum is over fp32's range: v is infinite, so rstd is 0 and Y the bias; a sum that is infinite
    # is the mean.  The rows beside them keep their values.
    r = gen(8)
    X, b = matrix(r, 5, N, BF16), vector(r, N, F32)
    want = g.layer_norm(X, None, b)
    X[1] *= 1e25
    X[3, N // 2] = float("-inf")
    mean, rstd = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    Y = g.layer_norm(X, None, b, mean=mean, rstd=rstd)
    same(Y[1], b.to(BF16))
    assert rstd[1].item() == 0 and bool(mean[1].isfinite())
    assert mean[3].item() == float("-inf") and bool(Y[3].isnan().all()) and bool(rstd[3].isnan())
    same(Y[[0, 2, 4]], want[[0, 2, 4]])


@pytest.mark.parametrize("M,N", NORMS + [(700, 200), (2500, 72)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_layer_norm_grad(g, M, N, dtype):
    r = gen(M + 3 * N)
    X = matrix(r, M, N, dtype, scale=2.0)
    X += torch.randn((M, 1), generator=r, device="cuda").to(dtype)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    g.layer_norm(X, eps=1e-2, mean=mean, rstd=rstd)
    for w_dtype, with_res, dw_dtype, db_dtype, beta in ((F32, True, F32, F32, 0.0), (dtype, False, dtype, F32, 0.5),
                                                        (None, True, None, dtype, 0.0), (F32, False, F32, None, -1.0),
                                                        (F32, True, None, None, 0.0)):
        dY = matrix(r, M, N, dtype)
        w = None if w_dtype is None else vector(r, N, w_dtype, offset=1)
        res = matrix(r, M, N, dtype, pad=2) if with_res else None
        dw0, db0 = vector(r, N, dw_dtype or F32), vector(r, N, db_dtype or F32)
        dX = Guarded(M, N, dtype)
        dw = None if dw_dtype is None else Guarded(1, N, dw_dtype, init=dw0[None] if beta else None)
        db = None if db_dtype is None else Guarded(1, N, db_dtype, init=db0[None] if beta else None)
        g.layer_norm_grad(dY, X, mean, rstd, w, residual=res, out=dX.t, dweight=None if dw is None else dw.t[0],
                          dbias=None if db is None else db.t[0], beta=beta)
        x, a, b = gref.layer_norm_grad(dY, X, mean, rstd, w, res, dtype, (dw_dtype or F32, db_dtype or F32), beta, dw0, db0)
        gref.assert_within(dX.t, x, f"dX {w_dtype} {with_res}")
        dX.check()
        if dw is not None:
            gref.assert_within(dw.t[0], a, "dw")
            dw.check()
        if db is not None:
            gref.assert_within(db.t[0], b, "db")
            db.check()
    for source in ("dY", "residual"):
        buf = Guarded(M, N, dtype, init=dY if source == "dY" else res)
        g.layer_norm_grad(buf.t if source == "dY" else dY, X, mean, rstd, w, residual=res if source == "dY" else buf.t, out=buf.t)
        same(buf.t, g.layer_norm_grad(dY, X, mean, rstd, w, residual=res), "in place of " + source)
        buf.check()


# Lengths of every shape of the kernel, ragged and full, with rows enough that a group of warps takes four or more (on 152 SMs), and
# not the same number in every group.
GRAD_LOOPS = [(9800, 200), (9900, 256), (9801, 500), (9901, 512), (5003, 1000), (5001, 1024), (2605, 2000), (2603, 2048), (1301, 3000),
              (1303, 4096), (801, 5000), (803, 8192)]


@pytest.mark.parametrize("M,N", GRAD_LOOPS)
def test_layer_norm_grad_rows_ahead(g, M, N):
    # The places of the rows in flight are filled again and again, their statistics fetched a row ahead.
    r = gen(M + N)
    for dtype, with_res in ((BF16, True), (F16, False)):
        X = matrix(r, M, N, dtype, scale=2.0)
        X += torch.randn((M, 1), generator=r, device="cuda").to(dtype)
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        g.layer_norm(X, eps=1e-2, mean=mean, rstd=rstd)
        dY, w, res = matrix(r, M, N, dtype), vector(r, N, F32), matrix(r, M, N, dtype, pad=2) if with_res else None
        dX, dw, db = Guarded(M, N, dtype), Guarded(1, N, F32), Guarded(1, N, F32)
        g.layer_norm_grad(dY, X, mean, rstd, w, residual=res, out=dX.t, dweight=dw.t[0], dbias=db.t[0])
        x, a, b = gref.layer_norm_grad(dY, X, mean, rstd, w, res, dtype, (F32, F32))
        gref.assert_within(dX.t, x, "dX"), gref.assert_within(dw.t[0], a, "dw"), gref.assert_within(db.t[0], b, "db")
        dX.check(), dw.check(), db.check()
        for source in ("dY", "residual") if with_res else ("dY",):
            buf = Guarded(M, N, dtype, init=dY if source == "dY" else res)
            g.layer_norm_grad(buf.t if source == "dY" else dY, X, mean, rstd, w, residual=res if source == "dY" else buf.t, out=buf.t)
            same(buf.t, dX.t, "in place of " + source)
            buf.check()


@pytest.mark.parametrize("M,N", [(6, 64), (700, 500), (400, 3000), (320, 8192), (9, 9000)])
def test_layer_norm_grad_special_rows(g, M, N):
    # A NaN or infinity of X or dY reaches its own row of dX alone (and the sums of its columns); where rstd is 0, since the
    # squares' sum was over fp32's range, x^ is 0: dX is the residual, and nothing comes to dw.
    r = gen(9)
    dY, X, res, w = matrix(r, M, N, BF16), matrix(r, M, N, BF16), matrix(r, M, N, BF16), vector(r, N, F32)
    stats = torch.empty((2, M), device="cuda")

    def grad(dY, X):
        g.layer_norm(X, mean=stats[0], rstd=stats[1])
        dw, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        return g.layer_norm_grad(dY, X, stats[0], stats[1], w, residual=res, dweight=dw, dbias=db), dw, db

    want, _, db = grad(dY, X)
    huge = Guarded(M, N, BF16, init=X).t
    huge[2] = torch.where(torch.arange(N, device="cuda") % 4 < 2, 2e38, -2e38).to(BF16)  # (its sum stays in range)
    zeroed = Guarded(M, N, BF16, init=dY).t
    zeroed[2] = 0
    dX, dw, db_huge = grad(dY, huge)
    assert stats[1, 2].item() == 0
    same(dX[2], res[2], "rstd of 0")
    same(db_huge, db, "db")
    others = torch.arange(M, device="cuda") != 2
    same(dX[others], want[others], "beside it")
    same(dw, grad(zeroed, X)[1], "dw without the row")
    X[1, 3], X[4, N - 1], dY[3, N // 2] = float("nan"), float("inf"), float("inf")
    dX, _, db = grad(dY, X)
    others[[1, 3, 4]] = False
    others[2] = True
    same(dX[others], want[others], "beside NaN and infinities")
    assert bool(dX[[1, 4]].isnan().all()) and bool((~dX[3].isfinite()).any())
    assert db[N // 2].item() == float("inf") and bool(db[torch.arange(N, device="cuda") != N // 2].isfinite().all())


@pytest.mark.parametrize("N", [100, 500, 3001, 9001])
def test_layer_norm_grad_of_a_constant_row_far_from_zero(g, N):
    # X - mean is 0; past a ragged row's end it is -mean, and that times rstd is over fp32's range: it must not count.
    r = gen(10)
    dY, X, w = matrix(r, 5, N, BF16), matrix(r, 5, N, BF16), vector(r, N, F32)
    X[1] = 3e34
    mean, rstd = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    g.layer_norm(X, eps=1e-12, mean=mean, rstd=rstd)
    same(mean[1].double(), X[1, 0].double())
    assert (mean[1] * rstd[1]).item() == float("inf")
    dw, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    dX = g.layer_norm_grad(dY, X, mean, rstd, w, dweight=dw, dbias=db)
    x, a, b = gref.layer_norm_grad(dY, X, mean, rstd, w, None, BF16, (F32, F32))
    gref.assert_within(dX, x, "dX"), gref.assert_within(dw, a, "dw"), gref.assert_within(db, b, "db")


def test_layer_norm_grad_against_differences(g):
    # L = sum(C * norm(x) w + b) along a direction of x, w and b, by central differences in fp64; dX is rounded to fp16
    # (2^-11 of each term), the differences are off by h^2 times third derivatives (under 100 in sum here).
    r = gen(12)
    M, N, h = 20, 200, 1e-4
    X, C, w, b = matrix(r, M, N, F16), matrix(r, M, N, F16), vector(r, N, F32), vector(r, N, F32)
    mean, rstd, dw, db = (torch.empty(n, device="cuda") for n in (M, M, N, N))
    g.layer_norm(X, w, b, mean=mean, rstd=rstd)
    dX = g.layer_norm_grad(C, X, mean, rstd, w, dweight=dw, dbias=db)

    def loss(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return (C.double() * (c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w + b)).sum()

    at = [X.double(), w.double(), b.double()]
    for i, grad in enumerate((dX, dw, db)):
        for _ in range(4):
            v = torch.randn(grad.shape, generator=r, device="cuda", dtype=torch.float64)
            plus, minus = list(at), list(at)
            plus[i], minus[i] = at[i] + h * v, at[i] - h * v
            want = ((loss(*plus) - loss(*minus)) / (2 * h)).item()
            terms = grad.double() * v
            assert abs(terms.sum().item() - want) <= 2.0 ** -11 * terms.abs().sum().item() + 1e-4, i


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_layer_norm_grad_of_one_column(g, dtype):
    # The norm of one column is its bias, whatever X: nothing but the residual reaches dX, however large rstd is.
    r = gen(5)
    dY, X, res, w = matrix(r, 50, 1, dtype), matrix(r, 50, 1, dtype), matrix(r, 50, 1, dtype), vector(r, 1, F32)
    mean, rstd = torch.empty(50, device="cuda"), torch.empty(50, device="cuda")
    g.layer_norm(X, w, eps=1e-5, mean=mean, rstd=rstd)
    assert bool((rstd > 300).all())
    same(g.layer_norm_grad(dY, X, mean, rstd, w, residual=res), res)
    assert bool((g.layer_norm_grad(dY, X, mean, rstd, w) == 0).all())


def test_layer_norm_grad_no_rows(g):
    dw, db = torch.ones(24, device="cuda"), torch.full((24,), 2.0, device="cuda")
    none = torch.zeros((0, 24), dtype=F16, device="cuda")
    stat = torch.zeros(0, device="cuda")
    g.layer_norm_grad(none, none, stat, stat, dweight=dw, dbias=db, beta=0.5)
    assert bool((dw == 0.5).all()) and bool((db == 1).all())
    g.layer_norm_grad(none, none, stat, stat, dbias=db)
    assert bool((dw == 0.5).all()) and bool((db == 0).all())
    assert g.layer_norm(none).shape == (0, 24)
    g.layer_norm(torch.zeros((3, 0), dtype=F16, device="cuda"))


# ------------------------------------------------------------------ a block of them together

class Block:
    """y = x + down(act(gate(n)) * up(n)), n = norm(x): weights, and its passes by a handle's calls."""

    def __init__(self, r, M, D, F, act="silu"):
        self.act, self.F = act, F
        self.x, self.dy = matrix(r, M, D, BF16), matrix(r, M, D, BF16)
        self.w, self.b = vector(r, D, F32), vector(r, D, F32)
        self.W, self.bias = matrix(r, 2 * F, D, BF16, scale=D ** -0.5), vector(r, 2 * F, F32)
        self.V = matrix(r, D, F, BF16, scale=F ** -0.5)
        e = lambda *s, t=F32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.mean, self.rstd, self.Z = e(M), e(M), e(M, 2 * F, t=BF16)
        self.dbias, self.dw, self.db = e(2 * F), e(D), e(D)

    def train(self, g, stream=None):
        s = {"stream": stream}
        n = g.layer_norm(self.x, self.w, self.b, mean=self.mean, rstd=self.rstd, **s)
        H = g.linear_glu(n, self.W, self.bias, act=self.act, preact=self.Z, **s)
        y = g.linear(H, self.V, residual=self.x, **s)
        dV = g.linear_wgrad(self.dy, H, **s)
        dZ = g.linear_glu_dgrad(self.dy, self.V, self.Z, act=self.act, dbias=self.dbias, **s)
        dW, dn = g.linear_wgrad(dZ, n, **s), g.linear_dgrad(dZ, self.W, **s)
        dx = g.layer_norm_grad(dn, self.x, self.mean, self.rstd, self.w, residual=self.dy, dweight=self.dw, dbias=self.db, **s)
        return {"y": y, "dV": dV, "dW": dW, "dbias": self.dbias, "dx": dx, "dw": self.dw, "db": self.db}

    def exact(self):
        names = ("x", "w", "b", "W", "bias", "V")
        t = {n: getattr(self, n).double().requires_grad_(True) for n in names}
        c = t["x"] - t["x"].mean(1, keepdim=True)
        n = c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * t["w"] + t["b"]
        z = n @ t["W"].t() + t["bias"]
        y = t["x"] + (ref.act_value(z[:, :self.F], self.act) * z[:, self.F:]) @ t["V"].t()
        grads = torch.autograd.grad((y * self.dy.double()).sum(), [t[n] for n in names])
        return {"y": y.detach(), **dict(zip(("dx", "dw", "db", "dW", "dbias", "dV"), grads))}


@pytest.mark.parametrize("M,D,F", [(1, 64, 128), (40, 136, 264), (300, 520, 1000), (1500, 256, 704)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_block_trained(g, M, D, F, act):
    # Each value passes up to five roundings to bf16 (n, Z or H, dZ, dn, the result), 2^-9 of a value on average each: in norm
    # the gradients stay within 5 x 2^-8 of autograd's in fp64.
    block = Block(gen(M + D), M, D, F, act)
    got, want = block.train(g), block.exact()
    for name, v in got.items():
        err = (v.double() - want[name]).norm() / want[name].norm().clamp_min(1e-6)
        assert err.item() < 5 * 2.0 ** -8, (name, err.item())


@pytest.mark.parametrize("M,D,F", [(1, 512, 1024), (33, 1024, 2056), (300, 640, 1000)])
def test_block_served_in_8_bits(g, M, D, F):
    # norm, 8 bits, gated layer, 8 bits, layer with the residual: every step against its plain form on the step's own inputs.
    r = gen(M)
    x, w = matrix(r, M, D, BF16), vector(r, D, F32)
    halves = [matrix(r, F, D, BF16, scale=D ** -0.5) for _ in range(2)]
    parts = [g.quantize(h, 128) for h in halves]
    W, ws = torch.cat([q for q, _ in parts]), torch.cat([s for _, s in parts])
    if F % 128 == 0:  # stacked first, quantized at once: the same blocks
        q, s = g.quantize(torch.cat(halves), 128)
        same(q.float(), W.float()), same(s, ws)
    V, vs = g.quantize(matrix(r, D, F, BF16, scale=F ** -0.5), 128)
    n8, ns = g.quantize(g.layer_norm(x, w))
    H = g.linear_glu(n8, W, x_scales=ns, w_scales=ws)
    h, _ = gated_form(n8, W, ns, ws, None, "silu", BF16, 1.0)
    gref.assert_within(H, h, "H")
    h8, hs = g.quantize(H)
    y = g.linear_scaled(h8, V, hs, vs, residual=x)
    z, e = gref.scaled_product(gref.scaled(h8, hs, 1), gref.scaled(V, vs, 128))
    want = z + x.double()
    gref.assert_within(y, (want, ref.rounded(e + 2 * ref.U * (want.abs() + x.double().abs()), want, BF16)), "y")


# ------------------------------------------------------------------ streams, graphs, threads, determinism

def clones(d):
    return {k: v.clone() for k, v in d.items()}


@pytest.mark.parametrize("M,D,F", [(8, 512, 1024), (700, 520, 1000)])
def test_block_same_bits_on_a_stream_in_a_graph_and_again(g, M, D, F):
    block = Block(gen(3), M, D, F)
    first = clones(block.train(g))
    for _ in range(3):
        for k, v in block.train(g).items():
            same(v, first[k], k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on_stream = block.train(g, stream=s)
    s.synchronize()
    for k, v in on_stream.items():
        same(v, first[k], "stream " + k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = block.train(g)
    other = Block(gen(4), M, D, F)
    for name in ("x", "dy", "w", "W", "V"):
        getattr(block, name).copy_(getattr(other, name))
    graph.replay()
    torch.cuda.synchronize()
    replayed = clones(captured)
    for k, v in block.train(g).items():
        same(replayed[k], v, "graph " + k)


def test_serving_calls_captured(g):
    r = gen(5)
    x, W, V = matrix(r, 5, 512, BF16), g.quantize(matrix(r, 2048, 512, BF16), 128), g.quantize(matrix(r, 512, 1024, BF16), 128)

    def step():
        n8, ns = g.quantize(g.layer_norm(x))
        h8, hs = g.quantize(g.linear_glu(n8, W[0], x_scales=ns, w_scales=W[1]))
        return g.linear_scaled(h8, V[0], hs, V[1], residual=x)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    x.copy_(matrix(r, 5, 512, BF16))
    graph.replay()
    torch.cuda.synchronize()
    got = y.clone()
    same(got, step())


def test_module_functions_from_two_threads_on_two_streams():
    blocks_ = [Block(gen(20 + i), 300, 520, 1000) for i in range(2)]
    want = [clones(b.train(native)) for b in blocks_]
    torch.cuda.synchronize()
    failures = []

    def work(i):
        s = torch.cuda.Stream()
        try:
            for _ in range(10):
                with torch.cuda.stream(s):
                    got = blocks_[i].train(native)
                    s.synchronize()
                    for k, v in got.items():
                        if not torch.equal(v, want[i][k]):
                            failures.append((i, k))
        except Exception as e:  # noqa: BLE001
            failures.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads], [t.join() for t in threads]
    assert failures == []


def test_wide_layers_pass_32_bit_offsets(g):
    # 150000 rows of Z hold over 2^31 elements; rows at both ends and in between are checked, and the sums.
    M, N, K = 150000, 8192, 64
    r = gen(30)
    X, W = matrix(r, M, K, BF16, pad=0), matrix(r, 2 * N, K, BF16, scale=K ** -0.5, pad=0)
    Z = torch.empty((M, 2 * N), dtype=BF16, device="cuda")
    H = g.linear_glu(X, W, preact=Z)
    rows = torch.tensor([0, 1, 70000, 131071, 131072, 149998, 149999], device="cuda")
    h, z = gated_form(X[rows], W, None, None, None, "silu", BF16, 1.0)
    gref.assert_within(H[rows], h, "H")
    gref.assert_within(Z[rows], z, "Z")
    dY, V = matrix(r, M, K, BF16, pad=0), matrix(r, K, N, BF16, scale=K ** -0.5, pad=0)
    dZ, db = torch.empty_like(Z), torch.empty(2 * N, device="cuda")
    del H
    g.linear_glu_dgrad(dY, V, Z, out=dZ, dbias=db)
    d, _ = gref.glu_dgrad(*ref.product(dY[rows], V), Z[rows], "silu", BF16, F32)
    gref.assert_within(dZ[rows], d, "dZ")
    part = dZ[:, ::1024].double().sum(0)
    assert bool(((db[::1024].double() - part).abs() <= 2.0 ** -9 * dZ[:, ::1024].double().abs().sum(0)).all())
    w, mean, rstd = vector(r, 2 * N, F32), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    Y = g.layer_norm(Z, w, out=dZ, mean=mean, rstd=rstd)
    gref.assert_within(Y[rows], gref.layer_norm(Z[rows], w, None, 1e-5, BF16)[0], "norm")
    Q, S = g.quantize(Z)
    want = gref.quantize(Z[rows], 1, E4M3)
    same(Q[rows].float(), want[0].float()), same(S[rows], want[1])


# ------------------------------------------------------------------ refusals and the watchdog

def test_refusals(g):
    r = gen(40)
    x, w8, x8 = matrix(r, 8, 64, BF16, pad=0), matrix(r, 32, 64, E4M3, pad=0), matrix(r, 8, 64, E4M3, pad=0)
    W, Z, V = matrix(r, 32, 64, BF16, pad=0), matrix(r, 8, 32, BF16, pad=0), matrix(r, 64, 16, BF16, pad=0)
    one, s = torch.ones((8, 1), device="cuda"), torch.ones((1, 1), device="cuda")
    stat = torch.ones(8, device="cuda")
    bad = [
        lambda: g.linear_glu(x, W[:31]),                                     # an odd number of rows
        lambda: g.linear_glu(x, W, x_scales=one),                            # scales of 16-bit operands
        lambda: g.linear_glu(x, W.half()),
        lambda: g.linear_glu(x, W, act="swish"),
        lambda: g.linear_glu(x, W, bias=stat),
        lambda: g.linear_glu(x, W, out_dtype=F16),
        lambda: g.linear_glu(x8, w8, x_scales=one, w_scales=s),              # w_scales of one half
        lambda: g.linear_glu(x8, w8, x_scales=one.half()),
        lambda: g.linear_glu(x8, w8, x_scales=one.cpu()),
        lambda: g.linear_glu(x, W, preact=Z[:, :16]),
        lambda: g.linear_glu(x, matrix(r, 24, 64, BF16), preact=matrix(r, 8, 24, BF16)),  # N = 12: U's rows off 16 bytes
        lambda: g.linear_glu_dgrad(x, V, Z[:, :16]),
        lambda: g.linear_glu_dgrad(x, V, Z.half()),
        lambda: g.linear_glu_dgrad(x, matrix(r, 64, 12, BF16), matrix(r, 8, 24, BF16)),
        lambda: g.linear_glu_dgrad(x, V, Z, dbias=torch.ones(16, device="cuda")),
        lambda: g.linear_scaled(x, W, None, None),                           # 16-bit operands
        lambda: g.linear_scaled(x8, w8, one[:7], s),
        lambda: g.linear_scaled(x8, w8, one, torch.ones((2, 1), device="cuda")),
        lambda: g.linear_scaled(x8, w8.view(E5M2), one, s),
        lambda: g.linear_scaled(x8, w8, one, s, alpha=float("nan")),
        lambda: g.quantize(x8),
        lambda: g.quantize(x, block_rows=64),
        lambda: g.quantize(x, dtype=F16),
        lambda: g.quantize(x, scales=torch.ones((8, 2), device="cuda")),
        lambda: g.quantize(x[:, 1:]),                                        # a base off 16 bytes
        lambda: g.layer_norm(x.float()),
        lambda: g.layer_norm(x, eps=-1.0),
        lambda: g.layer_norm(x, eps=float("inf")),
        lambda: g.layer_norm(x, weight=stat),
        lambda: g.layer_norm(x, mean=stat[:7]),
        lambda: g.layer_norm(x, rstd=stat.double()),
        lambda: g.layer_norm(x.t()),
        lambda: g.layer_norm_grad(x, x[:7], stat, stat),
        lambda: g.layer_norm_grad(x, x, stat, stat, dweight=stat),
        lambda: g.layer_norm_grad(x, x, stat, stat, beta=float("nan")),
        lambda: g.layer_norm_grad(x, x, stat.half(), stat),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, native.GemmError)):
            call()
            raise AssertionError(f"call {i} was taken")
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["glu", "glu_cluster", "glu_8", "glu_8_cluster", "scaled", "scaled_cluster", "dgrad",
                                  "dgrad_cluster"])
def test_watchdog(g, kind):
    # A stage that never arrives: the launch is given up, reported, and the next one works.
    r = gen(41)
    M = 8 if "cluster" in kind else 600
    x, W = matrix(r, M, 512, BF16, ints=True), matrix(r, 1024, 512, BF16, ints=True)
    x8, w8 = matrix(r, M, 512, E4M3, ints=True), matrix(r, 1024, 512, E4M3, ints=True)
    Z, V = matrix(r, M, 1024, BF16, ints=True), matrix(r, 512, 512, BF16, ints=True)
    call = {"glu": lambda: g.linear_glu(x, W, act="relu"), "glu_8": lambda: g.linear_glu(x8, w8, act="relu"),
            "scaled": lambda: g.linear_scaled(x8, w8, None, None),
            "dgrad": lambda: g.linear_glu_dgrad(x, V, Z, act="relu", dbias=torch.empty(1024, device="cuda"))}[kind.split("_cluster")[0]]
    want = call().clone()
    assert g.sync_status() == native.OK
    g.set_option(native.OPT_TIMEOUT_NS, 20_000_000)
    g.set_option(native.OPT_FAULT_INJECT, 1)
    try:
        call()
        assert g.sync_status() == native.ERR_TIMEOUT
        assert g.error_info()[0] == 1
    finally:
        g.set_option(native.OPT_FAULT_INJECT, 0)
        g.set_option(native.OPT_TIMEOUT_NS, 2_000_000_000)
    same(call(), want)


def test_raw_calls_check_pointers_and_pitches(g):
    # What the binding cannot pass: null and misaligned pointers, small pitches and workspaces, unknown types.
    so, buf = native.load(), torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = buf.data_ptr()

    def glu(**k):
        a = dict(X=p, W=p, H=p, M=8, N=16, K=64, ldx=64, ldw=64, ldh=16, ldz=32, dtype=1, out_dtype=1, act=4, alpha=1.0)
        a.update(k)
        return so.gemm_run_linear_glu(g._h, ctypes.byref(native.gemm_glu_args_t(**a)), None)

    def norm_grad(**k):
        a = dict(dY=p, X=p, mean=p, rstd=p, dX=p, M=8, N=64, lddy=64, ldx=64, lddx=64, dtype=1)
        a.update(k)
        return so.gemm_run_layer_norm_grad(g._h, ctypes.byref(native.gemm_layer_norm_grad_args_t(**a)), None)

    def quantize(**k):
        a = dict(X=p, Q=p, scales=p, M=8, K=64, ldx=64, ldq=64, lds=1, dtype=1, q_dtype=2, block_rows=1)
        a.update(k)
        return so.gemm_run_quantize(g._h, ctypes.byref(native.gemm_quantize_args_t(**a)), None)

    inv, uns = native.ERR_INVALID_ARG, native.ERR_UNSUPPORTED
    assert glu(X=None) == inv and glu(H=None) == inv and glu(ldw=63) == inv and glu(W=p + 2) == uns and glu(ldh=20) == uns
    assert glu(dtype=7) == inv and glu(act=9) == inv and glu(alpha=float("inf")) == inv and glu(N=-1) == inv
    assert glu(Z=p, ldz=16) == inv and glu(Z=p, N=12, ldz=24) == uns and glu(x_scales=p) == inv
    assert glu(dtype=2, K=256, ldx=256, ldw=256, x_scales=p, ld_xs=1) == inv and glu(dtype=2, x_scales=p + 2, ld_xs=1) == uns
    assert glu(N=1 << 30, ldh=1 << 30) == uns
    assert norm_grad(mean=None) == inv and norm_grad(dX=None) == inv and norm_grad(dweight=p, dweight_dtype=0) == inv
    assert norm_grad(dweight=p, dweight_dtype=4, workspace=p, workspace_bytes=64) == inv
    assert norm_grad(dweight=p, dweight_dtype=4, M=304, N=4096, lddy=4096, ldx=4096, lddx=4096) == inv  # no workspace
    assert norm_grad(residual=p, ldr=60) == inv and norm_grad(rstd=p + 1) == uns
    assert quantize(scales=None) == inv and quantize(lds=0) == inv and quantize(block_rows=2) == inv and quantize(q_dtype=1) == inv
    assert quantize(Q=p + 8) == uns and quantize(ldq=72) == uns and quantize(scales=p + 2) == uns
