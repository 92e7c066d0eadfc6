"""The linear-layer operators on the GPU against plain 64-bit forms: sizes from one element to several tiles, ragged
edges, padded and strided rows, empty dimensions, every activation and type, in-place forms, streams, graphs, refusals.

On integer data with act none or relu every sum is exact, so results must match bit for bit; elsewhere they must lie
within the bounds that linear_reference derives.  Inputs sit in NaN-padded rows, outputs in sentinel-filled buffers:
reading or writing outside a matrix shows.
"""
import ctypes

import pytest
import torch

import linear_reference as ref
from dense_tiled_gemm_04_gb300 import native

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
SENTINEL = 0x77
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


def gen(seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    return r


def pitch(cols, dtype, pad=0):
    e = 16 // torch.empty(0, dtype=dtype).element_size()
    return (max(-(-cols // e), 1) + pad) * e


def matrix(r, rows, cols, dtype, ints=False, scale=1.0, pad=1):
    """A rows x cols matrix in NaN-padded rows."""
    x = torch.randint(-2, 3, (rows, cols), generator=r, device="cuda").float() if ints else \
        torch.randn((rows, cols), generator=r, device="cuda") * scale
    buf = torch.full((rows + 1, pitch(cols, dtype, pad)), float("nan"), device="cuda").to(dtype)
    buf[:rows, :cols] = x.to(dtype)
    return buf[:rows, :cols]


def vector(r, n, dtype, ints=False, offset=0):
    """n values that start `offset` elements into a buffer (any alignment of the type)."""
    buf = torch.full((n + offset + 1,), float("nan"), device="cuda", dtype=dtype)
    buf[offset:offset + n] = torch.randint(-3, 4, (n,), generator=r, device="cuda").to(dtype) if ints else \
        torch.randn(n, generator=r, device="cuda").to(dtype)
    return buf[offset:offset + n]


class Guarded:
    """An output window in a buffer of sentinel bytes."""

    def __init__(self, rows, cols, dtype, init=None, pad=1):
        e = torch.empty(0, dtype=dtype).element_size()
        self.bytes = torch.full((rows + 2, pitch(cols, dtype, pad) * e), SENTINEL, dtype=torch.uint8, device="cuda")
        self.t = self.bytes.view(dtype)[:rows, :cols]
        self.t.fill_(float("nan"))  # an output that is read shows too
        if init is not None:
            self.t.copy_(init)

    def check(self, what=""):
        b = self.bytes.clone()
        rows, cols = self.t.shape
        b[:rows, :cols * self.t.element_size()] = SENTINEL
        assert bool((b == SENTINEL).all()), f"{what}: a write outside the output"


def same(a, b, what=""):
    assert torch.equal(a, b) or bool(((a == b) | (a.isnan() & b.isnan())).all()), f"{what}: results differ"


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 520), (2, 8, 8), (7, 33, 129), (16, 128, 64), (17, 257, 1000), (33, 1024, 512),
          (64, 130, 2048), (65, 97, 130), (100, 1000, 264), (128, 256, 192), (129, 300, 70), (300, 257, 200),
          (1003, 131, 77), (513, 1030, 520)]


# ------------------------------------------------------------------ forward

@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype,out", [(F16, F16), (BF16, BF16), (E4M3, BF16), (E5M2, F16)])
def test_linear_integers_are_exact(g, M, N, K, dtype, out):
    r = gen(M + N + K)
    X, W = matrix(r, M, K, dtype, ints=True), matrix(r, N, K, dtype, ints=True, pad=0)
    bias, res = vector(r, N, F32, ints=True, offset=1), matrix(r, M, N, out, ints=True)
    for act in ("none", "relu"):
        Y, Z = Guarded(M, N, out), Guarded(M, N, out)
        g.linear(X, W, bias, act=act, residual=res, out=Y.t, preact=Z.t)
        z = (X.double() @ W.double().t() + bias.double())
        y = ref.act_value(z, act) + res.double()
        same(Z.t, z.to(out), "Z")
        same(Y.t, y.to(out), "Y")
        Y.check("Y"), Z.check("Z")


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ref.ACTS)
def test_linear_against_64_bits(g, M, N, K, act):
    r = gen(7 * M + N + K)
    for dtype, out in ((F16, F16), (BF16, BF16), (E4M3, F16), (E5M2, BF16)):
        X, W = matrix(r, M, K, dtype), matrix(r, N, K, dtype, scale=1.0 if dtype in (E4M3, E5M2) else K ** -0.5)
        alpha = K ** -0.5 if dtype in (E4M3, E5M2) else 1.5
        for bias_dtype, with_res, with_z in ((F32, True, False), (out, False, True), (None, True, True), (None, False, False)):
            bias = None if bias_dtype is None else vector(r, N, bias_dtype, offset=3)
            res = matrix(r, M, N, out, pad=2) if with_res else None
            Y, Z = Guarded(M, N, out), Guarded(M, N, out)
            got = g.linear(X, W, bias, act=act, residual=res, out=Y.t, preact=Z.t if with_z else None, alpha=alpha)
            y, z = ref.linear(X, W, bias, act, res, out, alpha)
            what = f"{(M, N, K)} {dtype} {act} bias {bias_dtype}"
            ref.assert_within(got, y, "Y " + what)
            if with_z:
                ref.assert_within(Z.t, z, "Z " + what)
            Y.check(what), Z.check(what)


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("dtype,out", [(F16, F16), (BF16, BF16), (E4M3, BF16), (E4M3, F16), (E5M2, BF16), (E5M2, F16)])
def test_linear_every_tile(g, config, dtype, out):
    g.set_option(native.OPT_CONFIG, config)
    for M, N, K in ((300, 520, 1100), (257, 1000, 300), (700, 300, 4100)):
        for ctas in (0, 6):
            g.set_option(native.OPT_MAX_CTAS, ctas)
            r = gen(M)
            X, W, bias = matrix(r, M, K, dtype), matrix(r, N, K, dtype), vector(r, N, F32)
            res = matrix(r, M, N, out)
            Y, Z = Guarded(M, N, out), Guarded(M, N, out)
            g.linear(X, W, bias, act="gelu", residual=res, out=Y.t, preact=Z.t, alpha=K ** -0.5)
            y, z = ref.linear(X, W, bias, "gelu", res, out, K ** -0.5)
            ref.assert_within(Y.t, y, f"{(M, N, K)} {ctas} Y")
            ref.assert_within(Z.t, z, f"{(M, N, K)} {ctas} Z")
            Y.check(), Z.check()


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (5, 2056, 8192), (20, 1000, 2050), (48, 520, 4104), (90, 300, 8192),
                                   (256, 1030, 4100), (1000, 1000, 1000), (600, 136, 5000)])
@pytest.mark.parametrize("dtype,out", [(F16, F16), (BF16, BF16), (E4M3, BF16), (E5M2, F16)])
def test_linear_split_over_a_cluster(g, M, N, K, dtype, out):
    # Few tiles and a long contraction: the K blocks are shared by the CTAs of a cluster.
    r = gen(M + K)
    X, W, bias, res = matrix(r, M, K, dtype), matrix(r, N, K, dtype), vector(r, N, out, offset=1), matrix(r, M, N, out)
    Y, Z = Guarded(M, N, out), Guarded(M, N, out)
    g.linear(X, W, bias, act="silu", residual=res, out=Y.t, preact=Z.t, alpha=K ** -0.5)
    y, z = ref.linear(X, W, bias, "silu", res, out, K ** -0.5)
    ref.assert_within(Y.t, y, "Y")
    ref.assert_within(Z.t, z, "Z")
    Y.check(), Z.check()


@pytest.mark.parametrize("M,N,K", [(1, 2048, 520), (70, 4100, 300), (130, 1000, 1030), (300, 2048, 136), (1003, 520, 1000),
                                   (20, 8192, 8000), (9000, 200, 130), (40, 16500, 72)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients_split_over_a_cluster(g, M, N, K, dtype):
    r = gen(M + K)
    dY, W, Z, X = matrix(r, M, N, dtype), matrix(r, N, K, dtype, scale=N ** -0.5), matrix(r, M, K, dtype), matrix(r, M, K, dtype)
    for sums in (True, False):
        dX, db = Guarded(M, K, dtype), Guarded(1, K, F32)
        g.linear_dgrad(dY, W, Z, act="gelu_tanh", out=dX.t, dbias=db.t[0] if sums else None)
        d, b = ref.through_act(*ref.product(dY, W), Z, "gelu_tanh", dtype, F32)
        ref.assert_within(dX.t, d, "dX")
        dX.check()
        if sums:
            ref.assert_within(db.t[0], b, "dbias")
            db.check()
    for out in (F32, dtype):
        dW0 = matrix(r, N, K, out)
        dW = Guarded(N, K, out, init=dW0)
        g.linear_wgrad(dY, X, out=dW.t, beta=0.5)
        ref.assert_within(dW.t, ref.wgrad(dY, X, out, 1.0, 0.5, dW0), f"dW {out}")
        dW.check()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_in_place_residual(g, M):
    r = gen(1)
    X, W, res = matrix(r, M, 264, BF16), matrix(r, 1000, 264, BF16, scale=0.06), matrix(r, M, 1000, BF16)
    y, _ = ref.linear(X, W, None, "none", res, BF16)
    buf = Guarded(M, 1000, BF16, init=res)
    g.linear(X, W, residual=buf.t, out=buf.t)
    ref.assert_within(buf.t, y)
    buf.check()


@pytest.mark.parametrize("M,N,K", [(0, 8, 8), (5, 0, 8), (1, 24, 0), (200, 300, 0)])
def test_linear_empty_dimensions(g, M, N, K):
    r = gen(2)
    X, W = torch.zeros((M, K), dtype=F16, device="cuda"), torch.zeros((N, K), dtype=F16, device="cuda")
    bias, res = vector(r, N, F16), matrix(r, M, N, F16)
    Y, Z = Guarded(M, N, F16), Guarded(M, N, F16)
    g.linear(X, W, bias, act="silu", residual=res, out=Y.t, preact=Z.t)
    z = bias.double().expand(M, N)
    same(Z.t, z.to(F16))
    y = ref.act_value(z, "silu") + res.double()
    ref.assert_within(Y.t, (y, ref.rounded(2.0 ** -19 * (z.abs() + 1), y, F16)))
    Y.check(), Z.check()


def test_linear_special_values(g):
    # One NaN or infinity of X reaches its own row alone; fp16 overflow becomes infinity.
    r = gen(3)
    for M in (4, 200):
        X, W = matrix(r, M, 64, F16), matrix(r, 72, 64, F16).abs()
        X[0, 0], X[2, 5] = float("nan"), float("inf")
        Y = g.linear(X, W, act="gelu_tanh")
        assert bool(Y[0].isnan().all()) and bool((Y[2] == float("inf")).all())
        assert bool(Y[1].isfinite().all()) and bool(Y[3:].isfinite().all())
        X = torch.full((M, 64), 60000.0, dtype=F16, device="cuda")
        assert bool((g.linear(X, W.abs() + 1, act="relu") == float("inf")).all())
        big = torch.full((M, 64), 1e30, dtype=BF16, device="cuda")
        one = torch.ones((8, 64), dtype=BF16, device="cuda")
        for act in ("gelu", "gelu_tanh", "silu"):
            assert bool((g.linear(-big, one, act=act) == 0).all()), act
            assert bool(g.linear(big, one, act=act).isfinite().all()), act
            assert bool((g.linear(-big * 1e9, one, act=act) == 0).all()), act  # -infinity: the limit
            assert bool((g.linear(big * 1e9, one, act=act) == float("inf")).all()), act
            assert bool(g.linear(big * float("nan"), one, act=act).isnan().all()), act


# ------------------------------------------------------------------ backward through the weights

BACK = [(1, 8, 8), (1, 520, 1000), (7, 33, 129), (65, 97, 130), (128, 192, 256), (300, 257, 200), (1003, 131, 77),
        (513, 520, 1030), (260, 2100, 300)]


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_dgrad_integers_are_exact(g, M, N, K, dtype):
    r = gen(M + N)
    dY, W, Z = matrix(r, M, N, dtype, ints=True), matrix(r, N, K, dtype, ints=True), matrix(r, M, K, dtype, ints=True)
    dX, db = Guarded(M, K, dtype), Guarded(1, K, F32, init=torch.ones((1, K), device="cuda"))
    g.linear_dgrad(dY, W, Z, act="relu", out=dX.t, dbias=db.t[0], beta_bias=3.0, alpha=2.0)
    d = 2 * (dY.double() @ W.double()) * ref.act_slope(Z.double(), "relu")
    same(dX.t, d.to(dtype), "dX")
    same(db.t[0], (d.sum(0) + 3).float(), "dbias")
    dX.check(), db.check()


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_dgrad_against_64_bits(g, M, N, K, act, dtype):
    r = gen(5 * M + N)
    dY, W = matrix(r, M, N, dtype), matrix(r, N, K, dtype, scale=N ** -0.5)
    Z = None if act == "none" else matrix(r, M, K, dtype, scale=2.0)
    for db_dtype, beta in ((F32, 0.0), (dtype, 0.0), (F32, -0.5), (None, 0.0)):
        b0 = vector(r, K, F32)
        dX, db = Guarded(M, K, dtype), None
        if db_dtype is not None:
            db = Guarded(1, K, db_dtype, init=b0[None] if beta else None)
        g.linear_dgrad(dY, W, Z, act=act, out=dX.t, dbias=None if db is None else db.t[0], beta_bias=beta, alpha=0.75)
        p, e = ref.product(dY, W, 0.75)
        d, b = ref.through_act(p, e, Z, act, dtype, db_dtype or F32, b0, beta)
        ref.assert_within(dX.t, d, f"dX {act}")
        dX.check()
        if db is not None:
            ref.assert_within(db.t[0], b, f"dbias {act} {db_dtype} {beta}")
            db.check()


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_dgrad_every_tile(g, config, dtype):
    g.set_option(native.OPT_CONFIG, config)
    for M, N, K in ((300, 1100, 520), (257, 300, 1000), (700, 4100, 300)):
        for ctas in (0, 6):
            g.set_option(native.OPT_MAX_CTAS, ctas)
            r = gen(M)
            dY, W, Z = matrix(r, M, N, dtype), matrix(r, N, K, dtype, scale=N ** -0.5), matrix(r, M, K, dtype)
            dX, db = Guarded(M, K, dtype), Guarded(1, K, F32)
            g.linear_dgrad(dY, W, Z, act="gelu", out=dX.t, dbias=db.t[0])
            d, b = ref.through_act(*ref.product(dY, W), Z, "gelu", dtype, F32)
            ref.assert_within(dX.t, d, f"{(M, N, K)} {ctas}")
            ref.assert_within(db.t[0], b, f"{(M, N, K)} {ctas}")
            dX.check(), db.check()


@pytest.mark.parametrize("M,N,K", [(0, 8, 24), (5, 8, 0), (70, 0, 200)])
def test_dgrad_empty_dimensions(g, M, N, K):
    r = gen(4)
    dY, W = torch.zeros((M, N), dtype=F16, device="cuda"), torch.zeros((N, K), dtype=F16, device="cuda")
    Z, b0 = matrix(r, M, K, F16), vector(r, K, F32)
    dX, db = Guarded(M, K, F16), b0.clone()
    g.linear_dgrad(dY, W, Z, act="silu", out=dX.t, dbias=db, beta_bias=2.0)
    assert bool((dX.t == 0).all())
    same(db, b0 * 2)
    g.linear_dgrad(dY, W, Z, act="silu", out=dX.t, dbias=db)
    assert bool((db == 0).all())


def test_dgrad_rows_past_the_end_stay_out_of_the_sums(g):
    # An infinite weight times the zeros that fill a ragged tile would be NaN: those rows must not count.
    r = gen(5)
    dY, W = matrix(r, 130, 64, BF16).abs(), matrix(r, 64, 200, BF16)
    W[3, 7] = float("inf")
    Z, db = matrix(r, 130, 200, BF16).abs() + 1, torch.empty(200, device="cuda")
    dX = g.linear_dgrad(dY, W, Z, act="relu", dbias=db)
    assert bool((dX[:, 7] == float("inf")).all()) and db[7].item() == float("inf")
    others = torch.arange(200, device="cuda") != 7
    assert bool(db[others].isfinite().all())


# ------------------------------------------------------------------ weight gradient

@pytest.mark.parametrize("M,N,K", BACK + [(5000, 130, 70), (1, 1, 1), (3, 1000, 520)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_wgrad(g, M, N, K, dtype):
    r = gen(3 * M + N)
    for out in (F32, dtype):
        dY, X = matrix(r, M, N, dtype, ints=True), matrix(r, M, K, dtype, ints=True)
        dW0 = matrix(r, N, K, out, ints=True)
        dW = Guarded(N, K, out, init=dW0)
        g.linear_wgrad(dY, X, out=dW.t, alpha=2.0, beta=-1.0)
        same(dW.t, (2 * (dY.double().t() @ X.double()) - dW0.double()).to(out), "integers")
        dW.check()
        dY, X = matrix(r, M, N, dtype), matrix(r, M, K, dtype)
        for alpha, beta in ((1.0, 0.0), (0.5, 1.0)):
            dW = Guarded(N, K, out, init=dW0 if beta else None)  # beta == 0: dW starts as NaN
            g.linear_wgrad(dY, X, out=dW.t, alpha=alpha, beta=beta)
            ref.assert_within(dW.t, ref.wgrad(dY, X, out, alpha, beta, dW0), f"{out} {beta}")
            dW.check()


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("dtype,out", [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)])
def test_wgrad_every_tile(g, config, dtype, out):
    g.set_option(native.OPT_CONFIG, config)
    for M, N, K in ((1100, 300, 520), (300, 257, 1000), (4100, 700, 301)):
        for ctas in (0, 6):
            g.set_option(native.OPT_MAX_CTAS, ctas)
            r = gen(M)
            dY, X, dW0 = matrix(r, M, N, dtype), matrix(r, M, K, dtype), matrix(r, N, K, out)
            dW = Guarded(N, K, out, init=dW0)
            g.linear_wgrad(dY, X, out=dW.t, beta=1.0)
            ref.assert_within(dW.t, ref.wgrad(dY, X, out, 1.0, 1.0, dW0), f"{(M, N, K)} {ctas}")
            dW.check()


@pytest.mark.parametrize("rows", [1100, 890, 1500])
def test_last_tiles_shared_after_whole_ones(g, rows):
    # Four CTAs, a long contraction, and tiles that do not divide by four (9, 7): whole tiles, then, where it pays, the K
    # blocks of the rest shared out and joined.
    L = 12288
    r = gen(rows)
    g.set_option(native.OPT_CONFIG, native.CONFIG_128x128)
    g.set_option(native.OPT_MAX_CTAS, 4)
    for dtype in (F16, BF16):
        X, W, res = matrix(r, rows, L, dtype), matrix(r, 100, L, dtype, scale=L ** -0.5), matrix(r, rows, 100, dtype)
        Y = Guarded(rows, 100, dtype)
        g.linear(X, W, act="gelu", residual=res, out=Y.t)
        ref.assert_within(Y.t, ref.linear(X, W, None, "gelu", res, dtype)[0], "forward")
        Y.check()
        dY, Wd, Z = X, matrix(r, L, 100, dtype, scale=L ** -0.5), matrix(r, rows, 100, dtype)
        for sums in (True, False):
            dX, db = Guarded(rows, 100, dtype), Guarded(1, 100, F32)
            g.linear_dgrad(dY, Wd, Z, act="silu", out=dX.t, dbias=db.t[0] if sums else None)
            d, b = ref.through_act(*ref.product(dY, Wd), Z, "silu", dtype, F32)
            ref.assert_within(dX.t, d, "dgrad")
            dX.check()
            if sums:
                ref.assert_within(db.t[0], b, "dbias")
        A, B = matrix(r, L, rows, dtype), matrix(r, L, 100, dtype)
        for out in (F32, dtype):
            dW = Guarded(rows, 100, out)
            g.linear_wgrad(A, B, out=dW.t)
            ref.assert_within(dW.t, ref.wgrad(A, B, out), f"wgrad {out}")
            dW.check()


@pytest.mark.parametrize("out", [F16, F32])
def test_wgrad_no_tokens(g, out):
    dY, X = torch.zeros((0, 40), dtype=F16, device="cuda"), torch.zeros((0, 56), dtype=F16, device="cuda")
    dW0 = matrix(gen(6), 40, 56, out, ints=True)
    dW = Guarded(40, 56, out, init=dW0)
    g.linear_wgrad(dY, X, out=dW.t, beta=-2.0)
    same(dW.t, dW0 * -2)
    g.linear_wgrad(dY, X, out=dW.t)
    assert bool((dW.t == 0).all())
    dW.check()


def test_fp32_sums_keep_their_precision(g):
    # The sums of a long contraction lose no more than a fp32 chain would: the relative error of the whole
    # gradient stays under 2e-6 (a tensor-core accumulator alone, which truncates, is 10 times further off here).
    r = gen(7)
    dY, X = matrix(r, 16384, 256, BF16), matrix(r, 16384, 256, BF16)
    for n in (256, 40):  # tiles of both kinds of kernel
        got = g.linear_wgrad(dY[:, :n], X).double()
        want = dY[:, :n].double().t() @ X.double()
        assert ((got - want).norm() / want.norm()).item() < 2e-6


# ------------------------------------------------------------------ activation's backward

@pytest.mark.parametrize("M,N", [(1, 1), (1, 1000), (2, 64), (33, 7), (65, 1000), (300, 257), (1003, 2056), (4097, 40)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", ref.ACTS)
def test_act_grad(g, M, N, dtype, act):
    r = gen(M + N)
    dY, Z = matrix(r, M, N, dtype), None if act == "none" else matrix(r, M, N, dtype, scale=3.0)
    b0 = vector(r, N, F32)
    for db_dtype, beta in ((F32, 0.0), (dtype, 0.0), (F32, 1.0), (None, 0.0)):
        dZ, db = Guarded(M, N, dtype), None
        if db_dtype is not None:
            db = Guarded(1, N, db_dtype, init=b0[None] if beta else None)
        g.act_grad(dY, Z, act=act, out=dZ.t, dbias=None if db is None else db.t[0], beta_bias=beta)
        d, b = ref.through_act(dY.double(), torch.zeros_like(dY.double()), Z, act, dtype, db_dtype or F32, b0, beta)
        ref.assert_within(dZ.t, d, act)
        dZ.check()
        if db is not None:
            ref.assert_within(db.t[0], b, f"{act} {db_dtype} {beta}")
            db.check()


def test_act_grad_sums_only_in_place_and_empty(g):
    r = gen(8)
    dY, Z = matrix(r, 77, 136, BF16), matrix(r, 77, 136, BF16)
    d, b = ref.through_act(dY.double(), torch.zeros_like(dY.double()), Z, "silu", BF16, F32)
    db = torch.empty(136, device="cuda")
    assert g.act_grad(dY, Z, act="silu", dbias=db, sums_only=True) is None
    ref.assert_within(db, b)
    buf = Guarded(77, 136, BF16, init=dY)
    g.act_grad(buf.t, Z, act="silu", out=buf.t, dbias=db)
    ref.assert_within(buf.t, d)
    ref.assert_within(db, b)
    buf.check()
    db = torch.ones(24, device="cuda")
    g.act_grad(torch.zeros((0, 24), dtype=F16, device="cuda"), dbias=db, beta_bias=0.5)
    assert bool((db == 0.5).all())


def test_z_is_not_read_without_an_activation(g):
    r = gen(15)
    dY, W, Z = matrix(r, 40, 64, F16, ints=True), matrix(r, 64, 72, F16, ints=True), matrix(r, 40, 72, F16) * float("nan")
    same(g.linear_dgrad(dY, W, Z, act="none"), (dY.double() @ W.double()).half())
    same(g.act_grad(dY, matrix(r, 40, 64, F16) * float("nan")), dY)


def test_act_grad_special_values(g):
    inf, nan = float("inf"), float("nan")
    Z = torch.tensor([[inf, -inf, nan, 0.0, -0.0, 3e4, -3e4, 1e-7]], dtype=F16, device="cuda")
    one = torch.ones_like(Z)
    want = {"relu": [1, 0, nan, 0, 0, 1, 0, 1], "gelu": [1, 0, nan, .5, .5, 1, 0, .5],
            "gelu_tanh": [1, 0, nan, .5, .5, 1, 0, .5], "silu": [1, 0, nan, .5, .5, 1, 0, .5]}
    for act, w in want.items():
        same(g.act_grad(one, Z, act=act), torch.tensor([w], dtype=F16, device="cuda"), act)
    Zb = torch.tensor([[1e30, -1e30, 3e38, -3e38, 20.0, -200.0, 0, 0]], dtype=BF16, device="cuda")
    for act in ref.ACTS[1:]:
        got = g.act_grad(torch.ones_like(Zb), Zb, act=act)
        same(got[:, :6], torch.tensor([[1, 0, 1, 0, 1, 0]], dtype=BF16, device="cuda"), act)


@pytest.mark.parametrize("act", ref.ACTS[1:])
def test_slopes_against_differences(g, act):
    # act'(z) against (act(z + h) - act(z - h)) / 2h in fp64: the difference is within h^2 of the slope (third
    # derivatives of these functions stay under 6) plus the rounding of the values over h.
    z = torch.linspace(-9, 9, 4096, device="cuda").to(F16).reshape(8, 512)
    if act == "relu":
        z = torch.where(z == 0, torch.ones_like(z), z)
    h = 2.0 ** -12
    zd = z.double()
    want = (ref.act_value(zd + h, act) - ref.act_value(zd - h, act)) / (2 * h)
    got = g.act_grad(torch.ones_like(z), z, act=act)
    ref.assert_within(got, (want, ref.rounded(torch.full_like(want, 2.0 ** -17 + 6 * h * h), want, F16)), act)


# ------------------------------------------------------------------ the layer's gradients together

def test_layer_gradients_against_differences(g):
    # L = sum(G * act(X W^T + b)): dL along a direction of each parameter, from the kernels' gradients, against
    # central differences of L in fp64.  The kernels round dZ and Z to bf16 (2^-8 of a value at most, 2^-9 on
    # average): the bound is 2^-8 of the sum of the terms' magnitudes for dZ, the average for the other roundings, and
    # h^2 times third derivatives (under 6 per element) of a direction of unit entries.
    r = gen(9)
    M, N, K, act = 70, 200, 96, "gelu_tanh"
    X, W, b = matrix(r, M, K, BF16), matrix(r, N, K, BF16, scale=0.1), vector(r, N, BF16)
    G = matrix(r, M, N, BF16)
    Z, db = torch.empty((M, N), dtype=BF16, device="cuda"), torch.empty(N, device="cuda")
    g.linear(X, W, b, act=act, preact=Z)
    dZ = g.act_grad(G, Z, act=act, dbias=db)
    dX, dW = g.linear_dgrad(dZ, W), g.linear_wgrad(dZ, X)

    def loss(x, w, c):
        return (G.double() * ref.act_value(x @ w.t() + c, act)).sum()

    x, w, c = X.double(), W.double(), b.double()
    h = 1e-4
    for name, grad, at in (("X", dX, 0), ("W", dW, 1), ("b", db, 2)):
        for _ in range(4):
            v = torch.randn(grad.shape, generator=r, device="cuda", dtype=torch.float64)
            plus, minus = [x, w, c], [x, w, c]
            plus[at], minus[at] = plus[at] + h * v, minus[at] - h * v
            want = ((loss(*plus) - loss(*minus)) / (2 * h)).item()
            terms = grad.double() * v
            # dZ's own rounding (Z is rounded to bf16 before its slope is taken: 2^-9 |Z| on average times a second
            # derivative under 1.2) enters every gradient through magnitudes, not signed sums.
            dz = (G.double().abs() * (2.0 ** -8 + 2.0 ** -9 * 1.2 * Z.double().abs()))
            mags = {0: dz @ w.abs(), 1: dz.t() @ x.abs(), 2: dz.sum(0)}[at]
            bound = (mags * v.abs()).sum().item() + 2.0 ** -9 * terms.abs().sum().item() + 1e-3
            assert abs(terms.sum().item() - want) <= bound, name
            # ... and, rounding being unbiased, far closer than that worst case
            assert abs(terms.sum().item() - want) <= 0.05 * bound + 1e-3, name


# ------------------------------------------------------------------ streams, graphs, determinism, large offsets

def every_op(g, r, M=300, N=257, K=520, stream=None):
    X, W, b = matrix(r, M, K, BF16), matrix(r, N, K, BF16, scale=K ** -0.5), vector(r, N, F32)
    Z = torch.empty((M, pitch(N, BF16)), dtype=BF16, device="cuda")[:, :N]
    db = torch.empty(N, device="cuda")
    db2 = torch.empty(K, device="cuda")
    torch.cuda.synchronize()
    Zk = matrix(r, M, K, BF16)
    torch.cuda.synchronize()

    def call():
        Y = g.linear(X, W, b, act="silu", preact=Z, stream=stream)
        dZ = g.act_grad(Y, Z, act="silu", dbias=db, stream=stream)
        dX = g.linear_dgrad(dZ, W, Zk, act="gelu", dbias=db2, stream=stream)
        dW = g.linear_wgrad(dZ, X, stream=stream)
        return [Y, Z, dZ, db, dX, db2, dW]
    return call


@pytest.mark.parametrize("M", [9, 300])
def test_runs_repeat_bit_for_bit(g, M):
    call = every_op(g, gen(10), M=M)
    first = [t.clone() for t in call()]
    for _ in range(5):
        for a, b in zip(first, call()):
            same(a, b)


def test_side_stream(g):
    want = [t.clone() for t in every_op(g, gen(11))()]
    s = torch.cuda.Stream()
    for arg in (s, s.cuda_stream):
        got = every_op(g, gen(11), stream=arg)()
        assert g.sync_status(s) == native.OK
        for a, b in zip(want, got):
            same(a, b)


def test_graph_capture(g):
    call = every_op(g, gen(12), M=64)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for t in out:
        t.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, out):
        same(a, b)


def test_offsets_past_32_bits(g):
    # Rows 2^16 elements apart and 40000 of them: the last ones start past 2^31 elements and 2^32 bytes.
    M, ld = 40000, 1 << 16
    r = gen(13)
    bufs = [torch.empty((M, ld), dtype=BF16, device="cuda") for _ in range(3)]
    X, Y, Z = (b[:, :64] for b in bufs)
    X.copy_(torch.randn((M, 64), generator=r, device="cuda"))
    Z.copy_(torch.randn((M, 64), generator=r, device="cuda"))
    W, db = matrix(r, 64, 64, BF16, scale=0.125), torch.empty(64, device="cuda")
    g.linear(X, W, act="relu", residual=Z, out=Y)
    ref.assert_within(Y, ref.linear(X, W, None, "relu", Z, BF16)[0], "linear")
    g.linear_dgrad(X, W, Z, act="silu", out=Y, dbias=db)
    d, b = ref.through_act(*ref.product(X, W), Z, "silu", BF16, F32)
    ref.assert_within(Y, d, "dgrad")
    ref.assert_within(db, b, "dgrad dbias")
    g.act_grad(X, Z, act="silu", out=Y, dbias=db)
    d, b = ref.through_act(X.double(), torch.zeros_like(X.double()), Z, "silu", BF16, F32)
    ref.assert_within(Y, d, "act_grad")
    ref.assert_within(db, b, "act_grad dbias")
    ref.assert_within(g.linear_wgrad(X, Z), ref.wgrad(X, Z, F32), "wgrad")


# ------------------------------------------------------------------ refusals

def struct(cls, base, **changes):
    a = cls(**base)
    for k, v in changes.items():
        setattr(a, k, v)
    return ctypes.byref(a)


INV, UNS = native.ERR_INVALID_ARG, native.ERR_UNSUPPORTED


def test_refusals(g):
    buf = torch.zeros(1 << 16, dtype=F16, device="cuda")
    p = buf.data_ptr()
    lib, h = g._lib, g._h
    fwd = dict(X=p, W=p, Y=p, M=16, N=16, K=16, ldx=16, ldw=16, ldy=16, ldr=16, ldz=16, alpha=1.0)
    for bad, want in [(dict(X=None), INV), (dict(W=None), INV), (dict(Y=None), INV), (dict(M=-1), INV), (dict(K=-1), INV),
                      (dict(ldx=8), INV), (dict(ldw=8), INV), (dict(ldy=8), INV), (dict(residual=p, ldr=8), INV),
                      (dict(Z=p, ldz=8), INV), (dict(dtype=4), INV), (dict(dtype=9), INV), (dict(out_dtype=1), INV),
                      (dict(out_dtype=4), INV), (dict(dtype=2, out_dtype=2), INV), (dict(act=5), INV), (dict(act=-1), INV),
                      (dict(alpha=float("nan")), INV), (dict(alpha=float("inf")), INV), (dict(bias=p, bias_dtype=1), INV),
                      (dict(X=p + 2), UNS), (dict(W=p + 8), UNS), (dict(Y=p + 4), UNS), (dict(ldx=20), UNS),
                      (dict(dtype=2, ldx=24), UNS), (dict(residual=p + 2), UNS), (dict(Z=p, ldz=20), UNS),
                      (dict(bias=p + 1), UNS), (dict(bias=p + 2, bias_dtype=4), UNS), (dict(M=1 << 31), UNS),
                      (dict(M=0, X=None, Y=None), native.OK), (dict(N=0, W=None), native.OK)]:
        got = lib.gemm_run_linear(h, struct(native.gemm_linear_args_t, fwd, **bad), None)
        assert got == want, (bad, got)
    bwd = dict(dY=p, W=p, Z=p, dX=p, dbias=p, workspace=p, workspace_bytes=1 << 12, M=16, N=16, K=16, lddy=16, ldw=16,
               ldz=16, lddx=16, act=1, alpha=1.0, dbias_dtype=4)
    for bad, want in [(dict(Z=None), INV), (dict(dY=None), INV), (dict(dX=None), INV), (dict(dtype=2), INV),
                      (dict(workspace=None, M=1 << 20), INV), (dict(workspace_bytes=255), INV), (dict(dbias_dtype=1), INV),
                      (dict(beta_bias=float("nan")), INV), (dict(ldz=8), INV), (dict(act=7), INV), (dict(N=-1), INV),
                      (dict(workspace=p + 4), UNS), (dict(ldz=20), UNS), (dict(dbias=p + 2), UNS), (dict(dX=p + 2), UNS),
                      (dict(K=0, dX=None), native.OK)]:
        got = lib.gemm_run_linear_dgrad(h, struct(native.gemm_dgrad_args_t, bwd, **bad), None)
        assert got == want, (bad, got)
    wg = dict(dY=p, X=p, dW=p, M=16, N=16, K=16, lddy=16, ldx=16, lddw=16, out_dtype=4, alpha=1.0)
    for bad, want in [(dict(dY=None), INV), (dict(dW=None), INV), (dict(out_dtype=1), INV), (dict(dtype=2), INV),
                      (dict(beta=float("inf")), INV), (dict(lddw=8), INV), (dict(lddw=18), UNS), (dict(dW=p + 4), UNS),
                      (dict(out_dtype=0, lddw=20), UNS), (dict(N=0, dW=None), native.OK)]:
        got = lib.gemm_run_linear_wgrad(h, struct(native.gemm_wgrad_args_t, wg, **bad), None)
        assert got == want, (bad, got)
    ag = dict(dY=p, Z=p, dZ=p, dbias=p, workspace=p, workspace_bytes=1 << 12, M=16, N=16, lddy=16, ldz=16, lddz=16, act=2,
              dbias_dtype=4)
    for bad, want in [(dict(dY=None), INV), (dict(Z=None), INV), (dict(workspace=None, M=1 << 20), INV), (dict(lddz=8), INV),
                      (dict(dtype=4), INV), (dict(dZ=p + 2), UNS), (dict(lddy=20), UNS), (dict(N=0, dY=None), native.OK)]:
        got = lib.gemm_run_act_grad(h, struct(native.gemm_act_grad_args_t, ag, **bad), None)
        assert got == want, (bad, got)


def test_binding_refusals(g):
    X, W = torch.zeros((8, 16), dtype=F16, device="cuda"), torch.zeros((24, 16), dtype=F16, device="cuda")
    for call in (lambda: g.linear(X, W.bfloat16()), lambda: g.linear(X, W, out_dtype=BF16),
                 lambda: g.linear(X, W, torch.zeros(24, dtype=BF16, device="cuda")), lambda: g.linear(X.float(), W.float()),
                 lambda: g.linear_wgrad(X, X, out_dtype=BF16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: g.linear(X, W[:, :8]), lambda: g.linear(X, W, act="tanh"), lambda: g.linear(X, W, torch.zeros(23, device="cuda")),
                 lambda: g.linear(X, W, residual=X), lambda: g.linear(X.t(), W.t()), lambda: g.linear(X, W.cpu()),
                 lambda: g.linear_dgrad(X, W.t().contiguous(), act="gelu"), lambda: g.linear_wgrad(X, W),
                 lambda: g.linear_wgrad(X, X, beta=1.0), lambda: g.act_grad(X, act="relu"), lambda: g.act_grad(X, sums_only=True),
                 lambda: g.linear(X, W, torch.zeros(48, device="cuda")[::2])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(native.GemmError):
        g.linear(torch.zeros((8, 12), dtype=F16, device="cuda"), torch.zeros((8, 12), dtype=F16, device="cuda"))


# ------------------------------------------------------------------ the watchdog

@pytest.mark.parametrize("M,config", [(4, native.CONFIG_AUTO), (100, native.CONFIG_AUTO), (600, native.CONFIG_128x128),
                                      (600, native.CONFIG_128x256), (600, native.CONFIG_256x256)])
def test_a_wait_that_runs_out_is_reported(g, M, config):
    # A stage that never arrives (the library's own test hook): each wait gives up after its limit, the kernel
    # leaves, the host reads the status, and the next call is right.
    r = gen(14)
    X, W, Z = matrix(r, M, 1024, BF16), matrix(r, 520, 1024, BF16, scale=0.03), matrix(r, M, 1024, BF16)
    dY, db = matrix(r, M, 520, BF16), torch.empty(1024, device="cuda")
    calls = [lambda: g.linear(X, W, act="gelu"), lambda: g.linear_dgrad(dY, W, Z, act="gelu", dbias=db),
             lambda: g.linear_wgrad(dY, X)]
    g.set_option(native.OPT_CONFIG, config)
    want = [c().clone() for c in calls]
    assert g.sync_status() == native.OK
    for call, w in zip(calls, want):
        g.set_option(native.OPT_TIMEOUT_NS, 50_000_000)
        g.set_option(native.OPT_FAULT_INJECT, 1)
        try:
            call()
            assert g.sync_status() == native.ERR_TIMEOUT
            assert g.error_info()[0] == 1
        finally:
            g.set_option(native.OPT_FAULT_INJECT, 0)
            g.set_option(native.OPT_TIMEOUT_NS, 2_000_000_000)
        same(call(), w)
        assert g.sync_status() == native.OK


# ------------------------------------------------------------------ the operators together

def test_feed_forward_example(g):
    import importlib.util
    import os

    from conftest import ROOT

    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, off = example.train(tokens=520, width=264, hidden=1000, steps=12)
    assert losses[-1] < 0.8 * losses[0] and all(b < a for a, b in zip(losses, losses[1:]))
    # The same products in other tiles: the sums differ in order alone, by less than a bf16 step of values under 8.
    assert off <= 2.0 ** -5


def test_feed_forward_gradients_against_autograd(g):
    # The block's gradients in bf16 against autograd's in fp64 on the same (bf16) weights: each bf16 rounding on the way
    # (H, Z, dZ) is 2^-9 of its value on average, so the norms agree within 1 %.
    import importlib.util
    import os

    from conftest import ROOT

    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    block = example.FeedForward(256, 520, seed=3)
    block.master["b1"].copy_(torch.randn(520, generator=gen(1), device="cuda"))
    r = gen(20)
    X, dY = matrix(r, 300, 256, BF16, pad=0), matrix(r, 300, 256, BF16, pad=0)
    Y, saved = block.forward(X)
    dX = block.backward(dY, saved)
    x, w1, b1, w2, b2 = (t.double().requires_grad_(True) for t in (X, block.W1, block.master["b1"], block.W2, block.master["b2"]))
    h = ref.act_value(x @ w1.t() + b1, block.act)
    y = h @ w2.t() + b2 + x
    want = torch.autograd.grad((y * dY.double()).sum(), (x, w1, b1, w2, b2))
    assert ((Y.double() - y).norm() / y.norm()).item() < 0.01
    for name, got, w in zip(("X", "W1", "b1", "W2", "b2"), (dX, block.grad["W1"], block.grad["b1"], block.grad["W2"], block.grad["b2"]), want):
        assert ((got.double() - w).norm() / w.norm()).item() < 0.01, name
