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


# ------------------------------------------------------------------ several streams at once

def test_module_functions_on_two_streams_at_once(g):  # noqa: F811
    # Column sums, stream-K parts and counters of unordered calls must not meet.
    r = gen(40)
    cases = []
    for seed, (M, N, K) in enumerate([(1000, 136, 520), (2000, 72, 264)]):
        dY, W, Z = matrix(r, M, N, BF16, ints=True), matrix(r, N, K, BF16, ints=True), matrix(r, M, K, BF16, ints=True)
        G, Zn = matrix(r, M, K, BF16, ints=True), matrix(r, M, K, BF16, ints=True)
        slope = ref.act_slope(Z.double(), "relu")
        cases.append((dY, W, Z, G, Zn, ((dY.double() @ W.double()) * slope).sum(0).float(),
                      (G.double() * ref.act_slope(Zn.double(), "relu")).sum(0).float()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    rounds = 40
    out = [[(torch.empty(c[5].shape, device="cuda"), torch.empty(c[6].shape, device="cuda")) for _ in range(rounds)] for c in cases]
    torch.cuda.synchronize()
    for i in range(rounds):
        for s, c, o in zip(streams, cases, out):
            native.linear_dgrad(c[0], c[1], c[2], act="relu", dbias=o[i][0], stream=s)
            native.act_grad(c[3], c[4], act="relu", dbias=o[i][1], sums_only=True, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, out):
        for db, dz in o:
            same(db, c[5], "dgrad's sums")
            same(dz, c[6], "act_grad's sums")


def test_module_functions_captured_on_a_stream_of_their_own(g):  # noqa: F811
    # The capture stream's handle is made during the capture; the graph's replays and eager calls do not share a workspace.
    r = gen(41)
    dY, W, Z = matrix(r, 1000, 136, BF16, ints=True), matrix(r, 136, 520, BF16, ints=True), matrix(r, 1000, 520, BF16, ints=True)
    db, db2 = torch.zeros(520, device="cuda"), torch.zeros(520, device="cuda")
    want = ((dY.double() @ W.double()) * ref.act_slope(Z.double(), "relu")).sum(0).float()
    native.linear_dgrad(dY, W, Z, act="relu", dbias=db)
    same(db, want, "eager")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    db.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        dX = native.linear_dgrad(dY, W, Z, act="relu", dbias=db)
    for _ in range(10):
        with torch.cuda.stream(side):
            graph.replay()
        native.linear_dgrad(dY, W, Z, act="relu", dbias=db2)
        native.linear_wgrad(dY, Z)
    torch.cuda.synchronize()
    same(db, want, "replayed")
    same(db2, want, "beside the replays")
    same(dX, ((dY.double() @ W.double()) * ref.act_slope(Z.double(), "relu")).bfloat16(), "dX")


def test_a_handle_made_during_a_capture(g):  # noqa: F811
    x = matrix(gen(42), 64, 64, BF16, ints=True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        h = native.Gemm(0)
        y = h.linear(x, x)
    graph.replay()
    torch.cuda.synchronize()
    assert h.sync_status() == native.OK
    same(y, (x.double() @ x.double().t()).bfloat16())
    del graph
    h.close()


# ------------------------------------------------------------------ contractions longer than one accumulator keeps

# The tensor core's fp32 accumulator truncates: a chain of K products ends about 1.2e-9 K of its value nearer to zero.
# Chains stop at 8192 products of 16 bits (16384 of 8 bits, which are added two at a time), so whatever the length, the
# results' projection on the exact ones is short by no more than 1e-5 and what the fp32 additions of the chains add;
# the rounding to fp16 is unbiased, 2^-11 / sqrt(3) at most on average, over 1e5 results or more 1e-6.
def shrink(got, want):
    return ((got.double() - want) * want).sum().item() / (want * want).sum().item()


LONG = 2e-5


@pytest.mark.parametrize("config", [native.CONFIG_AUTO] + TILES)
@pytest.mark.parametrize("dtype", [F16, BF16, torch.float8_e4m3fn, torch.float8_e5m2])
def test_long_contractions_forward(g, config, dtype):  # noqa: F811
    g.set_option(native.OPT_CONFIG, config)
    r = gen(50)
    M, N, K = 300, 400, 100000
    out = BF16 if dtype == BF16 else F16
    X, W = matrix(r, M, K, dtype), matrix(r, N, K, dtype)
    bias, res = vector(r, N, F32), matrix(r, M, N, out)
    Y, Z = Guarded(M, N, out), Guarded(M, N, out)
    g.linear(X, W, bias, act="gelu", residual=res, out=Y.t, preact=Z.t, alpha=K ** -0.5)
    y, z = ref.linear(X, W, bias, "gelu", res, out, K ** -0.5)
    ref.assert_within(Y.t, y, "Y")
    ref.assert_within(Z.t, z, "Z")
    Y.check(), Z.check()
    if out == F16:
        assert abs(shrink(Z.t, z[0])) < LONG


@pytest.mark.parametrize("M,N,K", [(1, 128 * 160, 16400), (16, 2048, 262144), (20, 6000, 40000), (64, 20000, 12300), (120, 19000, 12400)])
@pytest.mark.parametrize("dtype", [F16, torch.float8_e4m3fn])
def test_long_contractions_of_few_tokens(g, M, N, K, dtype):  # noqa: F811
    # Shares of a rank longer than one accumulator keeps: further accumulators, or the tile kernels.
    r = gen(51)
    X, W = matrix(r, M, K, dtype), matrix(r, N, K, dtype)
    Y = Guarded(M, N, F16)
    g.linear(X, W, out=Y.t, alpha=K ** -0.5)
    y, _ = ref.linear(X, W, None, "none", None, F16, K ** -0.5)
    ref.assert_within(Y.t, y, "Y")
    assert abs(shrink(Y.t, y[0])) < LONG
    Y.check()


@pytest.mark.parametrize("config", [native.CONFIG_AUTO] + TILES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_long_contractions_backward(g, config, dtype):  # noqa: F811
    g.set_option(native.OPT_CONFIG, config)
    r = gen(52)
    L = 100000
    dY, W, Z = matrix(r, 300, L, dtype, scale=L ** -0.5), matrix(r, L, 392, dtype), matrix(r, 300, 392, dtype)
    dX = Guarded(300, 392, dtype)
    g.linear_dgrad(dY, W, Z, act="silu", out=dX.t)
    d, _ = ref.through_act(*ref.product(dY, W), Z, "silu", dtype, F32)
    ref.assert_within(dX.t, d, "dX")
    dX.check()
    A, B = matrix(r, L, 300, dtype, scale=L ** -0.5), matrix(r, L, 392, dtype)
    dW0 = matrix(r, 300, 392, dtype)
    dW = Guarded(300, 392, dtype, init=dW0)
    g.linear_wgrad(A, B, out=dW.t, beta=0.5)
    w = ref.wgrad(A, B, dtype, 1.0, 0.5, dW0)
    ref.assert_within(dW.t, w, "dW")
    dW.check()
    if dtype == F16:
        assert abs(shrink(dX.t, d[0])) < LONG
        assert abs(shrink(dW.t, w[0])) < LONG


# ------------------------------------------------------------------ streams by their numbers

def test_outputs_belong_to_the_stream_that_a_number_names(g, monkeypatch):  # noqa: F811
    # A new output's memory goes back to its stream's pool: it must be the stream that the call runs on.  0 is the
    # default stream.
    r = gen(60)
    X, W = matrix(r, 40, 64, F16, ints=True), matrix(r, 72, 64, F16, ints=True)
    side, real, seen = torch.cuda.Stream(), torch.cuda.stream, []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: seen.append(s.cuda_stream) or real(s))
    torch.cuda.synchronize()
    want = (X.double() @ W.double().t()).half()
    for number in (0, side.cuda_stream):
        Y = g.linear(X, W, stream=number)
        torch.cuda.synchronize()
        same(Y, want)
        assert seen.pop() == number and not seen


# ------------------------------------------------------------------ wide layers

@pytest.mark.parametrize("M,N,K", [(1, 28672, 264), (1, 128256, 520), (3, 39001, 1000), (33, 64000, 136)])
@pytest.mark.parametrize("dtype", [F16, BF16, torch.float8_e4m3fn])
def test_few_tokens_through_wide_layers(g, M, N, K, dtype):  # noqa: F811
    # More tiles of 128 features than the GPU runs at once in clusters: those products take the tile kernels.
    r = gen(70)
    out = F16 if dtype == F16 else BF16
    X, W = matrix(r, M, K, dtype, ints=True), matrix(r, N, K, dtype, ints=True)
    bias, res = vector(r, N, F32, ints=True), matrix(r, M, N, out, ints=True)
    Y = Guarded(M, N, out)
    g.linear(X, W, bias, act="relu", residual=res, out=Y.t)
    want = ref.act_value(X.double() @ W.double().t() + bias.double(), "relu") + res.double()
    same(Y.t, want.to(out), "Y")
    Y.check("Y")
