"""The linear layer's operators, as they are measured: their cases, inputs, plain forms and 64-bit values.

Four operators make up a linear layer Y = act(alpha X W^T + bias) + residual that is trained and served
(X: M tokens x K features, W: N x K as a layer stores it):

  linear     Y, and with "keep" the pre-activation Z = alpha X W^T + bias that the backward pass reads
  dgrad      dX = (dY W) * act'(Z), Z the pre-activation below this layer, and dbias, its column sums
  wgrad      dW = dY^T X in fp32 (or the operand type), added to a gradient buffer with "accumulate"
  act_grad   dZ = dY * act'(Z) and its column sums, where no product comes before the activation

The plain forms compute in fp32 and round once; exact() computes the same values in fp64.
Sizes: M tokens, N outputs, K inputs of the layer.  Rows whose length is not a multiple of 16 bytes are
padded to one, as the library's tensor-memory copies need.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
          "e5m2": torch.float8_e5m2}
SQRT_HALF = 0.7071067811865476      # sqrt(1/2)
SQRT_2_PI = 0.7978845608028654      # sqrt(2/pi): gelu_tanh's inner scale
INV_SQRT_2PI = 0.3989422804014327   # 1/sqrt(2 pi): the normal density at 0


def _linear(name, M, N, K, dtype, act, bias=True, residual=False, keep=False, out="bf16"):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "dtype": dtype, "out": dtype if out is None else out,
            "act": act, "bias": bias, "residual": residual, "keep": keep}


def _dgrad(name, M, N, K, dtype, act):
    return {"name": name, "op": "dgrad", "M": M, "N": N, "K": K, "dtype": dtype, "act": act}


def _wgrad(name, M, N, K, dtype, out, accumulate):
    return {"name": name, "op": "wgrad", "M": M, "N": N, "K": K, "dtype": dtype, "out": out, "accumulate": accumulate}


def _act_grad(name, M, N, dtype, act):
    return {"name": name, "op": "act_grad", "M": M, "N": N, "K": 0, "dtype": dtype, "act": act}


def listed():
    return [
        # One token of one sequence through a layer: the smallest serving call, bound by latency and the weights' bytes.
        _linear("token 4096x4096", 1, 4096, 4096, "bf16", "silu"),
        # A batch of 33 sequences, one token each, through the layer that returns to the residual stream.
        _linear("batch of 33 tokens", 33, 1024, 8192, "f16", "none", residual=True, out="f16"),
        # The benchmark's ragged cube with everything in the epilogue.
        _linear("ragged 1000", 1000, 1000, 1000, "f16", "gelu", residual=True, out="f16"),
        # A prompt through a layer with 8-bit weights and activations.
        _linear("prompt e4m3 4096", 4096, 4096, 4096, "e4m3", "relu"),
        # The training forward pass at the benchmark's headline size; keeps Z for the backward pass.
        _linear("training forward 8192", 8192, 8192, 8192, "bf16", "gelu_tanh", keep=True),
        # The benchmark's tall problem: back to the residual stream from a wide hidden layer.
        _linear("tall with residual", 16384, 1024, 8192, "f16", "none", residual=True, out="f16"),
        # The backward pass of that layer, through the activation below it.
        _dgrad("dgrad tall", 16384, 1024, 8192, "f16", "gelu"),
        # Backward of a small ragged batch.
        _dgrad("dgrad ragged", 1003, 520, 1000, "bf16", "silu"),
        # Weight gradient of the tall layer, added to the fp32 gradient of earlier micro-batches.
        _wgrad("wgrad tall accumulate", 16384, 1024, 8192, "bf16", "f32", True),
        # Weight gradient of a small ragged batch, in the operand type.
        _wgrad("wgrad ragged", 1003, 1000, 520, "f16", "f16", False),
        # An activation's backward pass on its own, at the headline width.
        _act_grad("act_grad 8192", 8192, 8192, "bf16", "gelu_tanh"),
        # The same for a handful of ragged rows: the smallest training call.
        _act_grad("act_grad ragged", 65, 1000, "f16", "silu"),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["linear", "linear", "linear", "dgrad", "wgrad", "act_grad"])
    acts = ["none", "relu", "gelu", "gelu_tanh", "silu"]
    M, N, K = size(1, 16384), size(64, 8192), size(64, 8192)
    while M * N * K > 8192 ** 3:
        M = size(1, 16384)
    if op == "linear":
        dtype = rng.choice(["f16", "bf16", "bf16", "e4m3", "e5m2"])
        out = rng.choice(["f16", "bf16"]) if dtype in ("e4m3", "e5m2") else dtype
        c = _linear("", M, N, K, dtype, rng.choice(acts), rng.random() < 0.8, rng.random() < 0.4, rng.random() < 0.3, out)
    elif op == "dgrad":
        c = _dgrad("", M, N, K, rng.choice(["f16", "bf16"]), rng.choice(acts))
    elif op == "wgrad":
        dtype = rng.choice(["f16", "bf16"])
        out = rng.choice(["f32", dtype])
        c = _wgrad("", M, N, K, dtype, out, out == "f32" and rng.random() < 0.5)
    else:
        c = _act_grad("", M, N, rng.choice(["f16", "bf16"]), rng.choice(acts[1:]))
    del c["name"]
    return c


def _padded(rows, cols, dtype):
    """An uninitialised rows x cols tensor whose rows are a multiple of 16 bytes apart."""
    e = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty((rows, -(-cols // e) * e), dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    dt = DTYPES[case["dtype"]]

    def normal(rows, cols, dtype, scale):
        t = _padded(rows, cols, dtype)
        t.copy_(torch.randn((rows, cols), generator=gen, device="cuda") * scale)
        return t

    s = dict(case)
    if op == "linear":
        out = DTYPES[case["out"]]
        f8 = case["dtype"] in ("e4m3", "e5m2")
        # 8-bit operands are kept at unit size and carry their scale beside them.
        s["alpha"] = K ** -0.5 if f8 else 1.0
        s["X"] = normal(M, K, dt, 1.0)
        s["W"] = normal(N, K, dt, 1.0 if f8 else K ** -0.5)
        s["bias_t"] = (torch.randn(N, generator=gen, device="cuda") * 0.5).to(out) if case["bias"] else None
        s["residual_t"] = normal(M, N, out, 1.0) if case["residual"] else None
        s["Y"] = _padded(M, N, out)
        s["Z"] = _padded(M, N, out) if case["keep"] else None
    elif op == "dgrad":
        s["dY"] = normal(M, N, dt, 1.0)
        s["W"] = normal(N, K, dt, N ** -0.5)
        s["Z"] = normal(M, K, dt, 1.0)
        s["dX"] = _padded(M, K, dt)
        s["dbias"] = torch.empty(K, dtype=torch.float32, device="cuda")
    elif op == "wgrad":
        s["dY"] = normal(M, N, dt, M ** -0.5)
        s["X"] = normal(M, K, dt, 1.0)
        out = DTYPES[case["out"]]
        s["dW"] = normal(N, K, out, 1.0) if case["accumulate"] else _padded(N, K, out)
    else:
        s["dY"] = normal(M, N, dt, 1.0)
        s["Z"] = normal(M, N, dt, 1.0)
        s["dZ"] = _padded(M, N, dt)
        s["dbias"] = torch.empty(N, dtype=torch.float32, device="cuda")
    return s


_native = None


def _library():
    global _native
    if _native is None:
        from dense_tiled_gemm_04_gb300 import native
        _native = native
    return _native


def run(s):
    op = s["op"]
    if own:
        lib = _library()
        if op == "linear":
            Y = lib.linear(s["X"], s["W"], s["bias_t"], act=s["act"], residual=s["residual_t"], out=s["Y"], preact=s["Z"],
                           alpha=s["alpha"])
            return {"Y": Y, "Z": s["Z"]} if s["keep"] else {"Y": Y}
        if op == "dgrad":
            dX = lib.linear_dgrad(s["dY"], s["W"], s["Z"], act=s["act"], out=s["dX"], dbias=s["dbias"])
            return {"dX": dX, "dbias": s["dbias"]}
        if op == "wgrad":
            return {"dW": lib.linear_wgrad(s["dY"], s["X"], out=s["dW"], beta=1.0 if s["accumulate"] else 0.0)}
        dZ = lib.act_grad(s["dY"], s["Z"], act=s["act"], out=s["dZ"], dbias=s["dbias"])
        return {"dZ": dZ, "dbias": s["dbias"]}
    if op == "linear":
        out = DTYPES[s["out"]]
        z = s["X"].float() @ s["W"].float().t()
        if s["alpha"] != 1.0:
            z = z * s["alpha"]
        if s["bias_t"] is not None:
            z = z + s["bias_t"].float()
        y = _act(z, s["act"])
        if s["residual_t"] is not None:
            y = y + s["residual_t"].float()
        return {"Y": y.to(out), "Z": z.to(out)} if s["keep"] else {"Y": y.to(out)}
    if op == "dgrad":
        d = (s["dY"].float() @ s["W"].float()) * _act_slope(s["Z"].float(), s["act"])
        return {"dX": d.to(s["dX"].dtype), "dbias": d.sum(0)}
    if op == "wgrad":
        d = s["dY"].float().t() @ s["X"].float()
        if s["accumulate"]:
            return {"dW": s["dW"].add_(d)}
        return {"dW": d.to(s["dW"].dtype)}
    d = s["dY"].float() * _act_slope(s["Z"].float(), s["act"])
    return {"dZ": d.to(s["dZ"].dtype), "dbias": d.sum(0)}


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * SQRT_HALF))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(SQRT_2_PI * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * SQRT_HALF)) + z * (INV_SQRT_2PI * torch.exp(-0.5 * z * z))
    if act == "gelu_tanh":
        t = torch.tanh(SQRT_2_PI * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * (SQRT_2_PI * (1 + 3 * 0.044715 * z * z))
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def work(case):
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    size = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}
    e = size[case["dtype"]]
    if op == "linear":
        o = size[case["out"]]
        return {"bytes": e * (M * K + N * K) + o * (M * N * (1 + case["residual"] + case["keep"]) + N * case["bias"]),
                "flops": 2 * M * N * K}
    if op == "dgrad":
        return {"bytes": e * (M * N + N * K + 2 * M * K) + 4 * K, "flops": 2 * M * N * K}
    if op == "wgrad":
        return {"bytes": e * (M * N + M * K) + size[case["out"]] * N * K * (2 if case["accumulate"] else 1),
                "flops": 2 * M * N * K}
    return {"bytes": 3 * e * M * N + 4 * N, "flops": 10 * M * N}


def exact(case, seed):
    """The outputs in fp64, from the definitions: Phi and phi are the normal distribution and its density, sigma the
    logistic function, and gelu_tanh(z) = z sigma(2u), u = sqrt(2/pi) (z + 0.044715 z^3)."""
    s = prepare(case, seed)
    op, act = case["op"], case.get("act", "none")
    d64 = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("Y", "dX", "dZ", "dbias")}

    def value(z):
        return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "gelu": lambda: z * torch.special.ndtr(z),
                "gelu_tanh": lambda: z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)),
                "silu": lambda: z * torch.sigmoid(z)}[act]()

    def slope(z):
        z = z.detach().requires_grad_(True)
        with torch.enable_grad():
            if act == "relu":
                return (z.detach() > 0).double()
            return torch.autograd.grad(value(z).sum(), z)[0] if act != "none" else torch.ones_like(z)

    if op == "linear":
        z = torch.matmul(d64["X"], d64["W"].t()).mul_(s["alpha"])
        if case["bias"]:
            z += d64["bias_t"]
        y = value(z)
        if case["residual"]:
            y = y + d64["residual_t"]
        return {"Y": y, "Z": z} if case["keep"] else {"Y": y}
    if op == "wgrad":
        d = torch.matmul(d64["dY"].t(), d64["X"])
        return {"dW": d + d64["dW"] if case["accumulate"] else d}
    g = torch.matmul(d64["dY"], d64["W"]) if op == "dgrad" else d64["dY"]
    g = g * slope(d64["Z"])
    return {"dX" if op == "dgrad" else "dZ": g, "dbias": g.sum(0)}
