"""The measured cases of the dense blocks' operators: the gated linear layer and its
gradient, quantisation in blocks of 128, and the linear and the gated layer on e4m3
operands with block scales.  Each case has a plain form in elementary torch operations
and, where `own` is set, the library's entry points."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
DEV = "cuda"
GROUP = 128  # values that share a scale


# ------------------------------------------------------------------------- cases
def _gated(M, N, K, act, dtype, out_dtype, bias, keep_z):
    return dict(op="gated", M=M, N=N, K=K, act=act, dtype=dtype, out_dtype=out_dtype, bias=bias, keep_z=keep_z)


def _gated_backward(M, N, K, act, dtype, bias):
    return dict(op="gated_backward", M=M, N=N, K=K, act=act, dtype=dtype, out_dtype=dtype, bias=bias)


def _quantise(M, K, dtype, block_rows):
    return dict(op="quantise", M=M, K=K, dtype=dtype, block_rows=block_rows)


def _linear_fp8(M, N, K, act, out_dtype, bias, residual, alpha):
    return dict(op="linear_fp8", M=M, N=N, K=K, act=act, out_dtype=out_dtype, bias=bias, residual=residual, alpha=alpha)


def _gated_fp8(M, N, K, act, out_dtype, bias):
    return dict(op="gated_fp8", M=M, N=N, K=K, act=act, out_dtype=out_dtype, bias=bias)


def listed():
    return [
        # a dense block's first half in one decode step of a small batch: bound by reading the weights
        dict(name="gated decode", **_gated(8, 4096, 4096, "silu", "bf16", "bf16", False, False)),
        # the same for a prefill's tokens
        dict(name="gated prefill", **_gated(16384, 4096, 2048, "silu", "bf16", "bf16", False, False)),
        # a training step's forward in half precision, sizes that no tile divides, rows at odd addresses
        dict(name="gated train odd", **_gated(8191, 2730, 2048, "gelu_tanh", "f16", "f16", True, True)),
        # its gradient at the prefill's size
        dict(name="gated gradient", **_gated_backward(16384, 4096, 2048, "silu", "bf16", False)),
        # a small layer's gradient, nothing divides
        dict(name="gated gradient odd", **_gated_backward(517, 1366, 1000, "gelu", "f16", True)),
        # a prefill's activations on their way into an FP8 layer
        dict(name="quantise tokens", **_quantise(16384, 2048, "bf16", 1)),
        # a weight matrix after an optimizer's step, in full precision
        dict(name="quantise weights", **_quantise(8192, 4096, "f32", 128)),
        # a projection back into the residual stream in one decode step
        dict(name="fp8 linear decode", **_linear_fp8(8, 4096, 4096, "none", "bf16", False, True, 1.0)),
        # a dense block's second half for a prefill
        dict(name="fp8 linear prefill", **_linear_fp8(16384, 2048, 4096, "none", "bf16", False, True, 1.0)),
        # ragged in every direction: the last scale group of the sum holds 70 values
        dict(name="fp8 linear odd", **_linear_fp8(1021, 1111, 1990, "gelu", "f32", True, False, 0.5)),
        # a dense block's first half in one decode step, its output ready for the second half
        dict(name="fp8 gated decode", **_gated_fp8(8, 4096, 4096, "silu", "e4m3", False)),
        # the same for a prefill's tokens
        dict(name="fp8 gated prefill", **_gated_fp8(16384, 4096, 2048, "silu", "e4m3", False)),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "gated_backward", "quantise", "linear_fp8", "linear_fp8", "gated_fp8", "gated_fp8"])
    if op == "quantise":
        K = _log(rng, 33, 8192)
        return _quantise(_log(rng, 1, min(16384, (1 << 25) // K)), K, rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice([1, 1, 128]))
    act = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu", "none"])
    bias = rng.random() < 0.4
    N = _log(rng, 8, 4096)
    if op in ("gated", "gated_backward"):
        K = 8 * _log(rng, 8, 512)  # rows that TMA can read
        M = _log(rng, 1, min(16384, (1 << 37) // (N * K)))
        dtype = rng.choice(["bf16", "bf16", "f16"])
        if op == "gated_backward":
            return _gated_backward(M, N, K, act, dtype, bias)
        return _gated(M, N, K, act, dtype, rng.choice([dtype, dtype, "f32"]), bias, rng.random() < 0.5)
    K = _log(rng, 64, 4096)  # rows are padded to whole 16 bytes
    if rng.random() < 0.5:
        K = (K + 127) // 128 * 128
    M = _log(rng, 1, min(16384, (1 << 37) // (N * K)))
    if op == "linear_fp8":
        return _linear_fp8(M, N, K, rng.choice(["none", "none", act]), rng.choice(["bf16", "bf16", "f16", "f32"]), bias,
                           rng.random() < 0.5, rng.choice([1.0, 1.0, 0.5]))
    return _gated_fp8(M, N, K, act, rng.choice(["e4m3", "e4m3", "bf16", "f32"]), bias)


# ------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _groups(v, block_rows):
    """v [M, K] with zeros up to whole blocks, as [M / block_rows, block_rows, K / 128, 128]."""
    M, K = v.shape
    m, k = -(-M // block_rows), -(-K // GROUP)
    full = torch.zeros(m * block_rows, k * GROUP, dtype=v.dtype, device=v.device)
    full[:M, :K] = v
    return full.view(m, block_rows, k, GROUP)


def _plain_quantise(v, block_rows):
    """(codes [M, K] e4m3, scales [M / block_rows, K / 128]) of v: amax / 448 per block, 1 for zeros."""
    M, K = v.shape
    b = _groups(v.float() if v.dtype != torch.float64 else v, block_rows)
    amax = b.abs().amax(dim=(1, 3))
    scale = amax / 448.0
    scale = torch.where(scale > 0, scale, 1.0)
    q = (b / scale[:, None, :, None]).clamp(-448.0, 448.0).reshape(b.shape[0] * block_rows, -1)[:M, :K]
    return q.float().to(torch.float8_e4m3fn).contiguous(), scale


def _values(codes, scale, block_rows, dtype=torch.float32):
    """What codes and scales stand for."""
    M, K = codes.shape
    s = scale.to(dtype).repeat_interleave(block_rows, 0)[:M].repeat_interleave(GROUP, 1)[:, :K]
    return codes.to(dtype) * s


def _padded(codes):
    """The same codes in rows of whole 16 bytes."""
    M, K = codes.shape
    ld = -(-K // 16) * 16
    if ld == K:
        return codes
    full = torch.zeros(M, ld, dtype=torch.uint8, device=codes.device)
    full[:, :K] = codes.view(torch.uint8)
    return full.view(torch.float8_e4m3fn)[:, :K]


def _tokens(g, M, K):
    """Activations: a few channels are an order of magnitude above the others."""
    x = _randn(g, M, K)
    loud = torch.rand(K, generator=g, device=DEV) < 0.01
    return x * torch.where(loud, 8.0, 1.0)


def _inputs(c, seed):
    g = _gen(seed)
    if c["op"] == "quantise":
        v = _tokens(g, c["M"], c["K"])
        if c["block_rows"] == GROUP:
            v = v / math.sqrt(c["K"])
        elif c["M"] > 1:
            v[-1] = 0.0  # a padding token
        return {"x": v.to(DTYPES[c["dtype"]])}
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] in ("gated", "gated_backward"):
        dt = DTYPES[c["dtype"]]
        st = {"x": _randn(g, M, K).to(dt), "w": (_randn(g, 2 * N, K) / math.sqrt(K)).to(dt)}
        if c["op"] == "gated":
            st["bias"] = 0.1 * _randn(g, 2 * N) if c["bias"] else None
        else:
            st["dh"] = (0.1 * _randn(g, M, N)).to(DTYPES[c["out_dtype"]])
            st["z"] = _randn(g, M, 2 * N).to(dt)
        return st
    st = {}
    q, st["x_scale"] = _plain_quantise(_tokens(g, M, K), 1)
    st["x"] = _padded(q)
    parts = 2 if c["op"] == "gated_fp8" else 1  # gate and up rows have scale blocks of their own
    w = [_plain_quantise(_randn(g, N, K) / math.sqrt(K), GROUP) for _ in range(parts)]
    st["w"] = _padded(torch.cat([v[0].view(torch.uint8) for v in w]).view(torch.float8_e4m3fn))
    st["w_scale"] = torch.stack([v[1] for v in w]) if parts == 2 else w[0][1]
    st["bias"] = 0.1 * _randn(g, parts * N) if c["bias"] else None
    if c["op"] == "linear_fp8":
        st["residual"] = _randn(g, M, N).to(DTYPES[c["out_dtype"]]) if c["residual"] else None
    return st


def prepare(case, seed):
    c, st = case, _inputs(case, seed)
    st["case"] = c
    if own:  # the descriptors, outputs and workspace that a program allocates once
        import mixture_experts_layer_index_gb300 as m

        dt = {"f32": m.MOE_DTYPE_F32, "bf16": m.MOE_DTYPE_BF16, "f16": m.MOE_DTYPE_F16, "e4m3": m.MOE_DTYPE_E4M3}
        acts = {"none": m.MOE_ACT_NONE, "relu": m.MOE_ACT_RELU, "silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU,
                "gelu_tanh": m.MOE_ACT_GELU_TANH}

        def empty(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=DEV)

        def scratch(n):
            return torch.empty(n, dtype=torch.uint8, device=DEV)

        st["m"] = m
        if c["op"] == "quantise":
            M, K, rows = c["M"], c["K"], c["block_rows"]
            ld = -(-K // 16) * 16
            st["p"] = m.quantise_problem(M, K, dtype=dt[c["dtype"]], block_rows=rows, ld_q=ld)
            codes = empty(M, ld, dtype=torch.uint8)
            st["out"] = (codes.view(torch.float8_e4m3fn)[:, :K], empty(-(-M // rows), -(-K // GROUP)))
            return st
        M, N, K = c["M"], c["N"], c["K"]
        if c["op"] in ("gated", "gated_backward"):
            st["p"] = m.gated_problem(M, N, K, dtype=dt[c["dtype"]], out_dtype=dt[c["out_dtype"]], act=acts[c["act"]])
            ct = DTYPES[c["dtype"]]
            if c["op"] == "gated":
                st["out"] = (empty(M, N, dtype=DTYPES[c["out_dtype"]]), empty(M, 2 * N, dtype=ct) if c["keep_z"] else None)
                st["ws"] = scratch(m.moe_gated_workspace_size(st["p"]))
            else:
                st["out"] = (empty(M, K, dtype=ct), empty(2 * N, K, dtype=ct), empty(2 * N) if c["bias"] else None)
                st["ws"] = scratch(m.moe_gated_backward_workspace_size(st["p"]))
            return st
        ld = -(-K // 16) * 16
        if c["op"] == "linear_fp8":
            st["p"] = m.linear_problem(M, N, K, dtype=dt["e4m3"], out_dtype=dt[c["out_dtype"]], act=acts[c["act"]],
                                       alpha=c["alpha"], ld_x=ld, ld_w=ld)
            st["out"] = empty(M, N, dtype=DTYPES[c["out_dtype"]])
            st["ws"] = scratch(m.moe_linear_fp8_workspace_size(st["p"]))
        else:
            coded = c["out_dtype"] == "e4m3"
            ld_h = -(-N // 16) * 16 if coded else N
            st["p"] = m.gated_problem(M, N, K, dtype=dt["e4m3"], out_dtype=dt[c["out_dtype"]], act=acts[c["act"]],
                                      ld_x=ld, ld_w=ld, ld_h=ld_h)
            h = empty(M, ld_h, dtype=torch.uint8).view(torch.float8_e4m3fn)[:, :N] if coded else empty(M, N, dtype=DTYPES[c["out_dtype"]])
            st["out"] = (h, empty(M, -(-N // GROUP)) if coded else None)
            st["ws"] = scratch(m.moe_gated_fp8_workspace_size(st["p"]))
    return st


# ------------------------------------------------------------------------- plain forms
def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    a = math.sqrt(2.0 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * 0.044715 * z * z)


def _plain_product(x, w, bias):
    z = torch.matmul(x, w.t())
    return z if bias is None else z + bias


def _plain_gated(st, c):
    N = c["N"]
    z = _plain_product(st["x"].float(), st["w"].float(), st["bias"])
    h = _plain_act(z[:, :N], c["act"]) * z[:, N:]
    return h.to(DTYPES[c["out_dtype"]]), z.to(st["x"].dtype) if c["keep_z"] else None


def _plain_gated_backward(st, c):
    N = c["N"]
    g, u = st["z"][:, :N].float(), st["z"][:, N:].float()
    dh = st["dh"].float()
    dz = torch.cat([dh * u * _plain_act_grad(g, c["act"]), dh * _plain_act(g, c["act"])], 1)
    dx = torch.matmul(dz, st["w"].float())
    dw = torch.matmul(dz.t(), st["x"].float())
    return dx.to(st["x"].dtype), dw.to(st["w"].dtype), dz.sum(0) if c["bias"] else None


def _plain_linear_fp8(st, c):
    z = _plain_product(_values(st["x"], st["x_scale"], 1), _values(st["w"], st["w_scale"], GROUP), st["bias"])
    y = c["alpha"] * _plain_act(z, c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(DTYPES[c["out_dtype"]])


def _gated_weights(st, c, dtype=torch.float32):
    N = c["N"]
    return torch.cat([_values(st["w"][:N], st["w_scale"][0], GROUP, dtype), _values(st["w"][N:], st["w_scale"][1], GROUP, dtype)])


def _plain_gated_fp8(st, c):
    N = c["N"]
    z = _plain_product(_values(st["x"], st["x_scale"], 1), _gated_weights(st, c), st["bias"])
    h = _plain_act(z[:, :N], c["act"]) * z[:, N:]
    return _plain_quantise(h, 1) if c["out_dtype"] == "e4m3" else (h.to(DTYPES[c["out_dtype"]]), None)


# ------------------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        if op == "quantise":
            return _plain_quantise(st["x"], c["block_rows"])
        return {"gated": _plain_gated, "gated_backward": _plain_gated_backward, "linear_fp8": _plain_linear_fp8,
                "gated_fp8": _plain_gated_fp8}[op](st, c)
    m, out = st["m"], st["out"]
    if op == "quantise":
        m.moe_quantise(st["p"], st["x"], out[0], out[1])
    elif op == "gated":
        m.moe_gated(st["p"], st["x"], st["w"], st["bias"], out[0], out[1], st["ws"])
    elif op == "gated_backward":
        m.moe_gated_backward(st["p"], st["dh"], st["x"], st["w"], st["z"], out[0], out[1], out[2], st["ws"])
    elif op == "linear_fp8":
        m.moe_linear_fp8(st["p"], st["x"], st["x_scale"], st["w"], st["w_scale"], st["bias"], st["residual"], out, st["ws"])
    else:
        m.moe_gated_fp8(st["p"], st["x"], st["x_scale"], st["w"], st["w_scale"], st["bias"], out[0], out[1], st["ws"])
    return out


# ------------------------------------------------------------------------- 64 bits
def _act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: torch.nn.functional.gelu(z),
            "gelu_tanh": lambda: torch.nn.functional.gelu(z, approximate="tanh")}[act]()


def _codes64(v, block_rows):
    """Codes and scales of v by the definition, block by block along the columns; a code is relative to the
    scale as it is stored, in 32 bits."""
    M, K = v.shape
    scales, codes = [], []
    for k in range(0, K, GROUP):
        part = v[:, k:k + GROUP]
        amax = part.abs().amax(1)
        if block_rows > 1:
            amax = torch.stack([a.amax() for a in amax.split(block_rows)])
        s = torch.where(amax > 0, amax / 448.0, 1.0).float().double()
        scales.append(s)
        codes.append((part / s.repeat_interleave(block_rows)[:M, None]).clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn))
    return torch.cat([q.view(torch.uint8) for q in codes], 1).view(torch.float8_e4m3fn), torch.stack(scales, 1)


def exact(case, seed):
    """The definitions in 64 bits; gradients by differentiating them."""
    c, st = case, _inputs(case, seed)
    if c["op"] == "quantise":
        return _codes64(st["x"].double(), c["block_rows"])
    N, act = c["N"], c["act"]
    if c["op"] == "gated_backward":
        z = st["z"].double().requires_grad_()
        (_act64(z[:, :N], act) * z[:, N:] * st["dh"].double()).sum().backward()
        dz = z.grad
        return dz @ st["w"].double(), dz.t() @ st["x"].double(), dz.sum(0) if c["bias"] else None
    if c["op"] == "gated":
        x, w = st["x"].double(), st["w"].double()
    else:
        x = _values(st["x"], st["x_scale"], 1, torch.float64)
        w = _gated_weights(st, c, torch.float64) if c["op"] == "gated_fp8" else _values(st["w"], st["w_scale"], GROUP, torch.float64)
    z = x @ w.t()
    if st["bias"] is not None:
        z = z + st["bias"].double()
    if c["op"] == "linear_fp8":
        y = c["alpha"] * _act64(z, act)
        return y if st["residual"] is None else y + st["residual"].double()
    h = _act64(z[:, :N], act) * z[:, N:]
    if c["op"] == "gated":
        return h, z if c["keep_z"] else None
    return _codes64(h, 1) if c["out_dtype"] == "e4m3" else (h, None)


# ------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "quantise":
        M, K = c["M"], c["K"]
        scales = -(-M // c["block_rows"]) * -(-K // GROUP)
        return {"bytes": M * K * (BYTES[c["dtype"]] + 1) + 4 * scales, "flops": 3 * M * K}
    M, N, K, y = c["M"], c["N"], c["K"], BYTES[c["out_dtype"]]
    k = -(-K // GROUP)
    if c["op"] == "gated":
        b = BYTES[c["dtype"]]
        n = b * (M * K + 2 * N * K) + y * M * N + (2 * b * M * N if c["keep_z"] else 0) + (8 * N if c["bias"] else 0)
        return {"bytes": n, "flops": 4 * M * N * K}
    if c["op"] == "gated_backward":
        b = BYTES[c["dtype"]]
        return {"bytes": 2 * b * (M * K + 2 * N * K) + 3 * b * M * N + (8 * N if c["bias"] else 0), "flops": 8 * M * N * K}
    parts = 2 if c["op"] == "gated_fp8" else 1
    n = M * K + parts * N * K + 4 * k * (M + parts * -(-N // GROUP)) + y * M * N + (4 * parts * N if c["bias"] else 0)
    if c["op"] == "linear_fp8":
        n += y * M * N if c["residual"] else 0
    elif c["out_dtype"] == "e4m3":
        n += 4 * M * -(-N // GROUP)
    return {"bytes": n, "flops": 2 * parts * M * N * K}
