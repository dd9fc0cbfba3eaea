"""The measured cases of the operators around the routed FFN: routing with its
gradient, the norms at a block's two ends with theirs, and the linear layer with
a fused epilogue and its gradient.  Each case has a plain form in elementary
torch operations and, where `own` is set, the library's entry points."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
DEV = "cuda"


# ------------------------------------------------------------------------- cases
def _route(T, E, k, score, renorm, bias, n_group, topk_group, group_best, scale, dtype, masked, backward):
    return dict(op="route_backward" if backward else "route", T=T, E=E, k=k, score=score, renorm=renorm, bias=bias,
                n_group=n_group, topk_group=topk_group, group_best=group_best, scale=scale, dtype=dtype,
                masked=masked)


def _norm(T, H, kind, post, pre, gate, h_dtype, o_dtype, w_dtype, bias, alpha, beta, backward):
    return dict(op="norm_backward" if backward else "norm", T=T, H=H, kind=kind, post=post, pre=pre, gate=gate,
                h_dtype=h_dtype, o_dtype=o_dtype, w_dtype=w_dtype, bias=bias, alpha=alpha, beta=beta)


def _linear(M, N, K, act, dtype, out_dtype, bias, residual, keep_z, alpha, backward):
    return dict(op="linear_backward" if backward else "linear", M=M, N=N, K=K, act=act, dtype=dtype,
                out_dtype=out_dtype, bias=bias, residual=residual, keep_z=keep_z, alpha=alpha)


def listed():
    return [
        # one decode step of a small batch: the router between two layers, all latency
        dict(name="route decode", **_route(8, 192, 8, "softmax", True, False, 1, 1, 1, 1.0, "f32", False, False)),
        # a prefill's tokens through a balanced router: biased selection inside the best expert groups, with
        # experts taken out of service and padding tokens masked
        dict(name="route prefill grouped",
             **_route(16384, 128, 8, "sigmoid", True, True, 8, 4, 2, 2.0, "f32", True, False)),
        # a training step's router gradient, every expert's probability in the softmax
        dict(name="route train", **_route(16384, 128, 8, "softmax", False, False, 1, 1, 1, 1.0, "f32", False, True)),
        # the boundary between two blocks in one decode step
        dict(name="norm decode", **_norm(8, 4096, "rms", True, True, "none", "bf16", "bf16", "bf16", False, 1.0, 1.0, False)),
        # the same boundary for a prefill, with a learned per-channel gate on the block's output
        dict(name="norm prefill",
             **_norm(16384, 2048, "rms", True, True, "channel", "bf16", "bf16", "f32", False, 1.0, 1.0, False)),
        # its gradient in a training step
        dict(name="norm train", **_norm(16384, 2048, "rms", True, True, "channel", "bf16", "bf16", "f32", False, 1.0, 1.0, True)),
        # layer norms with biases and a gate per token in full precision, sizes that nothing divides
        dict(name="norm train odd", **_norm(4099, 1023, "layer", True, True, "token", "f32", "f32", "f32", True, 0.5, 0.9, True)),
        # a projection back into the residual stream in one decode step: bound by reading the weights
        dict(name="linear decode", **_linear(8, 4096, 4096, "none", "bf16", "bf16", False, True, False, 1.0, False)),
        # the router's logits for a prefill: few columns, unrounded output
        dict(name="linear router", **_linear(16384, 128, 2048, "none", "bf16", "f32", True, False, False, 1.0, False)),
        # the first half of a dense FFN in training: the pre-activation is kept
        dict(name="linear ffn", **_linear(16384, 8192, 2048, "gelu", "bf16", "bf16", True, False, True, 1.0, False)),
        # the router's gradient: a long sum over tokens for a small weight
        dict(name="linear router train", **_linear(16384, 128, 2048, "none", "bf16", "bf16", False, False, False, 1.0, True)),
        # the dense FFN's gradient, a token count that no tile divides
        dict(name="linear ffn train", **_linear(8191, 4096, 2048, "silu", "f16", "f16", True, False, True, 1.0, True)),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "norm", "linear"])
    backward = rng.random() < 0.5
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * _log(rng, 4, 512 // n_group)
        topk_group = rng.randint(1, n_group)
        k = _log(rng, 2 if backward else 1, min(32, E // n_group * topk_group))  # one renormalised weight is constant
        score = rng.choice(["softmax", "sigmoid"])
        return _route(_log(rng, 1, 16384), E, k, score, rng.random() < 0.7, rng.random() < 0.5, n_group, topk_group,
                      rng.choice([1, 2]), rng.choice([1.0, 1.5, 2.0]), rng.choice(["f32", "f32", "bf16", "f16"]),
                      rng.random() < 0.4, backward)
    if op == "norm":
        H = _log(rng, 33, 8192)
        if rng.random() < 0.7:
            H = (H + 7) // 8 * 8
        T = _log(rng, 1, min(32768, (1 << 25) // H))
        h, o = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("f32", "f32")])
        post = rng.random() < 0.7
        pre = True if not post else rng.random() < 0.8
        return _norm(T, H, rng.choice(["rms", "rms", "layer"]), post, pre, rng.choice(["none", "channel", "token", "full"]),
                     h, o, rng.choice(["f32", o]), rng.random() < 0.5, rng.choice([1.0, 0.5, 0.22]), rng.choice([1.0, 0.9]),
                     backward)
    K = 8 * _log(rng, 8, 512)
    N = _log(rng, 8, 8192)
    M = _log(rng, 1, min(16384, (1 << (37 if backward else 38)) // (N * K)))
    act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    # a gradient comes in the layer's own type
    out = dtype if backward else rng.choice([dtype, dtype, "f32"])
    return _linear(M, N, K, act, dtype, out, rng.random() < 0.6, rng.random() < 0.5 and not backward,
                   act != "none" and (backward or rng.random() < 0.5), rng.choice([1.0, 1.0, 0.5]), backward)


# ------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _choice64(s, bias, c):
    """Keys, group sums and the keys of the groups that stay, in 64 bits."""
    T, E, G = c["T"], c["E"], c["n_group"]
    x = s.double()
    p = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    p = torch.nan_to_num(p, nan=0.0)  # a row that is masked as a whole
    live = x > -math.inf
    by_score = bias is None
    key = torch.where(live, x if by_score else p + bias.double(), -math.inf)
    rank = None
    kept = key
    if G > 1:
        pk = torch.where(live, p if by_score else key, -math.inf).view(T, G, E // G)
        if c["group_best"] == 1:
            rank = key.view(T, G, E // G).amax(2)
        else:
            two = pk.sort(2, descending=True).values[:, :, :2]
            rank = torch.where(two > -math.inf, two, 0.0).sum(2)
            rank = torch.where(two[:, :, 0] > -math.inf, rank, -math.inf)
        best = rank.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device=s.device).scatter_(1, best, True)
        kept = torch.where(stays.repeat_interleave(E // G, 1), key, -math.inf)
        kept = torch.where(stays.repeat_interleave(E // G, 1) & ~live, torch.finfo(torch.float64).min, kept)
    return p, key, rank, kept


def _near(v, n):
    """Rows whose first n + 1 largest values hold two that differ, but by less than 32-bit sums resolve."""
    v = v.sort(1, descending=True).values[:, :n + 1]
    gap = v[:, :-1] - v[:, 1:]
    return ((gap < 2e-6) & (v[:, 1:] > -1e30)).any(1) if v.shape[1] > 1 else torch.zeros(len(v), dtype=torch.bool, device=v.device)


def _scores(c, seed):
    """Router scores with unequal popularity, and the balancing bias.  Where the order is one of computed
    keys (a bias, or sums of two), the few rows whose order hangs on the last bits are drawn again, so that
    the selection does not depend on how a key was rounded."""
    g = _gen(seed)
    T, E = c["T"], c["E"]
    dt = DTYPES[c["dtype"]]
    popular = 0.5 * _randn(g, E)
    bias = 0.1 * _randn(g, E) if c["bias"] else None
    off = torch.zeros(E, dtype=torch.bool, device=DEV)
    pad = torch.zeros(T, dtype=torch.bool, device=DEV)
    if c["masked"]:
        off = torch.rand(E, generator=g, device=DEV) < 0.05
        pad = torch.rand(T, generator=g, device=DEV) < 0.02
        off[0] = False

    def fresh():
        s = (_randn(g, T, E) + popular).to(dt)
        return s.masked_fill(off, -math.inf).masked_fill(pad[:, None], -math.inf)

    s = fresh()
    if bias is not None or (c["n_group"] > 1 and c["group_best"] == 2):
        for _ in range(5):
            _, _, rank, kept = _choice64(s, bias, c)
            bad = _near(kept, c["k"]) if bias is not None else torch.zeros(T, dtype=torch.bool, device=DEV)
            if rank is not None and c["group_best"] == 2:
                bad = bad | _near(rank, c["topk_group"])
            s = torch.where(bad[:, None], fresh(), s)
    return s.contiguous(), bias


def _param(g, n, dt, mean):
    return (mean + 0.2 * _randn(g, n)).to(dt)


def _inputs(c, seed):
    if c["op"].startswith("route"):
        s, bias = _scores(c, seed)
        st = {"scores": s, "bias": bias}
        if c["op"] == "route_backward":
            g = _gen(seed + (1 << 40))
            _, _, _, kept = _choice64(s, bias, c)
            st["ids"] = kept.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]].int().contiguous()
            st["dw"] = _randn(g, c["T"], c["k"])
        return st
    g = _gen(seed)
    if c["op"].startswith("norm"):
        T, H = c["T"], c["H"]
        ht, ot, wt = DTYPES[c["h_dtype"]], DTYPES[c["o_dtype"]], DTYPES[c["w_dtype"]]
        st = {"h": (2.0 * _randn(g, T, H)).to(ht), "o": (0.3 * _randn(g, T, H) + 0.05).to(ot)}
        st["w_post"] = _param(g, H, wt, 1.0) if c["post"] else None
        st["w_pre"] = _param(g, H, wt, 1.0) if c["pre"] else None
        st["b_post"] = _param(g, H, wt, 0.0) if c["post"] and c["bias"] else None
        st["b_pre"] = _param(g, H, wt, 0.0) if c["pre"] and c["bias"] else None
        st["gate"] = {"none": lambda: None, "channel": lambda: _param(g, H, wt, 0.5),
                      "token": lambda: torch.sigmoid(_randn(g, T)),
                      "full": lambda: (0.5 * _randn(g, T, H)).to(ot)}[c["gate"]]()
        if c["op"] == "norm_backward":
            st["dh_out"] = _randn(g, T, H).to(ht)
            st["dx_out"] = _randn(g, T, H).to(ot) if c["pre"] else None
            del st["h"]
            st["h_out"] = (2.0 * _randn(g, T, H)).to(ht)
        return st
    M, N, K = c["M"], c["N"], c["K"]
    dt, yt = DTYPES[c["dtype"]], DTYPES[c["out_dtype"]]
    st = {"x": _randn(g, M, K).to(dt), "w": (_randn(g, N, K) / math.sqrt(K)).to(dt)}
    if c["op"] == "linear":
        st["bias"] = 0.1 * _randn(g, N) if c["bias"] else None
        st["residual"] = _randn(g, M, N).to(yt) if c["residual"] else None
    else:
        st["dy"] = (0.1 * _randn(g, M, N)).to(yt)
        st["z"] = _randn(g, M, N).to(dt) if c["act"] != "none" else None
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:  # the descriptors, outputs and workspace that a program allocates once
        import mixture_experts_layer_index_gb300 as m

        c = case
        dt = {"f32": m.MOE_DTYPE_F32, "bf16": m.MOE_DTYPE_BF16, "f16": m.MOE_DTYPE_F16}

        def empty(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=DEV)

        st["m"] = m
        if c["op"].startswith("route"):
            st["opt"] = m.route_options(score=c["score"], bias=st["bias"], n_group=c["n_group"], topk_group=c["topk_group"],
                                        group_best=c["group_best"], renormalise=c["renorm"], scale=c["scale"],
                                        dtype=dt[c["dtype"]])
            if c["op"] == "route":
                st["out"] = (empty(c["T"], c["k"], dtype=torch.int32), empty(c["T"], c["k"]))
            else:
                st["out"] = empty(c["T"], c["E"], dtype=DTYPES[c["dtype"]])
        elif c["op"].startswith("norm"):
            T, H = c["T"], c["H"]
            ht, ot = DTYPES[c["h_dtype"]], DTYPES[c["o_dtype"]]
            kind = {"rms": m.MOE_NORM_RMS, "layer": m.MOE_NORM_LAYER}[c["kind"]]
            gate = {"none": m.MOE_GATE_NONE, "channel": m.MOE_GATE_CHANNEL, "token": m.MOE_GATE_TOKEN, "full": m.MOE_GATE_FULL}
            st["p"] = m.norm_problem(T, H, post_norm=kind if c["post"] else m.MOE_NORM_NONE,
                                     pre_norm=kind if c["pre"] else m.MOE_NORM_NONE, gate=gate[c["gate"]],
                                     h_dtype=dt[c["h_dtype"]], o_dtype=dt[c["o_dtype"]], w_dtype=dt[c["w_dtype"]],
                                     eps=1e-6, alpha=c["alpha"], beta=c["beta"])
            if c["op"] == "norm":
                st["out"] = (empty(T, H, dtype=ht), empty(T, H, dtype=ot) if c["pre"] else None)
            else:
                dgate = {"none": lambda: None, "channel": lambda: empty(H), "token": lambda: empty(T),
                         "full": lambda: empty(T, H, dtype=ot)}[c["gate"]]()
                st["out"] = dict(dh=empty(T, H, dtype=ht), do=empty(T, H, dtype=ot), dgate=dgate,
                                 dw_post=empty(H) if c["post"] else None,
                                 db_post=empty(H) if c["post"] and c["bias"] else None,
                                 dw_pre=empty(H) if c["pre"] else None,
                                 db_pre=empty(H) if c["pre"] and c["bias"] else None)
                st["ws"] = torch.empty(m.moe_norm_backward_workspace_size(st["p"]), dtype=torch.uint8, device=DEV)
        else:
            M, N, K = c["M"], c["N"], c["K"]
            act = {"none": m.MOE_ACT_NONE, "relu": m.MOE_ACT_RELU, "silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU,
                   "gelu_tanh": m.MOE_ACT_GELU_TANH}[c["act"]]
            st["p"] = m.linear_problem(M, N, K, dtype=dt[c["dtype"]], out_dtype=dt[c["out_dtype"]],
                                       bias_dtype=m.MOE_DTYPE_F32, act=act, alpha=c["alpha"])
            ct = DTYPES[c["dtype"]]
            if c["op"] == "linear":
                st["out"] = (empty(M, N, dtype=DTYPES[c["out_dtype"]]), empty(M, N, dtype=ct) if c["keep_z"] else None)
                st["ws"] = torch.empty(m.moe_linear_workspace_size(st["p"]), dtype=torch.uint8, device=DEV)
            else:
                st["out"] = (empty(M, K, dtype=ct), empty(N, K, dtype=ct), empty(N) if c["bias"] else None)
                st["ws"] = torch.empty(m.moe_linear_backward_workspace_size(st["p"]), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------- plain forms
def _plain_p(s, c):
    live = s > -math.inf
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-s)), live
    top = torch.where(live, s, torch.finfo(torch.float32).min).amax(1, keepdim=True)
    e = torch.where(live, torch.exp(s - top), 0.0)
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0), live


def _plain_weights(p_sel, c):
    if not c["renorm"]:
        return p_sel * c["scale"]
    total = p_sel.sum(1, keepdim=True)
    return torch.where(total > 0, p_sel / total, 0.0) * c["scale"]


def _plain_route(st, c):
    T, E, G = c["T"], c["E"], c["n_group"]
    s = st["scores"].float()
    p, live = _plain_p(s, c)
    least = torch.finfo(torch.float32).min
    key = s + 0.0 if st["bias"] is None else p + st["bias"]
    key = torch.where(live, key, least)
    if G > 1:
        if c["group_best"] == 1:
            rank = key.view(T, G, E // G).amax(2)
        else:
            pk = key if st["bias"] is not None else torch.where(live, p, least)
            two = torch.sort(pk.view(T, G, E // G), dim=2, descending=True).values[:, :, :2]
            rank = torch.where(two[:, :, 0] > least, torch.where(two > least, two, 0.0).sum(2), least)
        best = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device=s.device)
        stays.scatter_(1, best, True)
        key = torch.where(stays.repeat_interleave(E // G, 1), key, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    return ids.int(), _plain_weights(p.gather(1, ids), c)


def _plain_route_backward(st, c):
    s = st["scores"].float()
    ids, dw, scale = st["ids"].long(), st["dw"], c["scale"]
    p, _ = _plain_p(s, c)
    ps = p.gather(1, ids)
    if c["renorm"]:
        total = ps.sum(1, keepdim=True)
        r = torch.where(total > 0, ps / total, 0.0)
        centred = scale * (dw - (dw * r).sum(1, keepdim=True))
        if c["score"] == "softmax":
            d = r * centred
        else:
            d = r * centred * (1.0 - ps)
        ds = torch.zeros_like(s).scatter_(1, ids, d)
    elif c["score"] == "sigmoid":
        ds = torch.zeros_like(s).scatter_(1, ids, scale * dw * ps * (1.0 - ps))
    else:
        g = torch.zeros_like(s).scatter_(1, ids, scale * dw)
        ds = p * (g - (scale * dw * ps).sum(1, keepdim=True))
    return ds.to(st["scores"].dtype)


def _stats(v, kind):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    return v * (1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6))


def _scaled(n, w, b):
    n = n if w is None else n * w.float()
    return n if b is None else n + b.float()


def _gate(st, c):
    if st["gate"] is None:
        return None
    g = st["gate"].float()
    return g[:, None] if c["gate"] == "token" else g


def _plain_norm(st, c):
    n = st["o"].float()
    if c["post"]:
        n = _scaled(_stats(n, c["kind"]), st["w_post"], st["b_post"])
    g = _gate(st, c)
    h = c["beta"] * st["h"].float() + c["alpha"] * (n if g is None else n * g)
    x = _scaled(_stats(h, c["kind"]), st["w_pre"], st["b_pre"]).to(st["o"].dtype) if c["pre"] else None
    return h.to(st["h"].dtype), x


def _plain_norm_grad(v, dn, kind):
    """Gradient into v of its normalised value, given dn: r (dn - n mean(dn n) [- mean(dn)])."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    n = v * r
    d = dn - n * (dn * n).mean(1, keepdim=True)
    if kind == "layer":
        d = d - dn.mean(1, keepdim=True)
    return r * d, n


def _plain_norm_backward(st, c):
    kind = c["kind"]
    out = dict(dh=None, do=None, dgate=None, dw_post=None, db_post=None, dw_pre=None, db_pre=None)
    G = st["dh_out"].float()
    if c["pre"]:
        dx = st["dx_out"].float()
        d, n = _plain_norm_grad(st["h_out"].float(), dx * st["w_pre"].float(), kind)
        G = G + d
        out["dw_pre"] = (dx * n).sum(0)
        if c["bias"]:
            out["db_pre"] = dx.sum(0)
    out["dh"] = (c["beta"] * G).to(st["h_out"].dtype)
    o = st["o"].float()
    g = _gate(st, c)
    dn = c["alpha"] * (G if g is None else G * g)
    n = o
    if c["post"]:
        do, unit = _plain_norm_grad(o, dn * st["w_post"].float(), kind)
        out["dw_post"] = (dn * unit).sum(0)
        if c["bias"]:
            out["db_post"] = dn.sum(0)
        n = _scaled(unit, st["w_post"], st["b_post"])
    else:
        do = dn
    out["do"] = do.to(st["o"].dtype)
    if g is not None:
        t = c["alpha"] * G * n
        out["dgate"] = {"channel": lambda: t.sum(0), "token": lambda: t.sum(1), "full": lambda: t.to(st["o"].dtype)}[c["gate"]]()
    return out


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


def _plain_linear(st, c):
    z = torch.matmul(st["x"].float(), st["w"].float().t())
    if st["bias"] is not None:
        z = z + st["bias"]
    y = c["alpha"] * _plain_act(z, c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(DTYPES[c["out_dtype"]]), z.to(st["x"].dtype) if c["keep_z"] else None


def _plain_linear_backward(st, c):
    dz = c["alpha"] * st["dy"].float()
    if c["act"] != "none":
        dz = dz * _plain_act_grad(st["z"].float(), c["act"])
    dx = torch.matmul(dz, st["w"].float())
    dw = torch.matmul(dz.t(), st["x"].float())
    return dx.to(st["x"].dtype), dw.to(st["w"].dtype), dz.sum(0) if c["bias"] else None


PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "norm": _plain_norm,
         "norm_backward": _plain_norm_backward, "linear": _plain_linear, "linear_backward": _plain_linear_backward}


# ------------------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        return PLAIN[op](st, c)
    m, out = st["m"], st["out"]
    if op == "route":
        m.moe_route_ex(st["opt"], st["scores"], c["T"], c["E"], c["k"], out[0], out[1])
    elif op == "route_backward":
        m.moe_route_backward(st["opt"], st["scores"], c["T"], c["E"], c["k"], st["ids"], st["dw"], out)
    elif op == "norm":
        m.moe_norm_forward(st["p"], st["h"], st["o"], st["gate"], st["w_post"], st["b_post"], st["w_pre"], st["b_pre"],
                           out[0], out[1])
    elif op == "norm_backward":
        m.moe_norm_backward(st["p"], st["dh_out"], st["dx_out"], st["h_out"], st["o"], st["gate"], st["w_post"],
                            st["b_post"], st["w_pre"], out["dh"], out["do"], out["dgate"], out["dw_post"],
                            out["db_post"], out["dw_pre"], out["db_pre"], st["ws"])
    elif op == "linear":
        m.moe_linear(st["p"], st["x"], st["w"], st["bias"], st["residual"], out[0], out[1], st["ws"])
    else:
        m.moe_linear_backward(st["p"], st["dy"], st["x"], st["w"], st["z"], out[0], out[1], out[2], st["ws"])
    return out


# ------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits; gradients by differentiating them."""
    c, st = case, _inputs(case, seed)
    if c["op"].startswith("route"):
        p, _, _, kept = _choice64(st["scores"], st["bias"], c)
        if c["op"] == "route":
            ids = kept.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
            w = p.gather(1, ids)
            if c["renorm"]:
                w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
            return ids.int(), w * c["scale"]
        s = st["scores"].double()
        dead = (s == -math.inf).all(1, keepdim=True)
        s = torch.where(dead, 0.0, s).requires_grad_()
        q = torch.softmax(s, 1) if c["score"] == "softmax" else torch.sigmoid(s)
        w = q.gather(1, st["ids"].long())
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        (c["scale"] * w * st["dw"].double()).sum().backward()
        return torch.where(dead, 0.0, s.grad)

    def norm(v, w, b):
        if c["kind"] == "layer":
            v = v - v.mean(1, keepdim=True)
        v = v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()
        v = v if w is None else v * w
        return v if b is None else v + b

    d = {k: (v.double() if torch.is_tensor(v) else v) for k, v in st.items()}
    if c["op"].startswith("norm"):
        back = c["op"] == "norm_backward"
        if back:
            for name in ("o", "gate", "w_post", "b_post", "w_pre", "b_pre", "h_out"):
                if d[name] is not None:
                    d[name].requires_grad_()
        n = norm(d["o"], d["w_post"], d["b_post"]) if c["post"] else d["o"]
        if d["gate"] is not None:
            n = n * (d["gate"][:, None] if c["gate"] == "token" else d["gate"])
        if not back:
            h = c["beta"] * d["h"] + c["alpha"] * n
            return h, norm(h, d["w_pre"], d["b_pre"]) if c["pre"] else None
        G = d["dh_out"]
        if c["pre"]:
            (norm(d["h_out"], d["w_pre"], d["b_pre"]) * d["dx_out"]).sum().backward()
            G = G + d["h_out"].grad
        (c["alpha"] * n * G).sum().backward()

        def grad(t):
            return None if t is None else t.grad

        return dict(dh=c["beta"] * G, do=d["o"].grad, dgate=grad(d["gate"]), dw_post=grad(d["w_post"]),
                    db_post=grad(d["b_post"]), dw_pre=grad(d["w_pre"]), db_pre=grad(d["b_pre"]))

    def act(z):
        return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
                "gelu": lambda: torch.nn.functional.gelu(z),
                "gelu_tanh": lambda: torch.nn.functional.gelu(z, approximate="tanh")}[c["act"]]()

    if c["op"] == "linear":
        z = d["x"] @ d["w"].t()
        z = z if d["bias"] is None else z + d["bias"]
        y = c["alpha"] * act(z)
        return y if d["residual"] is None else y + d["residual"], z if c["keep_z"] else None
    z = (torch.zeros_like(d["dy"]) if d["z"] is None else d["z"]).requires_grad_()
    (c["alpha"] * act(z) * d["dy"]).sum().backward()
    dz = z.grad
    return dz @ d["w"], dz.t() @ d["x"], dz.sum(0) if c["bias"] else None


# ------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"].startswith("route"):
        T, E, k, b = c["T"], c["E"], c["k"], BYTES[c["dtype"]]
        if c["op"] == "route":
            return {"bytes": T * E * b + T * k * 8 + (4 * E if c["bias"] else 0), "flops": 4 * T * E}
        whole = c["score"] == "softmax" and not c["renorm"]  # else the scores of the chosen experts suffice
        return {"bytes": T * E * b + T * (E if whole else k) * b + T * k * 8, "flops": 4 * T * (E if whole else k)}
    if c["op"].startswith("norm"):
        T, H = c["T"], c["H"]
        h, o, w = BYTES[c["h_dtype"]], BYTES[c["o_dtype"]], BYTES[c["w_dtype"]]
        gate = {"none": 0, "channel": w * H, "token": 4 * T, "full": o * T * H}[c["gate"]]
        vectors = (c["post"] + c["pre"]) * H * (2 if c["bias"] else 1)
        if c["op"] == "norm":
            return {"bytes": T * H * (2 * h + o + (o if c["pre"] else 0)) + gate + vectors * w,
                    "flops": 12 * T * H}
        dgate = {"none": 0, "channel": 4 * H, "token": 4 * T, "full": o * T * H}[c["gate"]]
        read = T * H * (h + o + ((h + o) if c["pre"] else 0))
        return {"bytes": read + T * H * (h + o) + gate + dgate + vectors * (w + 4), "flops": 30 * T * H}
    M, N, K, b, y = c["M"], c["N"], c["K"], BYTES[c["dtype"]], BYTES[c["out_dtype"]]
    if c["op"] == "linear":
        n = b * (M * K + N * K) + y * M * N + (4 * N if c["bias"] else 0)
        return {"bytes": n + (y * M * N if c["residual"] else 0) + (b * M * N if c["keep_z"] else 0), "flops": 2 * M * N * K}
    n = 2 * b * (M * K + N * K) + y * M * N + (b * M * N if c["act"] != "none" else 0) + (4 * N if c["bias"] else 0)
    return {"bytes": n, "flops": 4 * M * N * K}
