"""GPU parity of the operators around the routed FFN (routing rules, block norms,
linear layer and their gradients) against oracle/blocks.py in 64 bits.

Bounds on a result v: the rounding to its type, U |v|, and `factor` fp32 roundings
(2^-23 each) of the magnitudes that its sums run over (the oracle's `mag`)."""
import numpy as np
import pytest
import torch

from oracle import blocks as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step at 1: 24, 8 and 11 significant bits
STEP = 2.0 ** -23
NAMES = {v: k for k, v in DT.items()}


@pytest.fixture(scope="module")
def m():
    import __graft_entry__

    __graft_entry__.build()
    import mixture_experts_layer_index_gb300 as mod

    return mod


def code(m, name):
    return {"f32": m.MOE_DTYPE_F32, "bf16": m.MOE_DTYPE_BF16, "f16": m.MOE_DTYPE_F16}[name]


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(got, ref, mag, factor, what="", extra=0.0):
    u = U[NAMES[got.dtype]]
    g = f64(got)
    assert g.shape == np.shape(ref), what
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -126
    bound = (u * np.abs(ref) + (factor * STEP + extra) * mag) * (1 + u) + tiny
    # past the type's largest value the right answer is an infinity, next to it either
    top = float(torch.finfo(got.dtype).max)
    with np.errstate(invalid="ignore"):
        off = np.where(np.isinf(g) & (np.sign(g) == np.sign(ref)) & (np.abs(ref) + bound >= top), 0.0, np.abs(g - ref) - bound)
    g = np.where(off == 0.0, ref, g)
    assert np.all(np.isfinite(g)) and np.all(off <= 0), (what, float(np.max(off)), np.unravel_index(np.argmax(off), off.shape))


def rows(T, W, ld, dtype, gen, scale=1.0, offset=0):
    """[T, W] of ld-strided rows, `offset` elements into its allocation, NaN between the rows."""
    buf = torch.full((T * ld + offset + 8,), float("nan"), device=DEV, dtype=dtype)
    v = buf[offset:offset + T * ld].view(T, ld)[:, :W]
    v.copy_((scale * torch.randn(T, W, generator=gen, device=DEV)).to(dtype))
    return v


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# ----------------------------------------------------------------------------- routing
def _rule(m, dtype="f32", bias=None, **r):
    return m.route_options(score=r.get("score", "softmax"), bias=bias, n_group=r.get("n_group", 1),
                           topk_group=r.get("topk_group", 1), group_best=r.get("group_best", 1),
                           renormalise=r.get("renormalise", True), scale=r.get("scale", 1.0), dtype=code(m, dtype),
                           ld=r.get("ld", 0), ld_grad=r.get("ld_grad", 0))


def _route(m, s, k, dtype="f32", bias=None, **r):
    T, E = s.shape
    ids = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), float("nan"), device=DEV)
    d = torch.full((T, E), float("nan"), dtype=DT[dtype], device=DEV)
    opt = _rule(m, dtype, bias, **r)
    m.moe_route_ex(opt, s, T, E, k, ids, w)
    oracle = {n: v for n, v in r.items() if n not in ("ld", "ld_grad")}
    rid, rw, margin = B.route(f64(s), k, bias=None if bias is None else f64(bias), **oracle)
    # rows whose order hangs on the rounding of a computed key (fp32 sums of a few terms of size up to 2)
    # may be selected either way; they are rare and their ids are still valid and distinct
    sure = margin > 16 * STEP
    got = ids.cpu().numpy()
    assert np.array_equal(got[sure], rid[sure])
    assert np.mean(sure) > 0.98 or T < 50
    assert got.min() >= 0 and got.max() < E
    for row in got:
        assert len(set(row.tolist())) == k
    # exp of fp32 arguments up to 100: relative 100 * 2^-24, sums of at most 512 terms, 32 lanes wide
    wg = f64(w)
    assert np.all(np.abs(wg - rw)[sure] <= 2e-5 * np.abs(rw)[sure] + 1e-37)
    dw = torch.randn(T, k, generator=gen(T + E), device=DEV)
    m.moe_route_backward(opt, s, T, E, k, ids, dw, d)
    ref = B.route_backward(f64(s), got, f64(dw), oracle.get("score", "softmax"), oracle.get("renormalise", True),
                           oracle.get("scale", 1.0))
    p = B.probabilities(f64(s), oracle.get("score", "softmax"))
    scale = abs(oracle.get("scale", 1.0)) * np.abs(f64(dw)).max(axis=1, keepdims=True)
    if oracle.get("renormalise", True):
        sel = np.zeros_like(p)
        np.put_along_axis(sel, got.astype(np.int64), np.where(f64(w) > 0, np.abs(f64(w)), 0.0), 1)
        mag = 2 * scale * sel
    else:
        mag = 2 * scale * p
    off = np.abs(f64(d) - ref) - (U[dtype] * np.abs(ref) + 4e-5 * mag + 1e-37 + (2.0 ** -25 if dtype == "f16" else 0))
    assert np.all(off <= 0), float(np.max(off))
    return ids, w, d


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 192, 8), (3, 33, 33 - 1), (257, 8, 2), (130, 97, 5), (64, 512, 32),
                                   (9, 128, 8), (2, 31, 31)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_rules(m, T, E, k, score, renormalise):
    s = torch.randn(T, E, generator=gen(T * E), device=DEV) * 2
    _route(m, s, k, score=score, renormalise=renormalise, scale=1.5)


@pytest.mark.parametrize("E,n_group,topk_group,k", [(128, 8, 4, 8), (64, 32, 5, 7), (96, 3, 2, 32), (15, 5, 5, 15),
                                                    (512, 2, 1, 8), (36, 12, 1, 3), (7, 7, 3, 3), (256, 16, 16, 1)])
@pytest.mark.parametrize("group_best", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(m, E, n_group, topk_group, k, group_best, biased, score):
    g = gen(E + n_group)
    s = torch.randn(200, E, generator=g, device=DEV)
    bias = 0.2 * torch.randn(E, generator=g, device=DEV) if biased else None
    _route(m, s, k, bias=bias, score=score, n_group=n_group, topk_group=topk_group, group_best=group_best)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_types_and_ties(m, dtype, score):
    # 16-bit scores on a coarse grid: equal scores are common and go to the lower id
    s = (torch.randn(300, 64, generator=gen(4), device=DEV) * 4).round().div(4).to(DT[dtype])
    _route(m, s, 8, dtype, score=score)
    _route(m, s, 8, dtype, score=score, renormalise=False)
    _route(m, s, 8, dtype, score=score, n_group=4, topk_group=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("rule", [dict(), dict(renormalise=False), dict(n_group=4, topk_group=2),
                                  dict(n_group=4, topk_group=2, group_best=2), dict(n_group=4, topk_group=4, group_best=2)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masked_and_extreme_scores(m, score, rule, biased):
    E = 40
    s = torch.randn(64, E, generator=gen(8), device=DEV)
    s[0] = -float("inf")                       # nothing left
    s[1, 3:] = -float("inf")                   # fewer than k left
    s[2, ::2] = float("nan")
    s[3, 5] = float("inf")
    s[4] = torch.finfo(torch.float32).min      # lowest finite: not masked
    s[5, :20] = -float("inf")                  # whole groups masked
    s[6] = -200.0                              # every sigmoid underflows
    s[7] = -0.0
    s[7, 1::2] = 0.0
    s[8, 7] = torch.finfo(torch.float32).max
    s[9] = s[9] * 30
    bias = torch.linspace(-0.3, 0.3, E, device=DEV) if biased else None
    _, w, d = _route(m, s, 6, bias=bias, score=score, scale=2.0, **rule)
    assert torch.all(w[0] == 0) and torch.all(d[0] == 0)
    assert torch.isfinite(w).all() and torch.isfinite(d).all()


def test_route_strides_streams_and_empty(m):
    g = gen(11)
    T, E, k = 77, 50, 5
    s = rows(T, E, 53, torch.float32, g)
    d = torch.full((T, 61), 5.0, device=DEV)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    opt = _rule(m, ld=53, ld_grad=61, renormalise=False)
    dw = torch.randn(T, k, generator=g, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_route_ex(opt, s, T, E, k, ids, w, stream=side)
    m.moe_route_backward(opt, s, T, E, k, ids, dw, d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ids2, w2, d2 = torch.empty_like(ids), torch.empty_like(w), torch.empty(T, E, device=DEV)
    flat = _rule(m, renormalise=False)
    m.moe_route_ex(flat, s.contiguous(), T, E, k, ids2, w2)
    m.moe_route_backward(flat, s.contiguous(), T, E, k, ids2, dw, d2)
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(d[:, :E], d2)
    assert torch.all(d[:, E:] == 5.0)
    # an id that is no expert has no part in the gradient
    bad = ids.clone()
    bad[3, 1], bad[4, 0] = E, -1
    m.moe_route_backward(_rule(m, score="sigmoid", renormalise=False), s.contiguous(), T, E, k, bad, dw, d2)
    assert int((d2[3] != 0).sum()) == k - 1 and int((d2[4] != 0).sum()) == k - 1
    m.moe_route_ex(opt, None, 0, E, k, None, None)
    m.moe_route_backward(opt, None, 0, E, k, None, None, None)


def test_route_ex_agrees_with_route(m):
    s = torch.randn(500, 128, generator=gen(2), device=DEV)
    a, b = torch.empty(500, 8, dtype=torch.int32, device=DEV), torch.empty(500, 8, dtype=torch.int32, device=DEV)
    wa, wb = torch.empty(500, 8, device=DEV), torch.empty(500, 8, device=DEV)
    m.moe_route(s, 500, 128, 8, a, wa)
    m.moe_route_ex(_rule(m), s, 500, 128, 8, b, wb)
    assert torch.equal(a, b) and torch.allclose(wa, wb, rtol=1e-6, atol=0)


# ----------------------------------------------------------------------------- norms
def _norm_case(m, T, H, kind, post, pre, gate, h_dtype, o_dtype, w_dtype, biases, ld_h=0, ld_o=0, offset=0, eps=1e-5,
               alpha=0.7, beta=0.9, vectors=True, zero_row=False, no_dh=False):
    g = gen(T * 31 + H)
    ht, ot, wt = DT[h_dtype], DT[o_dtype], DT[w_dtype]
    lh, lo = ld_h or H, ld_o or H
    h, o = rows(T, H, lh, ht, g, 2.0, offset), rows(T, H, lo, ot, g, 0.5, offset)
    if zero_row:
        h[0] = 0
        o[0] = 0
    vec = lambda mean: (mean + 0.3 * torch.randn(H, generator=g, device=DEV)).to(wt)  # noqa: E731
    w_post = vec(1.0) if post and vectors else None
    w_pre = vec(1.0) if pre and vectors else None
    b_post = vec(0.0) if post and biases else None
    b_pre = vec(0.0) if pre and biases else None
    gt = {None: lambda: None, "channel": lambda: vec(0.5), "token": lambda: torch.randn(T, generator=g, device=DEV),
          "full": lambda: rows(T, H, lo, ot, g, 1.0, offset)}[gate]()
    gates = {None: m.MOE_GATE_NONE, "channel": m.MOE_GATE_CHANNEL, "token": m.MOE_GATE_TOKEN, "full": m.MOE_GATE_FULL}
    kinds = {"rms": m.MOE_NORM_RMS, "layer": m.MOE_NORM_LAYER}
    p = m.norm_problem(T, H, kinds[kind] if post else m.MOE_NORM_NONE, kinds[kind] if pre else m.MOE_NORM_NONE,
                       gates[gate], code(m, h_dtype), code(m, o_dtype), code(m, w_dtype), eps, alpha, beta, ld_h, ld_o)
    h_out, x_out = rows(T, H, lh, ht, g, 1.0, offset), rows(T, H, lo, ot, g, 1.0, offset) if pre else None
    m.moe_norm_forward(p, h, o, gt, w_post, b_post, w_pre, b_pre, h_out, x_out)
    og = None if gate is None else {"kind": gate, "values": f64(gt)}
    okind = (kind if post else None, kind if pre else None)
    ref_h, ref_x, mag_h, mag_x = B.norm(f64(h), f64(o), og, f64(w_post), f64(b_post), f64(w_pre), f64(b_pre), *okind,
                                        eps, alpha, beta)
    # a sum over a row: at most 16 values per thread and ten levels of a tree, then a dozen operations
    check(h_out, ref_h, mag_h, 32, "h_out")
    if pre:
        check(x_out, ref_x, mag_x, 64, "x_out")
    # gradient, from given h_out
    hs = rows(T, H, lh, ht, g, 2.0, offset)
    if zero_row:
        hs[0] = 0
    dh_out = None if no_dh else rows(T, H, lh, ht, g, 1.0, offset)
    dx_out = rows(T, H, lo, ot, g, 1.0, offset) if pre else None
    dh, do = rows(T, H, lh, ht, g, 1.0, offset), rows(T, H, lo, ot, g, 1.0, offset)
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
    dgate = {None: lambda: None, "channel": lambda: nan(H), "token": lambda: nan(T),
             "full": lambda: rows(T, H, lo, ot, g, 1.0, offset)}[gate]()
    sums = {n: nan(H) for n in (["dw_post", "db_post"] if post else []) + (["dw_pre", "db_pre"] if pre else [])}
    ws = torch.empty(m.moe_norm_backward_workspace_size(p), dtype=torch.uint8, device=DEV)
    m.moe_norm_backward(p, dh_out, dx_out, hs, o, gt, w_post, b_post, w_pre, dh, do, dgate, sums.get("dw_post"),
                        sums.get("db_post"), sums.get("dw_pre"), sums.get("db_pre"), ws)
    ref = B.norm_backward(f64(dh_out), f64(dx_out), f64(hs), f64(o), og, f64(w_post), f64(b_post), f64(w_pre), *okind,
                          eps, alpha, beta)
    check(dh, *ref["dh"], 64, "dh")
    check(do, *ref["do"], 128, "do")
    # a column: ceil(T / blocks) rows in a block, then the blocks by 32 and 32 sums
    chain = 64 + -(-T // 152) + 40
    for n, v in sums.items():
        check(v, *ref[n], chain, n)
    if gate:
        check(dgate, *ref["dgate"], 128 if gate == "full" else chain + 64, "dgate")


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_norm_forms(m, kind, gate, post, pre):
    _norm_case(m, 5, 200, kind, post, pre, gate, "bf16", "bf16", "f32", True)
    _norm_case(m, 5, 203, kind, post, pre, gate, "f32", "f32", "f32", False)


@pytest.mark.parametrize("h,o,w", [("f32", "f32", "f32"), ("f32", "bf16", "bf16"), ("f32", "f16", "f32"),
                                   ("bf16", "bf16", "bf16"), ("f16", "f16", "f16"), ("f16", "f16", "bf16")])
@pytest.mark.parametrize("H", [64, 63])
def test_norm_types(m, h, o, w, H):
    _norm_case(m, 33, H, "rms", True, True, "channel", h, o, w, False)
    _norm_case(m, 33, H, "layer", True, True, "full", h, o, w, True)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 4096), (3, 7), (2, 8), (700, 32), (2000, 96), (311, 1023), (5, 4096), (3, 4104),
                                 (2, 8192), (2, 8200), (2, 8191), (2, 16384), (1, 16383), (2500, 264)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_sizes(m, T, H, kind):
    _norm_case(m, T, H, kind, True, True, "channel", "bf16", "bf16", "f32", True)
    _norm_case(m, T, H, kind, True, True, "token", "f32", "f32", "f32", True)


# short rows, taken by groups of 4 to 32 lanes: the last groups without a row, odd widths
@pytest.mark.parametrize("T,H", [(1301, 33), (1301, 151), (1223, 40), (1229, 64), (311, 128), (2500, 249), (307, 256),
                                 (613, 512)])
@pytest.mark.parametrize("kind,gate", [("rms", "channel"), ("rms", None), ("layer", "token"), ("layer", "full")])
def test_norm_short_rows(m, T, H, kind, gate):
    _norm_case(m, T, H, kind, True, True, gate, "bf16", "bf16", "f32", kind == "layer")
    _norm_case(m, T, H, kind, True, kind == "rms", gate, "f32", "f32", "f32", True, zero_row=True, eps=1e-3)


# rows that start and end anywhere between 16-byte boundaries, shorter than one, one and two in shared memory
@pytest.mark.parametrize("T,H,ld_h,ld_o", [(7, 1, 1, 1), (9, 3, 5, 7), (11, 8, 9, 9), (40, 17, 17, 33), (700, 513, 513, 513),
                                           (310, 1023, 1025, 1031), (3, 4099, 4099, 4101), (3, 8191, 8191, 8191)])
@pytest.mark.parametrize("kind,gate", [("rms", "channel"), ("layer", "token")])
@pytest.mark.parametrize("h,o", [("bf16", "bf16"), ("f32", "f32"), ("f32", "f16")])
def test_norm_odd_rows(m, T, H, ld_h, ld_o, kind, gate, h, o):
    # a layer norm of one or three columns amplifies what its mean rounds
    eps = 1e-5 if H > 8 else 1e-1
    _norm_case(m, T, H, kind, True, True, gate, h, o, "f32", True, ld_h=ld_h, ld_o=ld_o, offset=1, eps=eps)
    _norm_case(m, T, H, kind, True, True, gate, h, o, "f32", False, ld_h=ld_h, ld_o=ld_o, offset=5, eps=eps, zero_row=True)


def test_norm_strides_and_alignment(m):
    _norm_case(m, 9, 128, "rms", True, True, "full", "bf16", "bf16", "f32", False, ld_h=136, ld_o=144)
    _norm_case(m, 9, 128, "rms", True, True, "full", "bf16", "bf16", "f32", False, ld_h=131, ld_o=129)
    _norm_case(m, 9, 128, "layer", True, True, "full", "f32", "bf16", "f32", True, offset=1)
    _norm_case(m, 9, 120, "layer", True, True, "channel", "bf16", "bf16", "bf16", True, ld_h=200, ld_o=123, offset=3)


def test_norm_without_vectors_zero_rows_and_no_residual_gradient(m):
    _norm_case(m, 4, 256, "rms", True, True, "token", "bf16", "bf16", "f32", False, vectors=False)
    _norm_case(m, 4, 256, "layer", True, True, None, "f32", "f32", "f32", True, vectors=False, zero_row=True)
    _norm_case(m, 4, 256, "rms", True, True, "channel", "f32", "f32", "f32", False, zero_row=True, no_dh=True)


def test_norm_in_place_stream_and_repeat(m):
    g = gen(21)
    T, H = 1300, 512
    p = m.norm_problem(T, H)
    h, o = rows(T, H, H, torch.bfloat16, g), rows(T, H, H, torch.bfloat16, g)
    w = torch.rand(H, generator=g, device=DEV) + 0.5
    a, b = torch.empty_like(h), torch.empty_like(o)
    m.moe_norm_forward(p, h, o, None, w, None, w, None, a, b)
    hc, oc = h.clone(), o.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_norm_forward(p, hc, oc, None, w, None, w, None, hc, oc, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, hc) and torch.equal(b, oc)
    ws = torch.empty(m.moe_norm_backward_workspace_size(p), dtype=torch.uint8, device=DEV)
    dh, dx = rows(T, H, H, torch.bfloat16, g), rows(T, H, H, torch.bfloat16, g)
    out = []
    for _ in range(2):
        r = [torch.empty_like(dh), torch.empty_like(dx), torch.empty(H, device=DEV), torch.empty(H, device=DEV)]
        m.moe_norm_backward(p, dh, dx, a, o, None, w, None, w, r[0], r[1], None, r[2], None, r[3], None, ws)
        out.append(r)
    assert all(torch.equal(x, y) for x, y in zip(*out))
    m.moe_norm_backward(p, dh, dx, a, o, None, w, None, w, dh, dx, None, None, None, None, None, ws)
    assert torch.equal(dh, out[0][0]) and torch.equal(dx, out[0][1])


def test_norm_empty(m):
    p = m.norm_problem(0, 64)
    m.moe_norm_forward(p, None, None, None, None, None, None, None, None, None)
    d = torch.full((64,), 3.0, device=DEV)
    m.moe_norm_backward(p, None, None, None, None, None, None, None, None, None, None, None, d, None, None, None, None, 0)
    assert torch.all(d == 0)


# ----------------------------------------------------------------------------- linear
def _linear_case(m, M, N, K, act="none", dtype="bf16", out="bf16", bias=None, residual=False, keep_z=False, alpha=1.0,
                 ld_x=0, ld_w=0, ld_y=0, in_place=False, gradient=True):
    g = gen(M * 7 + N * 3 + K)
    t, yt = DT[dtype], DT[out]
    x = rows(M, K, ld_x or K, t, g)
    w = rows(N, K, ld_w or K, t, g, K ** -0.5)
    b = None if bias is None else torch.randn(N, generator=g, device=DEV).to(DT[bias])
    r = rows(M, N, ld_y or N, yt, g) if residual else None
    y = r if in_place else rows(M, N, ld_y or N, yt, g)
    z = torch.full((M, N), float("nan"), dtype=t, device=DEV) if keep_z else None
    acts = {"none": m.MOE_ACT_NONE, "relu": m.MOE_ACT_RELU, "silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU,
            "gelu_tanh": m.MOE_ACT_GELU_TANH}
    p = m.linear_problem(M, N, K, code(m, dtype), code(m, out), code(m, bias or "f32"), acts[act], alpha, ld_x, ld_w, ld_y)
    ws = torch.full((m.moe_linear_workspace_size(p),), 255, dtype=torch.uint8, device=DEV)
    ref, rz, mag = B.linear(f64(x), f64(w), f64(b), f64(r), act, alpha)
    m.moe_linear(p, x, w, b, r, y, z, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    # the accumulator may round once per eight products; every activation's slope is below 1.13
    steps = K / 8 + 16
    if keep_z:
        check(z, rz, mag, steps, "z")
    check(y, ref, 1.13 * abs(alpha) * (mag + (8 * (1 + np.abs(rz))) / steps) + np.abs(ref) * 4 / steps, steps, "y")
    if not gradient:
        return
    dy = rows(M, N, ld_y or N, yt, g)
    zin = torch.randn(M, N, generator=g, device=DEV).to(t) if act != "none" else None
    dx = torch.full((M, K), float("nan"), dtype=t, device=DEV)
    dw = torch.full((N, K), float("nan"), dtype=t, device=DEV)
    db = torch.full((N,), float("nan"), device=DEV)
    ws = torch.full((m.moe_linear_backward_workspace_size(p),), 255, dtype=torch.uint8, device=DEV)
    m.moe_linear_backward(p, dy, x, w, zin, dx, dw, db, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    ref = B.linear_backward(f64(dy), f64(x), f64(w), f64(zin), act, alpha)
    u = U[dtype] * 1.01 + 16 * STEP  # dz is rounded to the operands' type
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    check(dx, ref["dx"][0], ref["dx"][1] + tiny, N / 8 + 16, "dx", u)
    check(dw, ref["dw"][0], ref["dw"][1] + tiny, M / 8 + 16, "dw", u)
    check(db, *ref["dbias"], 64 + -(-M // 256) + 40, "dbias")


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 100, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(128, 64), (1, 8), (129, 72), (256, 1024), (7, 200), (640, 136)])
def test_linear_sizes(m, M, N, K):
    _linear_case(m, M, N, K, bias="f32", residual=True)


# a few rows: one and two columns per warp, columns that do not divide, sums shorter than a warp's reach and longer
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 8), (3, 264), (130, 2048), (301, 1400), (2435, 72), (2433, 1032)])
@pytest.mark.parametrize("dtype,out,act", [("bf16", "f32", "none"), ("f16", "f16", "silu")])
def test_linear_few_rows(m, M, N, K, dtype, out, act):
    _linear_case(m, M, N, K, act=act, dtype=dtype, out=out, bias="f32", residual=True, keep_z=True, alpha=0.5,
                 ld_x=K + 8, ld_w=K + 16, ld_y=N + 3, gradient=False)  # the forward's own form


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype,out,bias", [("bf16", "bf16", "bf16"), ("f16", "f16", "f32"), ("bf16", "f32", None),
                                            ("f16", "f32", "f16")])
def test_linear_epilogues(m, act, dtype, out, bias):
    _linear_case(m, 70, 130, 128, act, dtype, out, bias, residual=True, keep_z=True, alpha=0.5)
    _linear_case(m, 5, 300, 512, act, dtype, out, bias, keep_z=act != "none")


@pytest.mark.parametrize("M,N,K", [(2500, 2176, 320), (4096, 2048, 64), (16384, 128, 256), (513, 4100, 1000)])
def test_linear_many_tiles(m, M, N, K):
    _linear_case(m, M, N, K, "silu", bias="f32", residual=True, keep_z=True)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "bf16")])
def test_linear_large_tiles(m, act, dtype, out):
    # over 38 tiles of 256 x 256, ragged in every direction
    _linear_case(m, 1500, 2056, 200, act, dtype, out, "f32", residual=True, keep_z=act != "none", alpha=0.5,
                 in_place=True)


@pytest.mark.parametrize("M,N,K", [(1, 64, 4096), (8, 4096, 4096), (40, 128, 7168), (3000, 64, 2048)])
def test_linear_long_sums(m, M, N, K):
    _linear_case(m, M, N, K, out="f32", bias="f32")
    _linear_case(m, M, N, K, dtype="f16", out="f16", residual=True)


def test_linear_strides(m):
    _linear_case(m, 50, 77, 100, bias="f32", residual=True, ld_x=104, ld_w=112, ld_y=81)
    _linear_case(m, 50, 77, 3, "gelu", keep_z=True, ld_x=8, ld_w=16, ld_y=80)
    _linear_case(m, 200, 96, 130, ld_x=136, ld_w=136, ld_y=104, residual=True, in_place=True)


def test_linear_repeats_bit_for_bit_on_streams(m):
    g = gen(3)
    for M, N, K in ((8, 512, 4096), (600, 512, 512)):
        x, w = rows(M, K, K, torch.bfloat16, g), rows(N, K, K, torch.bfloat16, g)
        p = m.linear_problem(M, N, K, out_dtype=m.MOE_DTYPE_F32)
        outs = []
        for side in (None, torch.cuda.Stream(), torch.cuda.Stream()):
            y = torch.empty(M, N, device=DEV)
            ws = torch.empty(m.moe_linear_workspace_size(p), dtype=torch.uint8, device=DEV)
            torch.cuda.synchronize()
            m.moe_linear(p, x, w, None, None, y, None, ws, stream=side)
            outs.append((y, ws))
        torch.cuda.synchronize()
        assert all(torch.equal(outs[0][0], y) for y, _ in outs[1:])


def test_linear_in_a_graph_and_empty(m):
    g = gen(9)
    M, N, K = 4, 256, 512
    x, w = rows(M, K, K, torch.bfloat16, g), rows(N, K, K, torch.bfloat16, g)
    p = m.linear_problem(M, N, K)
    ws = torch.empty(m.moe_linear_workspace_size(p), dtype=torch.uint8, device=DEV)
    y, want = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    m.moe_linear(p, x, w, None, None, want, None, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_linear(p, x, w, None, None, y, None, ws)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    q = m.linear_problem(0, N, K)
    m.moe_linear(q, None, None, None, None, None, None, None, 0)
    dw = torch.ones(N, K, dtype=torch.bfloat16, device=DEV)
    db = torch.ones(N, device=DEV)
    m.moe_linear_backward(q, None, None, None, None, None, dw, db, None, 0)
    assert torch.all(dw == 0) and torch.all(db == 0)
