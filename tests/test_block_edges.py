"""Edges of the operators around the routed FFN on the GPU: lengths, types, values and
empty parts at which a call is easily answered wrongly or refused.  Bounds as in
test_block_ops.py, whose cases and checks are used."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import blocks as B
from tests.test_block_ops import DEV, DT, STEP, U, _linear_case, _route, _rule, check, code, f64, gen, rows

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def m():
    import __graft_entry__

    __graft_entry__.build()
    import mixture_experts_layer_index_gb300 as mod

    return mod


def act_code(m, name):
    return getattr(m, "MOE_ACT_" + name.upper())


# sums that end inside 16 bytes, NaN behind them and between the rows
@pytest.mark.parametrize("M", list(range(1, 10)))
@pytest.mark.parametrize("K", [1, 3, 100, 1030])
@pytest.mark.parametrize("N,dtype,out", [(1, "bf16", "bf16"), (130, "f16", "f16"), (2435, "bf16", "f32")])
def test_linear_few_rows_of_any_length(m, M, K, N, dtype, out):
    ld = (K + 7) // 8 * 8
    _linear_case(m, M, N, K, dtype=dtype, out=out, bias="f32", residual=True, keep_z=True, alpha=0.5, ld_x=ld, ld_w=ld + 8,
                 ld_y=N + 3, gradient=False)


# rows of few products in a 16-bit type that is not the operands'
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("dtype,out", [("f16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("N,K", [(130, 264), (2435, 72)])
def test_linear_few_rows_to_the_other_16_bit_type(m, M, dtype, out, N, K):
    _linear_case(m, M, N, K, "silu", dtype, out, "f32", residual=True, keep_z=True, alpha=0.5, ld_y=N + 3, gradient=False)


# groups of few experts: two lanes take a row once there are many
@pytest.mark.parametrize("E,n_group,topk_group,k", [(8, 4, 2, 3), (24, 3, 2, 6), (32, 8, 4, 8), (33, 3, 2, 4)])
@pytest.mark.parametrize("T", [9727, 9728, 20000])
@pytest.mark.parametrize("group_best", [1, 2])
def test_route_groups_of_few_experts(m, E, n_group, topk_group, k, T, group_best):
    s = torch.randn(T, E, generator=gen(E + T), device=DEV)
    _route(m, s, k, n_group=n_group, topk_group=topk_group, group_best=group_best)


# four and more tiles of 256 x 256 per pair of SMs: both accumulators are filled again and again
@pytest.mark.parametrize("M,N,K,ld_y", [(8200, 2600, 72, 0), (8200, 2600, 8, 2603)])
@pytest.mark.parametrize("dtype,out,act", [("bf16", "f32", "silu"), ("f16", "f16", "gelu_tanh"), ("bf16", "bf16", "none")])
def test_linear_many_tiles_per_pair(m, M, N, K, ld_y, dtype, out, act):
    _linear_case(m, M, N, K, act, dtype, out, "f32", residual=True, keep_z=act != "none", alpha=0.5, ld_y=ld_y,
                 gradient=False)
    _linear_case(m, M, N, K, act, dtype, out, None, residual=True, in_place=True, ld_y=ld_y, gradient=False)


# unrounded outputs of long sums at sizes that pairs of SMs take, one accumulator per tile
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1300, 4100, 6152), (1500, 4096, 4096)])
def test_linear_long_sums_of_large_products(m, dtype, M, N, K):
    _linear_case(m, M, N, K, dtype=dtype, out="f32", bias="f32", gradient=False)


# a status word that nobody else writes
@pytest.mark.parametrize("M,N", [(5, 24), (300, 40), (0, 24), (5, 0)])
@pytest.mark.parametrize("wanted", ["dbias", "nothing", "all"])
def test_linear_backward_clears_its_status(m, M, N, wanted):
    p = m.linear_problem(M, N, 64)
    x, w, dy = (rows(max(n, 1), k, k, torch.bfloat16, gen(1))[:n] for n, k in ((M, 64), (N, 64), (M, max(N, 1))))
    out = dict(dbias=torch.full((N,), 7.0, device=DEV)) if wanted == "dbias" else {}
    if wanted == "all":
        out = dict(dx=torch.ones(M, 64, dtype=torch.bfloat16, device=DEV),
                   dw=torch.ones(N, 64, dtype=torch.bfloat16, device=DEV), dbias=torch.full((N,), 7.0, device=DEV))
    ws = torch.full((max(m.moe_linear_backward_workspace_size(p), 256),), 255, dtype=torch.uint8, device=DEV)
    m.moe_linear_backward(p, dy, x, w, None, out.get("dx"), out.get("dw"), out.get("dbias"), ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    if "dbias" in out and M and N:
        check(out["dbias"], f64(dy).sum(0), np.abs(f64(dy)).sum(0), 64 + 40, "dbias")
    elif "dbias" in out:
        assert not bool(out["dbias"].any())


@pytest.mark.parametrize("M,N", [(0, 24), (5, 0)])
def test_linear_of_nothing_clears_its_status(m, M, N):
    p = m.linear_problem(M, N, 64)
    ws = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
    m.moe_linear(p, None, None, None, None, None, None, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK


SPECIAL = [float("nan"), float("inf"), -float("inf"), -0.0, 0.0, 1e-30, -1e-30, 6e4, -6e4, 90.0, -90.0, -87.5, 20.0, -20.0,
           1.0, -1.278]
WIDE = [1e19, -1e19, 1e20, -1e20, 3e38, -3e38]  # squares and cubes pass the largest fp32


def same_values(got, ref, bound):
    """NaN where ref is NaN, infinities of the same sign, else within the bound."""
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (got, ref)
    assert np.array_equal(np.isinf(got), np.isinf(ref)) and np.array_equal(np.sign(got[np.isinf(got)]), np.sign(ref[np.isinf(ref)]))
    fine = np.isfinite(ref)
    assert np.all(np.abs(got[fine] - ref[fine]) <= bound[fine]), (got, ref)


# z = x * 1 holds each special value itself: a few rows, the tensor cores' tiles, and pairs of tiles
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(1, 8), (40, 24), (1500, 2056)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_special_values(m, act, M, N, dtype):
    t = DT[dtype]
    special = SPECIAL + (WIDE if dtype == "bf16" else [])
    v = torch.tensor(special, dtype=torch.float32, device=DEV).to(t)
    x = torch.zeros(M, 8, dtype=t, device=DEV)
    w = torch.zeros(N, 8, dtype=t, device=DEV)
    w[:, 0] = 1
    p = m.linear_problem(M, N, 8, code(m, dtype), m.MOE_DTYPE_F32, act=act_code(m, act))
    y = torch.empty(M, N, device=DEV)
    ws = torch.empty(m.moe_linear_workspace_size(p), dtype=torch.uint8, device=DEV)
    for i in range(0, len(special), M):
        n = min(M, len(special) - i)
        x.zero_()
        x[:n, 0] = v[i:i + n]
        m.moe_linear(p, x, w, None, None, y, None, ws)
        z = f64(v[i:i + n])
        with np.errstate(all="ignore"):
            ref = B.act(z, act)
        # an activation's error is relative to its argument (erf 1.5e-7, the others a few fp32 roundings)
        bound = 16 * STEP * np.where(np.isfinite(z), np.abs(z), 0.0) + 2.0 ** -126
        same_values(y[:n, 0], ref, bound)
        # the rows of w are the same, so every column is
        assert torch.equal(y[:n].nan_to_num(nan=7.0), y[:n, :1].nan_to_num(nan=7.0).expand(n, N))


# the slope at each special value, through dbias of a single row (fp32, unrounded)
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_slope_of_special_values(m, act, dtype):
    t = DT[dtype]
    special = SPECIAL + (WIDE if dtype == "bf16" else [])
    z = torch.tensor([special], dtype=torch.float32, device=DEV).to(t)
    N = len(special)
    p = m.linear_problem(1, N, 8, code(m, dtype), m.MOE_DTYPE_F32, act=act_code(m, act))
    dy = torch.full((1, N), 2.0, device=DEV)
    db = torch.full((N,), 9.0, device=DEV)
    ws = torch.empty(m.moe_linear_backward_workspace_size(p), dtype=torch.uint8, device=DEV)
    m.moe_linear_backward(p, dy, None, None, z, None, None, db, ws)
    with np.errstate(all="ignore"):
        ref = 2.0 * B.act_grad(f64(z)[0], act)
    # absolute: a slope is a sum of terms of size 1 and z (1 - s), of at most 1.3
    same_values(db, ref, np.full(N, 2 * 16 * STEP))


# a route to no expert has no part in y, whatever the experts hold, nor in the scale of the others
@pytest.mark.parametrize("quant,path", [("bf16", "grouped"), ("fp8_tensor", "grouped"), ("fp8_tensor", "route_direct"),
                                        ("fp8_block", "grouped"), ("fp8_block", "route_direct"), ("mxfp8", "grouped")])
@pytest.mark.parametrize("poison", [float("inf"), 1e4])
def test_a_route_to_no_expert_adds_nothing(m, quant, path, poison):
    T, E, k, H, I = 6, 16, 4, 256, 128
    d = {n: (None if v is None else v.to(DEV)) for n, v in W.make_inputs(W.Workload("t", T, E, k, H, I, quant, 5)).items()}
    ids = torch.stack([torch.randperm(E - 1, generator=torch.Generator().manual_seed(t))[:k] + 1 for t in range(T)])
    ids = ids.to(torch.int32).to(DEV)  # nobody asks for expert 0 ...
    w = torch.rand(T, k, generator=gen(2), device=DEV)
    if quant == "bf16":                # ... whose values are out of all proportion
        d["w1"][0] = poison
    else:
        d["w1_scale"][0] = poison if quant != "mxfp8" else 254 if poison == float("inf") else 140  # powers of two
    p = m.problem(T, E, k, H, I, quant, {"grouped": m.MOE_PATH_GROUPED, "route_direct": m.MOE_PATH_ROUTE_DIRECT}[path])
    ws = torch.full((m.moe_workspace_size(p),), 255, dtype=torch.uint8, device=DEV)

    def run(i, wt):
        y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
        m.moe_forward_routed(p, None, d["x"], i, wt, d["w1"], d["w2"], d["w1_scale"], d["w2_scale"], y, ws)
        return y, m.moe_read_device_status(ws)

    bad, twin, w0 = ids.clone(), ids.clone(), w.clone()
    for t, j, e in ((2, 1, E), (3, 0, -3), (5, 3, 1 << 30), (5, 2, -1)):
        bad[t, j], twin[t, j], w0[t, j] = e, ids[t, (j + 2) % k if t != 5 else 0], 0.0
    y, st = run(bad, w)
    assert st == m.MOE_ERR_DEVICE_BOUNDS
    # the same routes twice for a token, the second time with weight 0: the same h, so the same scales
    ref, st = run(twin, w0)
    assert st == m.MOE_OK and bool(torch.isfinite(ref).all())
    assert torch.equal(y, ref)
    v = m.moe_forward_views(p, ws)
    y, _ = run(torch.full_like(ids, -1), w)
    assert not bool(y.any())
    at = v.ids - ws.data_ptr()
    assert bool((ws[at:at + T * k * 4].view(torch.int32) == -1).all())


def test_route_as_many_tokens_as_there_can_be(m):
    T = (1 << 31) - 1
    s = torch.zeros(T, 1, dtype=torch.bfloat16, device=DEV)
    ids = torch.full((T, 1), -7, dtype=torch.int32, device=DEV)
    w = torch.zeros(T, 1, device=DEV)
    m.moe_route_ex(_rule(m, "bf16"), s, T, 1, 1, ids, w)
    assert int(ids.min()) == 0 and int(ids.max()) == 0 and float(w.min()) == 1.0 and float(w.max()) == 1.0
    d = torch.ones(T, 1, dtype=torch.bfloat16, device=DEV)
    m.moe_route_backward(_rule(m, "bf16"), s, T, 1, 1, ids, w, d)
    assert not bool(d.any())


def test_a_block_that_never_ran_reports_no_error(m):
    from mixture_experts_layer_index_gb300.block import Block

    H, E, I = 256, 8, 128
    d = {n: (None if v is None else v.to(DEV)) for n, v in W.make_inputs(W.Workload("t", 4, E, 2, H, I, "bf16", 5)).items()}
    ones = torch.ones(H, device=DEV)
    weight = torch.zeros(E, H, dtype=torch.bfloat16, device=DEV)
    torch.cuda.empty_cache()
    used = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in [256] * 64 + [1 << 20] * 4]
    torch.cuda.synchronize()
    del used  # their memory goes to whoever allocates next
    b = Block(4, E, 2, H, I, "bf16", (d["w1"], d["w2"], None, None), (weight, None), (ones, ones, None))
    assert b.status() == m.MOE_OK


# single rows: each gradient is one product, so the slope's own absolute error shows
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("N,K", [(130, 264), (2435, 72)])
def test_linear_single_row_gradient(m, act, dtype, out, N, K):
    g = gen(N + K)
    t = DT[dtype]
    x, w, dy = rows(1, K, K, t, g), rows(N, K, K + 8, t, g, K ** -0.5), rows(1, N, N, DT[out], g)
    z = torch.randn(1, N, generator=g, device=DEV).to(t) if act != "none" else None
    p = m.linear_problem(1, N, K, code(m, dtype), code(m, out), act=act_code(m, act), alpha=0.5, ld_w=K + 8)
    dx, dw = torch.full((1, K), float("nan"), dtype=t, device=DEV), torch.full((N, K), float("nan"), dtype=t, device=DEV)
    db = torch.full((N,), float("nan"), device=DEV)
    ws = torch.full((m.moe_linear_backward_workspace_size(p),), 255, dtype=torch.uint8, device=DEV)
    m.moe_linear_backward(p, dy, x, w, z, dx, dw, db, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    ref = B.linear_backward(f64(dy), f64(x), f64(w), f64(z), act, 0.5)
    # dz's rounding to the operands' type (f16: at least half the smallest step), and the
    # slope's error, which is relative to 1 + |z|
    u = U[dtype] * 1.01 + 16 * STEP
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    slope = np.zeros((1, N)) if z is None else 16 * STEP * 0.5 * np.abs(f64(dy)) * (1 + np.abs(f64(z)))
    dz = slope + tiny

    def close(got, name, more, factor, extra):
        val, mag = ref[name]
        ug = U[dtype] if got.dtype == t else U["f32"]
        off = np.abs(f64(got) - val) - (1 + ug) * (ug * np.abs(val) + (factor * STEP + extra) * (mag + tiny) + more) - (
            tiny + 2.0 ** -126)
        assert np.all(off <= 0), (name, float(off.max()))

    close(dx, "dx", dz @ np.abs(f64(w)), N / 8 + 16, u)
    close(dw, "dw", dz.T * np.abs(f64(x)), 16, u)
    close(db, "dbias", slope[0], 16, 0.0)
