"""GPU parity of the dense blocks' operators (gated linear layer and its gradient) against
oracle/dense.py in 64 bits.  Bounds as in tests/test_block_ops.py."""
import numpy as np
import pytest
import torch

from oracle import dense as D
from oracle.blocks import act as oracle_act
from tests.test_block_ops import DEV, DT, STEP, U, check, code, f64, gen, m, rows  # noqa: F401  (m: a fixture)

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def acts(m, name):
    return {"none": m.MOE_ACT_NONE, "relu": m.MOE_ACT_RELU, "silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU,
            "gelu_tanh": m.MOE_ACT_GELU_TANH}[name]


def gated_mag(z, mag, name, steps):
    """What `steps` roundings of g and u, and a few of the activation, are multiplied by in h = act(g)
    u; slopes of the activations are below 1.13."""
    N = z.shape[1] // 2
    g, u, mg, mu = z[:, :N], z[:, N:], mag[:, :N], mag[:, N:]
    a = np.abs(oracle_act(g, name))
    return 1.13 * mg * (np.abs(u) + steps * STEP * mu) + a * mu + (8 * (1 + np.abs(g)) * np.abs(u) + 4 * a * np.abs(u)) / steps


def strided(M, W, ld, dtype, g, scale=1.0):
    return rows(M, W, ld or W, dtype, g, scale)


def gated_case(m, M, N, K, act="silu", dtype="bf16", out="bf16", bias=None, keep_z=False, ld_x=0, ld_w=0, ld_h=0,
               forward=True, gradient=True, wanted=("dx", "dw", "dbias")):
    g = gen(M * 7 + N * 3 + K)
    t, ht = DT[dtype], DT[out]
    x = strided(M, K, ld_x, t, g)
    w = strided(2 * N, K, ld_w, t, g, K ** -0.5)
    b = None if bias is None else torch.randn(2 * N, generator=g, device=DEV).to(DT[bias])
    p = m.gated_problem(M, N, K, code(m, dtype), code(m, out), code(m, bias or "f32"), acts(m, act), ld_x, ld_w, ld_h)
    if forward:
        buf = torch.full((M + 2, ld_h or N), float("nan"), dtype=ht, device=DEV)
        h = buf[:M, :N]
        zbuf = torch.full((M + 2, 2 * N), float("nan"), dtype=t, device=DEV)
        z = zbuf[:M] if keep_z else None
        ws = torch.full((m.moe_gated_workspace_size(p),), 255, dtype=torch.uint8, device=DEV)
        m.moe_gated(p, x, w, b, h, z, ws)
        assert m.moe_read_device_status(ws) == m.MOE_OK
        ref, rz, mag = D.gated(f64(x), f64(w), f64(b), act)
        steps = K / 8 + 16  # the accumulator may round once per eight products
        if keep_z:
            check(z, rz, mag, steps, "z")
        check(h, ref, gated_mag(rz, mag, act, steps), steps, "h")
        assert torch.isnan(buf[:, N:]).all() and torch.isnan(buf[M:]).all()  # what lies between the rows and behind them
        assert torch.isnan(zbuf[M:]).all()
    if not gradient:
        return
    dh = strided(M, N, ld_h, ht, g)
    zin = torch.randn(M, 2 * N, generator=g, device=DEV).to(t)
    out_ = {"dx": torch.full((M, K), float("nan"), dtype=t, device=DEV),
            "dw": torch.full((2 * N, K), float("nan"), dtype=t, device=DEV),
            "dbias": torch.full((2 * N,), float("nan"), device=DEV)}
    ws = torch.full((m.moe_gated_backward_workspace_size(p),), 255, dtype=torch.uint8, device=DEV)
    m.moe_gated_backward(p, dh, x, w, zin, *[out_[n] if n in wanted else None for n in out_], ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    ref = D.gated_backward(f64(dh), f64(x), f64(w), f64(zin), act)
    # dz is rounded to the operands' type before the products; 16 roundings of the activation's scale
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    for n, terms, u in (("dx", 2 * N / 8 + 16, U[dtype] * 1.01), ("dw", M / 8 + 16, U[dtype] * 1.01),
                        ("dbias", 64 + -(-M // 256) + 40, 0.0)):
        if n in wanted:
            v, mag, soft = ref[n]
            # the products of the values lost below the type's least add up to tiny times the other operand
            lost = {"dx": np.abs(f64(w)).sum(0)[None, :], "dw": np.abs(f64(x)).sum(0)[None, :], "dbias": 0.0}[n] * tiny
            check(out_[n], v, mag + (16 * STEP * soft + lost) / (terms * STEP + u), terms, n, u)


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 100, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(64, 64), (1, 8), (129, 72), (200, 1024), (7, 200), (320, 136)])
def test_gated_sizes(m, M, N, K):  # noqa: F811
    gated_case(m, M, N, K, bias="f32", keep_z=True)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 8), (3, 264), (65, 2048), (301, 1400), (1217, 72)])
@pytest.mark.parametrize("dtype,out,act", [("bf16", "f32", "none"), ("f16", "f16", "silu")])
def test_gated_few_rows(m, M, N, K, dtype, out, act):  # noqa: F811
    gated_case(m, M, N, K, act, dtype, out, "f32", keep_z=True, ld_x=K + 8, ld_w=K + 16, ld_h=N + 3, gradient=False)


@pytest.mark.parametrize("M,N,K", [(2, 1024, 3000), (2, 1024, 3008), (2, 1025, 3008), (4, 1024, 2048), (3, 1025, 2048), (4, 64, 2056),
                                   (8, 1536, 1024), (7, 1537, 1024), (5, 64, 1032)])
def test_gated_few_rows_on_either_side_of_the_rule(m, M, N, K):  # noqa: F811
    gated_case(m, M, N, K, bias="f32", keep_z=True, gradient=False)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,out,bias", [("bf16", "bf16", "bf16"), ("f16", "f16", "f32"), ("bf16", "f32", None),
                                            ("f16", "f32", "f16"), ("bf16", "f16", "f32")])
def test_gated_epilogues(m, act, dtype, out, bias):  # noqa: F811
    gated_case(m, 70, 130, 128, act, dtype, out, bias, keep_z=True)
    gated_case(m, 5, 150, 512, act, dtype, out, bias)


# tiles of 256 x 128 by pairs of SMs: rows that TMA can store and rows that it cannot, ragged everywhere
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "bf16")])
def test_gated_large_tiles(m, act, dtype, out):  # noqa: F811
    gated_case(m, 1500, 1032, 200, act, dtype, out, "f32", keep_z=act != "none", gradient=False)
    gated_case(m, 1300, 1027, 136, act, dtype, out, "f32", keep_z=act != "none", gradient=False)


@pytest.mark.parametrize("M,N,K", [(2500, 1088, 320), (4096, 1024, 64), (16384, 64, 256), (513, 2050, 1000)])
def test_gated_many_tiles(m, M, N, K):  # noqa: F811
    gated_case(m, M, N, K, bias="f32", keep_z=True)


@pytest.mark.parametrize("M,N,K", [(1, 64, 4096), (8, 4096, 4096), (40, 128, 7168)])
def test_gated_long_sums(m, M, N, K):  # noqa: F811
    gated_case(m, M, N, K, out="f32", bias="f32", gradient=False)
    gated_case(m, M, N, K, dtype="f16", out="f16", gradient=False)


def test_gated_strides(m):  # noqa: F811
    gated_case(m, 50, 77, 100, bias="f32", ld_x=104, ld_w=112, ld_h=81)
    gated_case(m, 50, 77, 3, "gelu", keep_z=True, ld_x=8, ld_w=16, ld_h=80)
    gated_case(m, 1300, 1040, 130, ld_x=136, ld_w=136, ld_h=1048, keep_z=True, gradient=False)
    for N in (1025, 1030, 1035):  # rows that end inside 16 bytes
        gated_case(m, 1300, N, 136, ld_h=1048, keep_z=True, gradient=False)
        gated_case(m, 1300, N, 136, out="f32", ld_h=1048, gradient=False)


@pytest.mark.parametrize("M,N,K", [(517, 136, 100), (517, 133, 104), (40, 8, 64)])
@pytest.mark.parametrize("act,dtype,out", [("gelu", "f16", "f32"), ("silu", "bf16", "bf16"), ("relu", "bf16", "f16"),
                                           ("gelu_tanh", "f16", "f16"), ("none", "bf16", "f32")])
def test_gated_gradient_types(m, M, N, K, act, dtype, out):  # noqa: F811
    gated_case(m, M, N, K, act, dtype, out, ld_x=K + 12 if K % 8 else 0, ld_w=K + 20 if K % 8 else 0, forward=False)
    for wanted in (("dx",), ("dw",), ("dbias",), ("dx", "dbias")):
        gated_case(m, M, N, K, act, dtype, out, ld_x=K + 12 if K % 8 else 0, ld_w=K + 20 if K % 8 else 0, ld_h=N + 1,
                   forward=False, wanted=wanted)


def test_gated_empty(m):  # noqa: F811
    m.moe_gated(m.gated_problem(0, 64, 64), None, None, None, None, None, None, 0)
    m.moe_gated(m.gated_problem(4, 0, 64), None, None, None, None, None, None, 0)
    dw, db = torch.ones(128, 64, dtype=torch.bfloat16, device=DEV), torch.ones(128, device=DEV)
    m.moe_gated_backward(m.gated_problem(0, 64, 64), None, None, None, None, None, dw, db, None, 0)
    assert torch.all(dw == 0) and torch.all(db == 0)
    dx = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
    m.moe_gated_backward(m.gated_problem(4, 0, 64), None, None, None, None, dx, None, None, ws)
    assert torch.all(dx == 0) and m.moe_read_device_status(ws) == m.MOE_OK


def test_gated_special_values(m):  # noqa: F811
    """NaN and infinities in x reach their own rows only and do what the formulas do there."""
    M, N, K = 300, 130, 64
    for act in ("relu", "gelu", "none"):
        for Mi in (8, M, 1500):
            g = gen(5)
            x, w = rows(Mi, K, K, torch.bfloat16, g), rows(2 * N, K, K, torch.bfloat16, g)
            x[1, 3], x[4, 0] = float("nan"), float("inf")
            h = torch.zeros(Mi, N, dtype=torch.float32, device=DEV)
            p = m.gated_problem(Mi, N, K, out_dtype=m.MOE_DTYPE_F32, act=acts(m, act))
            ws = torch.empty(256, dtype=torch.uint8, device=DEV)
            m.moe_gated(p, x, w, None, h, None, ws)
            assert torch.isnan(h[1]).all()
            with np.errstate(invalid="ignore"):
                g4 = float("inf") * f64(w)[:N, 0]
                u4 = float("inf") * f64(w)[N:, 0]
                want = oracle_act(g4, act) * u4 if act != "gelu" else np.where(g4 > 0, np.inf, np.nan) * u4
            got = f64(h[4])
            assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])
            rest = [i for i in range(Mi) if i not in (1, 4)]
            assert torch.isfinite(h[rest]).all()


def test_gated_repeats_bit_for_bit_on_streams_and_in_a_graph(m):  # noqa: F811
    g = gen(3)
    for M, N, K in ((8, 256, 4096), (2, 64, 512), (600, 256, 512), (2000, 1024, 256)):
        x, w = rows(M, K, K, torch.bfloat16, g), rows(2 * N, K, K, torch.bfloat16, g, K ** -0.5)
        dh, z = rows(M, N, N, torch.bfloat16, g), rows(M, 2 * N, 2 * N, torch.bfloat16, g)
        p = m.gated_problem(M, N, K)
        outs = []
        for how in ("plain", "stream", "graph"):
            r = [torch.empty(M, N, dtype=torch.bfloat16, device=DEV), torch.empty(M, 2 * N, dtype=torch.bfloat16, device=DEV),
                 torch.empty(M, K, dtype=torch.bfloat16, device=DEV), torch.empty(2 * N, K, dtype=torch.bfloat16, device=DEV),
                 torch.empty(2 * N, device=DEV)]
            ws = torch.empty(m.moe_gated_workspace_size(p), dtype=torch.uint8, device=DEV)
            wb = torch.empty(m.moe_gated_backward_workspace_size(p), dtype=torch.uint8, device=DEV)

            def both(stream=None):
                m.moe_gated(p, x, w, None, r[0], r[1], ws, stream=stream)
                m.moe_gated_backward(p, dh, x, w, z, r[2], r[3], r[4], wb, stream=stream)

            torch.cuda.synchronize()
            if how == "graph":
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    both()
                for t in r:
                    t.zero_()
                graph.replay()
                graph.replay()
            else:
                both(torch.cuda.Stream() if how == "stream" else None)
            torch.cuda.synchronize()
            assert m.moe_read_device_status(ws) == m.MOE_OK and m.moe_read_device_status(wb) == m.MOE_OK
            outs.append(r)
        for r in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(outs[0], r))


@pytest.mark.parametrize("M", [8, 100, 1024])
def test_gated_fp32_output_of_long_sums(m, M):  # noqa: F811
    """No accumulator sums more than 512 values, 16 at a step, each step cut off at 2^-23 of the sum at
    most (linear_few.cu and the joins of partial sums round to nearest, 2^-24): h = g u, so twice that."""
    N, K = 1024, 4096
    g = gen(M)
    x, w = rows(M, K, K, torch.bfloat16, g), rows(2 * N, K, K, torch.bfloat16, g, K ** -0.5)
    h = torch.empty(M, N, device=DEV)
    p = m.gated_problem(M, N, K, out_dtype=m.MOE_DTYPE_F32, act=m.MOE_ACT_NONE)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    m.moe_gated(p, x, w, None, h, None, ws)
    z = x.double() @ w.double().T
    ref = z[:, :N] * z[:, N:]
    steps = 512 / 16 + K / 512 + 4
    assert float((h.double() - ref).norm() / ref.norm()) <= 2 * steps * 2.0 ** -24  # half a step each on average
