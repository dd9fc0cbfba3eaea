"""The gated layers at special arguments: activations and slopes over fp32's and the 16-bit types' whole ranges,
infinities and NaN, and a gradient that leaves fp16's range."""
import numpy as np
import pytest
import torch

from oracle.blocks import act as oracle_act, act_grad
from tests.test_block_ops import DEV, DT, STEP, code, f64, gen, m, rows  # noqa: F401  (m: a fixture)
from tests.test_dense_ops import ACTS, acts

pytestmark = pytest.mark.gpu

# gates: both ends of the range, where e^-z, z^2 and z^3 leave it, and around 0
SWEEP = np.array([v * s for v in (0.0, 1e-45, 1e-38, 1e-20, 1e-5, 0.5, 1, 3, 10, 20, 80, 86, 87, 88, 88.5, 89, 90, 103, 104, 105, 150, 199,
                                  200, 1e3, 1e6, 1e12, 1.8e19, 1e20, 1e25, 1e30, 1e38, 3.4e38, np.inf) for s in (1, -1)] + [np.nan], np.float32)


def check_sweep(h, g, act):
    """act(g) in fp32: a few roundings of 1 + |g|; far out 0 or g itself; infinities and NaN where the formula has
    them."""
    with np.errstate(all="ignore"):
        ref = oracle_act(g.astype(np.float64), act)
    assert np.array_equal(np.isnan(h), np.isnan(ref) & np.ones_like(h, bool))
    assert np.array_equal(np.isinf(h), np.isinf(ref) & np.ones_like(h, bool))
    far = np.isfinite(ref) & (np.abs(g) >= 200)
    near = np.isfinite(ref) & ~far
    want = g if act == "none" else np.maximum(g, 0)
    assert np.array_equal(h[:, far], np.broadcast_to(want[far], h[:, far].shape))
    assert np.all(np.abs(h[:, near] - ref[near]) <= 8 * STEP * (1 + np.abs(g[near])))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 72, 64), (2, 130, 64), (7, 200, 64), (40, 136, 64), (1500, 1032, 64)])
def test_activations_over_their_whole_range(m, act, M, N, K):  # noqa: F811
    """The products are zeros, so that the biases are gate and up: every form's epilogue."""
    g = np.resize(SWEEP, N)
    bias = torch.from_numpy(np.concatenate([g, np.ones(N, np.float32)])).to(DEV)
    h = torch.full((M, N), 7.0, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    x, w = rows(M, K, K, torch.bfloat16, gen(1)), torch.zeros(2 * N, K, dtype=torch.bfloat16, device=DEV)
    m.moe_gated(m.gated_problem(M, N, K, out_dtype=m.MOE_DTYPE_F32, act=acts(m, act)), x, w, bias, h, None, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    check_sweep(h.cpu().numpy(), g, act)
    h.fill_(7.0)
    p = m.gated_problem(M, N, K, m.MOE_DTYPE_E4M3, m.MOE_DTYPE_F32, act=acts(m, act))
    x, w = (torch.full(s, v, dtype=torch.uint8, device=DEV) for s, v in (((M, K), 0x38), ((2 * N, K), 0)))
    m.moe_gated_fp8(p, x, torch.ones(M, 1, device=DEV), w, torch.ones(2, -(-N // 128), 1, device=DEV), bias, h, None, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    check_sweep(h.cpu().numpy(), g, act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N", [65536, 65534, 65533])
def test_slopes_at_every_16_bit_gate(m, act, dtype, N):  # noqa: F811
    """One row with u = dh = 1: dbias is [act'(g), act(g)] unrounded, for every bit pattern of g (in rows that 8, 2
    and 1 values of an access fit)."""
    g = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(DT[dtype])[:N]
    z = torch.cat([g, torch.ones(N, dtype=DT[dtype], device=DEV)])[None]
    p = m.gated_problem(1, N, 8, code(m, dtype), code(m, dtype), act=acts(m, act))
    ws = torch.empty(m.moe_gated_backward_workspace_size(p), dtype=torch.uint8, device=DEV)
    db = torch.full((2 * N,), 7.0, device=DEV)
    m.moe_gated_backward(p, torch.ones(1, N, dtype=DT[dtype], device=DEV), None, None, z, None, None, db, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    g, db = f64(g), db.cpu().numpy()
    finite = np.isfinite(g)
    for got, formula in ((db[:N], act_grad), (db[N:], oracle_act)):
        with np.errstate(all="ignore"):
            ref = formula(g, act)
        assert np.isfinite(got[finite]).all()
        # as tests/test_dense_ops.py: 16 roundings of the activation's scale
        assert np.all(np.abs(got[finite] - ref[finite]) <= 16 * STEP * (1 + np.abs(g[finite])))
        assert np.array_equal(np.isnan(got[~finite]), np.isnan(ref[~finite]))
        inf = np.isinf(g) & ~np.isnan(ref)
        assert np.array_equal(got[inf], ref[inf])
    # far out the slope is 0 or 1 (with no activation 1) and not a rounding of |g|
    far = finite & (np.abs(g) >= 200)
    assert np.all(np.abs(db[:N][far] - act_grad(g[far], act)) <= 16 * STEP)


@pytest.mark.parametrize("M,N,K", [(3, 24, 64), (40, 24, 64), (600, 520, 256), (3000, 1024, 512)])
def test_gradient_that_leaves_fp16(m, M, N, K):  # noqa: F811
    """A dg past 65504 is infinite in the products' operand: its row of dx and its row of dw are no numbers, dbias and
    all other rows are what they are without it."""
    g = gen(M)
    f16 = torch.float16
    x, w = rows(M, K, K, f16, g), rows(2 * N, K, K, f16, g, K ** -0.5)
    z, dh = rows(M, 2 * N, 2 * N, f16, g), rows(M, N, N, f16, g)
    z[2, 5], z[2, N + 5] = 3.0, 4.0  # dg = 60000 x 4 x 1.09, du = 60000 x 2.86: both past fp16
    p = m.gated_problem(M, N, K, m.MOE_DTYPE_F16, m.MOE_DTYPE_F16)
    ws = torch.empty(m.moe_gated_backward_workspace_size(p), dtype=torch.uint8, device=DEV)
    outs = []
    for v in (0.0, 60000.0):
        dh[2, 5] = v
        out = [torch.full((M, K), 7.0, dtype=f16, device=DEV), torch.full((2 * N, K), 7.0, dtype=f16, device=DEV),
               torch.full((2 * N,), 7.0, device=DEV)]
        m.moe_gated_backward(p, dh, x, w, z, *out, ws)
        assert m.moe_read_device_status(ws) == m.MOE_OK
        outs.append(out)
    (dx0, dw0, db0), (dx, dw, db) = outs
    assert all(torch.isfinite(t).all() for t in outs[0])
    assert not torch.isfinite(dx[2]).any() and not torch.isfinite(dw[[5, N + 5]]).any()
    rest = [i for i in range(M) if i != 2]
    cols = [i for i in range(2 * N) if i not in (5, N + 5)]
    assert torch.equal(dx[rest], dx0[rest]) and torch.equal(dw[cols], dw0[cols]) and torch.equal(db[cols], db0[cols])
    for i, slope in ((5, act_grad), (N + 5, oracle_act)):
        want = float(db0[i]) + 60000 * (4.0 if i == 5 else 1.0) * float(slope(np.float64(3.0), "silu"))
        assert abs(float(db[i]) - want) <= (64 + M / 256 + 40) * STEP * (abs(want) + 20 * M)
