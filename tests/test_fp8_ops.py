"""GPU parity of the operators on e4m3 codes with block scales (quantisation, linear and gated
layer) against oracle/dense.py: codes and scales of the quantiser bit for bit, products within
bounds as in tests/test_block_ops.py."""
import numpy as np
import pytest
import torch

from oracle import dense as D
from oracle.blocks import act as oracle_act
from tests.test_block_ops import DEV, DT, STEP, check, code, f64, gen, m, rows  # noqa: F401  (m: a fixture)
from tests.test_dense_ops import ACTS, acts, gated_mag

pytestmark = pytest.mark.gpu


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


def same_codes(a, b):
    """Equal codes; a NaN's sign is free."""
    nan = (a & 0x7f) == 0x7f
    return np.array_equal(nan, (b & 0x7f) == 0x7f) and np.array_equal(a[~nan], b[~nan])


# ----------------------------------------------------------------------------- quantiser
def quantise_case(m, x, block_rows, ld_q=0, offset=0):  # noqa: F811
    M, K = x.shape
    name = {v: k for k, v in DT.items()}[x.dtype]
    ld = ld_q or K
    buf = torch.full((M * ld + offset + 64,), 0x55, dtype=torch.uint8, device=DEV)
    body = buf[offset:offset + M * ld].view(M, ld)
    q = body[:, :K]
    s = torch.full((-(-M // block_rows), -(-K // 128)), float("nan"), device=DEV)
    p = m.quantise_problem(M, K, code(m, name), block_rows, x.stride(0) if M > 1 else 0, ld_q)
    m.moe_quantise(p, x, q, s)
    codes, scales = D.quantise(x.float().cpu().numpy(), block_rows)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert same_codes(q.cpu().numpy(), codes)
    assert (buf[:offset] == 0x55).all() and (buf[-64:] == 0x55).all() and (body[:, K:] == 0x55).all()  # between the rows


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,K,ld", [(1, 1, 0), (1, 128, 0), (3, 129, 131), (130, 256, 0), (257, 1000, 1008), (5, 8192, 0),
                                    (64, 2056, 2064), (300, 130, 0), (33, 40, 48), (1027, 384, 385)])
def test_quantise(m, dtype, block_rows, M, K, ld):  # noqa: F811
    g = gen(M + K)
    x = rows(M, K, ld or K, DT[dtype], g)
    x *= torch.exp(2 * torch.randn(M, 1, generator=g, device=DEV)).to(x.dtype)
    if M > 2:
        x[1] = 0
    quantise_case(m, x, block_rows)
    quantise_case(m, x, block_rows, ld_q=(K + 15) // 16 * 16)
    quantise_case(m, rows(M, K, K + 3, DT[dtype], g, offset=1), block_rows, ld_q=K + 5, offset=3)


def test_quantise_every_midpoint(m):  # noqa: F811
    """Quotients on, and one fp32 step beside, every code and midpoint, under scales that are and are
    not powers of two and at both ends of fp32's range."""
    values = np.unique(np.abs(D.e4m3_decode(np.arange(0x7f, dtype=np.uint8)).astype(np.float64)))
    points = np.concatenate([values, (values[1:] + values[:-1]) / 2])
    for s in (1.0, 0.37, 3.3e-3, 1.7e12, 2.9e-30, 1.1e-38, 3e-41, 7e34):
        v = (points * s).astype(np.float32)
        v = np.concatenate([v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf))])
        v = v[v <= np.float32(448 * s)]
        v = np.concatenate([v, -v])
        x = np.zeros((-(-v.size // 127), 128), np.float32)
        x[:, 0] = np.float32(448 * s)
        x[:, 1:].reshape(-1)[:] = 0
        flat = np.zeros(x.shape[0] * 127, np.float32)
        flat[:v.size] = v
        x[:, 1:] = flat.reshape(-1, 127)
        quantise_case(m, torch.from_numpy(x).to(DEV), 1)
        quantise_case(m, torch.from_numpy(x).to(DEV), 128)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantise_special_values(m, dtype):  # noqa: F811
    x = rows(40, 300, 300, DT[dtype], gen(2))
    x[1, 5], x[2, 7], x[3, 200] = float("nan"), float("inf"), -float("inf")
    x[4] = float("nan")
    x[5] = 2.0 ** -149 if dtype == "f32" else 2.0 ** -24 if dtype == "f16" else 2.0 ** -133
    x[6, 0] = -0.0
    for block_rows in (1, 128):
        quantise_case(m, x, block_rows)


def test_quantise_empty(m):  # noqa: F811
    m.moe_quantise(m.quantise_problem(0, 128), None, None, None)


# ----------------------------------------------------------------------------- products
def operand(M, K, ld, block_rows, g, scale=1.0):
    """(codes in rows of ld bytes with NaN codes between them, scales, the values they stand for)"""
    v = (scale * torch.randn(M, K, generator=g, device=DEV)).cpu().numpy() * np.exp(np.random.default_rng(M).standard_normal((M, 1)))
    codes, s = D.quantise(v.astype(np.float32), block_rows)
    ld = ld or -(-K // 16) * 16
    buf = torch.full((M, ld), 0x7f, dtype=torch.uint8, device=DEV)
    buf[:, :K] = torch.from_numpy(codes).to(DEV)
    return buf[:, :K], torch.from_numpy(s).to(DEV), D.dequantise(codes, s, block_rows), ld


def linear_case(m, M, N, K, act="none", out="bf16", bias=None, residual=False, alpha=1.0, ld_x=0, ld_w=0, ld_y=0,  # noqa: F811
                in_place=False):
    g = gen(M * 7 + N * 3 + K)
    x, sx, xv, ld_x = operand(M, K, ld_x, 1, g)
    w, sw, wv, ld_w = operand(N, K, ld_w, 128, g, K ** -0.5)
    b = None if bias is None else torch.randn(N, generator=g, device=DEV).to(DT[bias])
    r = rows(M, N, ld_y or N, DT[out], g) if residual else None
    rv = f64(r)
    buf = torch.full((M + 2, ld_y or N), float("nan"), dtype=DT[out], device=DEV)
    y = r if in_place else buf[:M, :N]
    p = m.linear_problem(M, N, K, m.MOE_DTYPE_E4M3, code(m, out), code(m, bias or "f32"), acts(m, act), alpha, ld_x, ld_w, ld_y)
    ws = torch.full((m.moe_linear_fp8_workspace_size(p),), 255, dtype=torch.uint8, device=DEV)
    m.moe_linear_fp8(p, x, sx, w, sw, b, r, y, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    z, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    if b is not None:
        z, mag = z + f64(b), mag + np.abs(f64(b))
    ref = alpha * oracle_act(z, act) + (0.0 if rv is None else rv)
    steps = K / 8 + 16  # the accumulator may round once per eight products
    check(y, ref, 1.13 * abs(alpha) * (mag + 8 * (1 + np.abs(z)) / steps) + np.abs(ref) * 4 / steps, steps, "y")
    if not in_place:
        assert torch.isnan(buf[:, N:]).all() and torch.isnan(buf[M:]).all()


def gated_case(m, M, N, K, act="silu", out="e4m3", bias=None, ld_x=0, ld_w=0, ld_h=0):  # noqa: F811
    g = gen(M * 5 + N * 3 + K)
    x, sx, xv, ld_x = operand(M, K, ld_x, 1, g)
    wg, sg, wgv, ld_w = operand(N, K, ld_w, 128, g, K ** -0.5)
    wu, su, wuv, _ = operand(N, K, ld_w, 128, g, 0.5 * K ** -0.5)
    w = torch.full((2 * N, ld_w), 0x7f, dtype=torch.uint8, device=DEV)
    w[:N, :K], w[N:, :K] = wg, wu
    sw = torch.stack([sg, su]).contiguous()
    b = None if bias is None else torch.randn(2 * N, generator=g, device=DEV).to(DT[bias])
    ref, z, mag = D.gated(xv, np.concatenate([wgv, wuv]), f64(b), act)
    steps = K / 8 + 16
    hm = gated_mag(z, mag, act, steps)
    coded = out == "e4m3"
    ld = ld_h or (-(-N // 16) * 16 if coded else N)
    p = m.gated_problem(M, N, K, m.MOE_DTYPE_E4M3, m.MOE_DTYPE_E4M3 if coded else code(m, out), code(m, bias or "f32"),
                        acts(m, act), ld_x, ld_w, ld)
    ws = torch.full((m.moe_gated_fp8_workspace_size(p),), 255, dtype=torch.uint8, device=DEV)
    if not coded:
        buf = torch.full((M + 2, ld), float("nan"), dtype=DT[out], device=DEV)
        m.moe_gated_fp8(p, x, sx, w[:, :K], sw, b, buf[:M, :N], None, ws)
        assert m.moe_read_device_status(ws) == m.MOE_OK
        check(buf[:M, :N], ref, hm, steps, "h")
        assert torch.isnan(buf[:, N:]).all() and torch.isnan(buf[M:]).all()
        return
    buf = torch.full((M + 2, ld), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((M + 2, -(-N // 128)), float("nan"), device=DEV)
    m.moe_gated_fp8(p, x, sx, w[:, :K], sw, b, buf[:M, :N], s, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    assert (buf[:, N:] == 0x55).all() and (buf[M:] == 0x55).all() and torch.isnan(s[M:]).all()
    buf, s = buf[:M], s[:M]
    off = (steps * STEP) * hm
    pad = [(0, 0), (0, -N % 128)]
    amax = np.pad(np.abs(ref), pad).reshape(M, -1, 128).max(2)
    worst = np.pad(off, pad).reshape(M, -1, 128).max(2)
    sv = f64(s)
    want = np.where(amax > 0, amax / 448, 1.0)  # a group of zeros, as the quantiser has it
    assert np.all(np.abs(sv - want) <= worst / 448 + STEP * want)
    got = D.dequantise(buf[:, :N].cpu().numpy(), s.cpu().numpy(), 1)
    full = sv.repeat(128, 1)[:, :N]
    # half an e4m3 step, and where the value's own error carries it over a midpoint as much again as that error
    bound = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * full) * (1 + 4 * STEP) + 1.07 * off + worst.repeat(128, 1)[:, :N] * 2.0 ** -4
    assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) - bound))


SIZES = [(1, 64, 128), (2, 7, 16), (5, 130, 300), (8, 256, 2048), (9, 200, 1000), (16, 33, 4096), (17, 128, 128), (40, 300, 700),
         (100, 65, 5), (128, 256, 512), (129, 520, 130), (300, 1000, 257), (700, 129, 2000)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_sizes(m, M, N, K):  # noqa: F811
    linear_case(m, M, N, K, bias="f32", residual=True)
    linear_case(m, M, N, K, out="f32")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out,bias", [("bf16", "bf16"), ("f16", "f32"), ("f32", None), ("f32", "f16")])
@pytest.mark.parametrize("M,N,K", [(6, 50, 400), (12, 77, 256), (200, 130, 384)])
def test_linear_epilogues(m, act, out, bias, M, N, K):  # noqa: F811
    linear_case(m, M, N, K, act, out, bias, residual=True, alpha=0.5, ld_y=N + 3)
    linear_case(m, M, N, K, act, out, bias, in_place=True, residual=True, ld_y=(N + 7) // 8 * 8)


# pairs of SMs: rows that TMA can store and rows that it cannot, ragged everywhere
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_linear_large_tiles(m, act, out):  # noqa: F811
    linear_case(m, 4000, 2056, 700, act, out, "f32", residual=True, alpha=0.5)
    linear_case(m, 4100, 2051, 640, act, out, None, residual=act != "none")
    linear_case(m, 8192, 1024, 256, act, out, residual=True, in_place=True)
    linear_case(m, 4000, 2053, 256, act, out, ld_y=2064)  # rows that end inside 16 bytes


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", ["e4m3", "bf16"])
def test_gated_sizes(m, M, N, K, out):  # noqa: F811
    gated_case(m, M, N, K, out=out, bias="f32")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out,bias", [("e4m3", None), ("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("M,N,K", [(6, 50, 400), (12, 200, 256), (200, 130, 384)])
def test_gated_epilogues(m, act, out, bias, M, N, K):  # noqa: F811
    gated_case(m, M, N, K, act, out, bias, ld_h=(N + 31) // 16 * 16)


@pytest.mark.parametrize("out", ["e4m3", "bf16", "f32"])
def test_gated_large_tiles(m, out):  # noqa: F811
    gated_case(m, 4000, 1032, 700, "silu", out, "f32")
    gated_case(m, 4100, 1027, 640, "gelu", out)
    gated_case(m, 8192, 512, 256, "gelu_tanh", out, ld_h=528)
    gated_case(m, 4000, 1030, 256, "silu", out, ld_h=1040)


def test_long_sums_and_strides(m):  # noqa: F811
    linear_case(m, 8, 4096, 4096, out="f32", residual=True)
    linear_case(m, 33, 128, 8192, out="f32")
    linear_case(m, 50, 77, 100, ld_x=128, ld_w=144, ld_y=81, bias="f32")
    linear_case(m, 16, 144, 8192)
    linear_case(m, 12, 4160, 4096, out="f32")
    gated_case(m, 8, 1024, 4096)
    gated_case(m, 8, 4224, 4096)
    gated_case(m, 40, 96, 7168)
    gated_case(m, 50, 77, 100, ld_x=128, ld_w=144, ld_h=96)


def test_few_rows_on_either_side_of_the_rule(m):  # noqa: F811
    """Shapes next to where few rows go over to the tensor cores' form, by the sum and by the weights."""
    for out in ("e4m3", "bf16"):
        gated_case(m, 8, 70, 8192, out=out)
        gated_case(m, 8, 70, 8208, out=out)
    gated_case(m, 5, 6144, 130)
    gated_case(m, 5, 6160, 130)
    linear_case(m, 8, 130, 8320)
    linear_case(m, 16, 200, 4096, bias="f32")
    linear_case(m, 16, 200, 4112, bias="f32")
    linear_case(m, 3, 8192, 8208)


def test_empty(m):  # noqa: F811
    e = m.MOE_DTYPE_E4M3
    m.moe_linear_fp8(m.linear_problem(0, 64, 64, e), None, None, None, None, None, None, None, None, 0)
    m.moe_gated_fp8(m.gated_problem(4, 0, 64, e, e), None, None, None, None, None, None, None, None, 0)


@pytest.mark.parametrize("M", [5, 14, 200, 4096])
def test_special_scales_and_codes(m, M):  # noqa: F811
    """A NaN code or an infinite scale spoils its own row (of x) or column (of w) and no other; scales
    next to the ends of fp32's range, and zeros."""
    N, K = 512, 384
    g = gen(M)
    x, sx, xv, ld = operand(M, K, 0, 1, g)
    w, sw, wv, _ = operand(N, K, 0, 128, g, K ** -0.5)
    e = m.MOE_DTYPE_E4M3
    clean = torch.empty(M, N, device=DEV)
    p = m.linear_problem(M, N, K, e, m.MOE_DTYPE_F32)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    m.moe_linear_fp8(p, x, sx, w, sw, None, None, clean, ws)
    x, w, sx = x.clone(), w.clone(), sx.clone()
    x[1, 7], sx[3, 1], w[9, 200] = 0x7f, float("inf"), 0xff
    y = torch.empty(M, N, device=DEV)
    m.moe_linear_fp8(p, x, sx, w, sw, None, None, y, ws)
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 9]).all() and not torch.isfinite(y[3]).any()
    keep = [i for i in range(M) if i not in (1, 3)]
    cols = [i for i in range(N) if i != 9]
    assert torch.equal(y[keep][:, cols], clean[keep][:, cols])
    # h next to fp32's least: its group's scale has no normal reciprocal
    h, s = torch.zeros(M, N // 2, dtype=torch.uint8, device=DEV), torch.zeros(M, 2, device=DEV)
    q = m.gated_problem(M, N // 2, K, e, e, act=m.MOE_ACT_NONE)
    sw2 = torch.full((2, 2, 3), 1.0, device=DEV)
    sw2[0] = 2e-38
    _, sx, _, _ = operand(M, K, 0, 1, g)
    w[9, 200], x[1, 7] = 0, 0
    wq = torch.cat([w[:256], w[256:]])
    m.moe_gated_fp8(q, x, torch.full_like(sx, 1e-3), wq, sw2, None, h, s, ws)
    assert torch.isfinite(s).all() and ((h & 0x7f) != 0x7f).all()
    m.moe_gated_fp8(q, x, torch.zeros_like(sx), wq, sw2, None, h, s, ws)
    assert (s == 1).all() and ((h & 0x7f) == 0).all()


def test_repeats_bit_for_bit_on_streams_and_in_a_graph(m):  # noqa: F811
    e = m.MOE_DTYPE_E4M3
    for M, N, K in ((8, 256, 4096), (14, 128, 512), (40, 256, 4096), (600, 256, 512), (6000, 1024, 256)):
        g = gen(M)
        x, sx, _, _ = operand(M, K, 0, 1, g)
        w, sw, _, _ = operand(2 * N, K, 0, 128, g, K ** -0.5)
        w2, sw2, _, _ = operand(K, N, 0, 128, g, N ** -0.5)
        pg, pl = m.gated_problem(M, N, K, e, e), m.linear_problem(M, K, N, e)
        sw = sw.view(2, N // 128, -1)
        outs = []
        for how in ("plain", "stream", "graph"):
            h, hs = torch.empty(M, N, dtype=torch.uint8, device=DEV), torch.empty(M, N // 128, device=DEV)
            y = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
            ws = [torch.empty(256, dtype=torch.uint8, device=DEV) for _ in range(2)]

            def both(stream=None):
                m.moe_gated_fp8(pg, x, sx, w, sw, None, h, hs, ws[0], stream=stream)
                m.moe_linear_fp8(pl, h, hs, w2, sw2, None, None, y, ws[1], stream=stream)

            torch.cuda.synchronize()
            if how == "graph":
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    both()
                for t in (h, hs, y):
                    t.zero_()
                graph.replay()
                graph.replay()
            else:
                both(torch.cuda.Stream() if how == "stream" else None)
            torch.cuda.synchronize()
            assert all(m.moe_read_device_status(v) == m.MOE_OK for v in ws)
            outs.append((h, hs, y))
        for r in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(outs[0], r))


def test_two_streams_at_once(m):  # noqa: F811
    """Layers of every form side by side on two streams, each with outputs and workspaces of its own, leave
    what they leave one after the other."""
    e, g = m.MOE_DTYPE_E4M3, gen(8)
    calls = []
    for M, N, K in ((3000, 512, 384), (50, 256, 1024), (8, 512, 1024), (12, 256, 512)):
        x, sx, _, _ = operand(M, K, 0, 1, g)
        w, sw, _, _ = operand(2 * N, K, 0, 128, g, K ** -0.5)
        xb, wb = rows(M, K, K, torch.bfloat16, g), rows(2 * N, K, K, torch.bfloat16, g, K ** -0.5)
        pl, pg, pb = m.linear_problem(M, 2 * N, K, e), m.gated_problem(M, N, K, e, e), m.gated_problem(M, N, K)

        def call(out, stream, x=x, sx=sx, w=w, sw=sw, xb=xb, wb=wb, pl=pl, pg=pg, pb=pb):
            m.moe_linear_fp8(pl, x, sx, w, sw, None, None, out[0], out[4], stream=stream)
            m.moe_gated_fp8(pg, x, sx, w, sw.view(2, -1, sw.shape[1]), None, out[1], out[2], out[5], stream=stream)
            m.moe_gated(pb, xb, wb, None, out[3], None, out[6], stream=stream)

        def fresh(M=M, N=N):
            return ([torch.zeros(M, 2 * N, dtype=torch.bfloat16, device=DEV), torch.zeros(M, N, dtype=torch.uint8, device=DEV),
                     torch.zeros(M, N // 128, device=DEV), torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)] +
                    [torch.empty(256, dtype=torch.uint8, device=DEV) for _ in range(3)])

        calls.append((call, fresh))
    want = []
    for call, fresh in calls:
        want.append(fresh())
        call(want[-1], None)
        torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[fresh() for _, fresh in calls] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for k in range(len(calls)):
            for s, stream in enumerate(streams):
                i = (k + s) % len(calls)
                calls[i][0](got[s][i], stream)
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(a[:4], b[:4]))
            assert all(m.moe_read_device_status(ws) == m.MOE_OK for ws in a[4:])
