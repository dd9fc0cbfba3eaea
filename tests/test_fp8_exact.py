"""The gated layer's e4m3 output where its arithmetic is exact: every sum is a few products of small integers
times powers of two, so that codes and scales are the quantiser's bit for bit, in every form of the kernel."""
import numpy as np
import pytest
import torch

from oracle import dense as D
from tests.test_block_ops import DEV, m  # noqa: F401  (m: a fixture)
from tests.test_fp8_ops import same_codes

pytestmark = pytest.mark.gpu

# a few rows, one SM with the sum split, pairs of SMs
FORMS = [(1, 200, 128), (8, 512, 300), (40, 200, 2048), (100, 528, 4096), (300, 512, 256), (700, 1030, 128), (4096, 520, 128)]
SCALES = [(-15, 0, 0), (0, -10, 4), (-6, -60, -72), (28, 27, 27), (-30, -38, -40)]  # exponents of those of x, gate, up


def exact_case(M, N, K, ex, eg, eu, seed=0):
    """Codes and scales of x [M, K] and w [2 N, K], and the fp32 values of gate and up.  g = c n and u = d: quotients
    by a group's scale 448 c d / 448 are the n, which lie on e4m3's codes, on the midpoints between them, and at 448."""
    rng = np.random.default_rng(M + N + K + seed)
    c, d = (rng.choice(np.arange(1, 16, 2), M) * rng.choice([-1, 1], M) for _ in range(2))
    if M > 1:
        c[-1] = 0  # a row of zeros
    high = 16 * 2.0 ** rng.integers(-6, 4, N)
    low = high / 16 * rng.integers(0, 16, N)
    full = np.arange(N) % 128 == rng.integers(0, N % 128 or 128)  # 448 = 256 + 192 in each group
    high[full], low[full] = 256, 192
    k = rng.choice(K, 3, replace=False)  # where in the sum the products lie
    x, wg, wu = np.zeros((M, K)), np.zeros((N, K)), np.zeros((N, K))
    x[:, k[0]], x[:, k[1]], x[:, k[2]] = c, c, d
    wg[:, k[0]], wg[:, k[1]], wu[:, k[2]] = high, low, 1
    for v in (x, wg, wu):
        assert np.array_equal(D.e4m3_decode(D.e4m3_encode(v.astype(np.float32))), v)
    nk, nb = -(-K // 128), -(-N // 128)
    sx = torch.full((M, nk), 2.0 ** ex, device=DEV)
    sw = torch.stack([torch.full((nb, nk), 2.0 ** e, device=DEV) for e in (eg, eu)])
    x, wg, wu = (torch.from_numpy(D.e4m3_encode(v.astype(np.float32))).to(DEV) for v in (x, wg, wu))
    g, u = np.outer(c, high + low) * 2.0 ** (ex + eg), np.outer(d, np.ones(N)) * 2.0 ** (ex + eu)
    return x, sx, torch.cat([wg, wu]), sw, g.astype(np.float32), u.astype(np.float32)


def padded(q):
    M, K = q.shape
    buf = torch.full((M, -(-K // 16) * 16), 0x7f, dtype=torch.uint8, device=DEV)
    buf[:, :K] = q
    return buf[:, :K], buf.shape[1]


def gated(m, x, sx, w, sw, N, bias=None, ld=0):  # noqa: F811
    """Codes and scales of the layer with no activation."""
    M, K = x.shape
    (x, ld_x), (w, ld_w) = padded(x), padded(w)
    ld = ld or -(-N // 32) * 32
    e = m.MOE_DTYPE_E4M3
    p = m.gated_problem(M, N, K, e, e, act=m.MOE_ACT_NONE, ld_x=ld_x, ld_w=ld_w, ld_h=ld)
    h = torch.full((M, ld), 0x7f, dtype=torch.uint8, device=DEV)  # what no call may leave
    s = torch.full((M, -(-N // 128)), float("nan"), device=DEV)
    ws = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
    m.moe_gated_fp8(p, x, sx, w, sw, bias, h[:, :N], s, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    return h[:, :N].cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("ex,eg,eu", SCALES)
def test_codes_of_h_are_the_quantisers(m, M, N, K, ex, eg, eu):  # noqa: F811
    """Quotients on e4m3's midpoints under scales that are no powers of two, up to fp32's largest, and down to
    subnormal ones (1e-43) without a reciprocal in fp32."""
    for seed in range(6 if M <= 8 else 1):
        x, sx, w, sw, g, u = exact_case(M, N, K, ex, eg, eu, seed)
        want, scales = D.quantise(g * u, 1)
        if 2 * ex + eg + eu < -135:
            assert 0 < scales.min() < 2.9e-39
        for ld in (0, (N + 15) // 16 * 16):
            got, s = gated(m, x, sx, w, sw, N, ld=ld)
            assert np.array_equal(s, scales)
            assert same_codes(got, want)


@pytest.mark.parametrize("M,N,K", FORMS)
def test_infinite_and_nan_h(m, M, N, K):  # noqa: F811
    """An infinite h makes its group's scale infinite, its own code NaN and the others 0; a NaN has no part in the
    scale and the code NaN: what the quantiser does with the same h."""
    x, sx, w, sw, g, u = exact_case(M, N, K, 0, 0, 0)
    bias = torch.zeros(2 * N, device=DEV)
    bias[3], bias[N - 2], bias[N + 7] = float("inf"), float("nan"), -float("inf")
    b = bias.cpu().numpy()
    with np.errstate(invalid="ignore"):
        want, scales = D.quantise((g + b[:N]) * (u + b[N:]), 1)
    assert np.isinf(scales[:, 0]).all() and np.isfinite(scales[:, -1]).all()
    got, s = gated(m, x, sx, w, sw, N, bias)
    assert np.array_equal(s, scales)
    assert same_codes(got, want)


ENDS = {"low": (-80, -60, 1.0), "high": (58, 66, 2.0 ** -9)}  # exponents of the scales, least code


def end_case(M, N, K, end, up=False):
    """Codes and scales whose products pass fp32's normal range: x, sx, w, sw with one set of weights or, for the
    gated layer, one and an up projection's in the middle of the range.  Every third row's scales make normal
    products.  The second group has codes of 0 in every other row, and there and in the next rows a product of
    scales that overflows; the third has a scale of 0 beside a large one."""
    lo, hi, least = ENDS[end]
    rng = np.random.default_rng(M + N + K + up)
    scale = lambda *s: (rng.uniform(1, 2, s) * 2.0 ** rng.integers(lo, hi, s)).astype(np.float32)  # noqa: E731
    nk, nb, parts = -(-K // 128), -(-N // 128), 2 if up else 1
    x, w = (rng.integers(-3, 4, s) * least for s in ((M, K), (parts, N, K)))
    sx, sw = scale(M, nk), scale(parts, nb, nk)
    sx[::3] = 2.0 ** -5 if end == "low" else 2.0 ** 40
    if up:
        sw[1] = (2.0 ** 62 if end == "low" else 2.0 ** -58) * (1 + np.arange(nk) / 8)
    x[::2, 128:256] = 0
    sx[:, 1] = np.where(np.arange(M) % 4 < 2, 1e30, 0)
    sw[..., 1] = 1e20
    sx[:, 2], sw[..., 2] = 0, 3e38
    return x, sx, w, sw


def sums(x, sx, w, sw):
    """z and the sum of its terms' magnitudes, with the definition's order of rounding: the product of a group's
    scales in fp32, all else in 64 bits."""
    z, mag = np.zeros((2, x.shape[0], w.shape[0]))
    with np.errstate(all="ignore"):
        for kb in range(sx.shape[1]):
            at = np.s_[:, kb * 128:(kb + 1) * 128]
            f = (sx[:, kb, None] * sw[:, kb].repeat(128)[:w.shape[0]]).astype(np.float64)
            z += f * (x[at] @ w[at].T)
            mag += np.abs(f) * (np.abs(x[at]) @ np.abs(w[at]).T)
    return z, mag


def on_device(x, sx, w, sw):
    code = lambda v: padded(torch.from_numpy(D.e4m3_encode(v.astype(np.float32))).to(DEV))  # noqa: E731
    (x, ld_x), (w, ld_w) = code(x), code(w.reshape(-1, w.shape[2]))
    return x, torch.from_numpy(sx).to(DEV), w, torch.from_numpy(sw).to(DEV), ld_x, ld_w


def compare(got, ref, bound):
    got = got.double().cpu().numpy()
    finite = np.isfinite(ref)
    assert 0.1 < finite.mean() < 1
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    assert np.all(np.abs(got[finite] - ref[finite]) <= bound[finite])


# few rows in both widths, one SM, one SM with the sum split, pairs of SMs
@pytest.mark.parametrize("M,N,K", [(5, 200, 600), (14, 512, 700), (40, 200, 520), (40, 264, 4096), (200, 512, 640), (4096, 520, 520)])
@pytest.mark.parametrize("end", ENDS)
def test_scales_whose_product_is_no_normal_number(m, M, N, K, end):  # noqa: F811
    """The scales' product is rounded to fp32 before the sum is multiplied by it: subnormal, it has fewer bits; an
    infinite one makes a sum infinite, and one of 0 NaN."""
    e, f32 = m.MOE_DTYPE_E4M3, m.MOE_DTYPE_F32
    steps = K / 8 + 16  # roundings on a sum's way, as in tests/test_fp8_ops.py
    least = 2.0 ** -149 * (K / 128 + 1)  # a subnormal result is rounded to the least of them
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    case = end_case(M, N, K, end)
    x, sx, w, sw, ld_x, ld_w = on_device(*case)
    y = torch.full((M, N), 7.0, device=DEV)
    m.moe_linear_fp8(m.linear_problem(M, N, K, e, f32, ld_x=ld_x, ld_w=ld_w), x, sx, w, sw, None, None, y, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    z, mag = sums(case[0], case[1], case[2][0], case[3][0])
    assert np.nanmax(np.where(np.isinf(z), 0, np.abs(z))) < 3e38
    compare(y, z, steps * 2.0 ** -24 * mag + least)

    case = end_case(M, N, K, end, up=True)
    x, sx, w, sw, ld_x, ld_w = on_device(*case)
    h = torch.full((M, N), 7.0, device=DEV)
    p = m.gated_problem(M, N, K, e, f32, act=m.MOE_ACT_NONE, ld_x=ld_x, ld_w=ld_w)
    m.moe_gated_fp8(p, x, sx, w, sw, None, h, None, ws)
    assert m.moe_read_device_status(ws) == m.MOE_OK
    (g, mg), (u, mu) = (sums(case[0], case[1], case[2][i], case[3][i]) for i in range(2))
    with np.errstate(all="ignore"):
        ref = g * u
        # each factor's roundings times the other, the product's own
        bound = 2.01 * steps * 2.0 ** -24 * mg * mu + least * (np.abs(u) + 1) + 2.0 ** -24 * np.abs(ref)
    assert np.nanmax(np.where(np.isinf(ref), 0, np.abs(ref))) < 3e38
    compare(h, ref, bound)
