"""Refusals of the dense blocks' operators: every bad argument is turned down on the host,
before anything is launched (no GPU is needed)."""
import pytest

FAKE = 1 << 20  # an aligned, never-dereferenced address


@pytest.fixture(scope="module")
def m():
    import __graft_entry__

    __graft_entry__.build()
    import mixture_experts_layer_index_gb300 as mod

    return mod


def test_gated_refusals(m):
    bad, unsup = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED
    names, bnames = ["x", "w", "bias", "h", "z"], ["dh", "x", "w", "z", "dx", "dw", "dbias"]

    def fwd(p, ws=FAKE, nb=256, **kw):
        given = dict(x=FAKE, w=FAKE, h=FAKE) | kw
        return m.raw_status("moe_gated", p, *[given.get(n) for n in names], ws, nb, None)

    def bwd(p, ws=FAKE, nb=1 << 40, **kw):
        given = dict(dh=FAKE, x=FAKE, w=FAKE, z=FAKE, dx=FAKE, dw=FAKE) | kw
        return m.raw_status("moe_gated_backward", p, *[given.get(n) for n in bnames], ws, nb, None)

    ok = m.gated_problem(4, 24, 64)
    for kw in (dict(x=None), dict(w=None), dict(h=None), dict(x=FAKE + 8), dict(w=FAKE + 2), dict(h=FAKE + 1),
               dict(bias=FAKE + 2), dict(z=FAKE + 1)):
        assert fwd(ok, **kw) == bad, kw
    for kw in (dict(dh=None), dict(x=None), dict(w=None), dict(z=None), dict(x=FAKE + 8), dict(dx=FAKE + 1), dict(dw=FAKE + 1),
               dict(dbias=FAKE + 2), dict(dh=FAKE + 1), dict(z=FAKE + 1)):
        assert bwd(ok, **kw) == bad, kw
    for p in (m.gated_problem(-1, 24, 64), m.gated_problem(4, -1, 64), m.gated_problem(4, 24, 0), m.gated_problem(4, 24, 64, dtype=4),
              m.gated_problem(4, 24, 64, out_dtype=-1), m.gated_problem(4, 24, 64, bias_dtype=9), m.gated_problem(4, 24, 64, act=5),
              m.gated_problem(4, 24, 64, ld_x=56), m.gated_problem(4, 24, 64, ld_w=56), m.gated_problem(4, 24, 64, ld_h=23)):
        assert fwd(p) == bad and bwd(p) == bad
        assert m.moe_gated_workspace_size(p) == 0 and m.moe_gated_backward_workspace_size(p) == 0
    for p in (m.gated_problem(4, 24, 64, dtype=m.MOE_DTYPE_F32), m.gated_problem(4, 24, 60), m.gated_problem(4, 24, 64, ld_x=68),
              m.gated_problem(4, 24, 64, ld_w=65), m.gated_problem(1 << 30, 1 << 29, 64), m.gated_problem(4, (1 << 29) + 1, 64)):
        assert fwd(p) == unsup and bwd(p) == unsup
        assert m.moe_gated_workspace_size(p) == 0 and m.moe_gated_backward_workspace_size(p) == 0
    assert fwd(None) == bad and bwd(None) == bad
    for f, need in ((fwd, m.moe_gated_workspace_size(ok)), (bwd, m.moe_gated_backward_workspace_size(ok))):
        assert need >= 256
        assert f(ok, ws=None) == m.MOE_ERR_WORKSPACE
        assert f(ok, ws=FAKE + 16) == m.MOE_ERR_WORKSPACE
        assert f(ok, nb=need - 1) == m.MOE_ERR_WORKSPACE
    empty = m.gated_problem(0, 24, 64)
    assert fwd(empty, x=None, w=None, h=None, ws=None, nb=0) == m.MOE_OK


def test_gated_binding_checks_rows(m):
    torch = pytest.importorskip("torch")
    p = m.gated_problem(4, 24, 64)
    with pytest.raises(ValueError, match="device tensor"):
        m.moe_gated(p, torch.zeros(4, 64), FAKE, None, FAKE, None, FAKE, 256, stream=0)
    with pytest.raises(m.MoeError) as e:
        m.moe_gated(p, FAKE, None, None, FAKE, None, FAKE, 256, stream=0)
    assert e.value.status == m.MOE_ERR_INVALID_ARG


def test_quantise_refusals(m):
    bad, unsup = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED

    def call(p, **kw):
        given = dict(x=FAKE, q=FAKE, scale=FAKE) | kw
        return m.raw_status("moe_quantise", p, given["x"], given["q"], given["scale"], None)

    ok = m.quantise_problem(4, 200)
    for kw in (dict(x=None), dict(q=None), dict(scale=None), dict(x=FAKE + 1), dict(scale=FAKE + 2)):
        assert call(ok, **kw) == bad, kw
    assert call(m.quantise_problem(4, 200, m.MOE_DTYPE_F32), x=FAKE + 2) == bad
    for p in (m.quantise_problem(-1, 200), m.quantise_problem(4, 0), m.quantise_problem(4, 200, dtype=m.MOE_DTYPE_E4M3),
              m.quantise_problem(4, 200, block_rows=2), m.quantise_problem(4, 200, ld_x=199), m.quantise_problem(4, 200, ld_q=199)):
        assert call(p) == bad
    assert call(None) == bad
    assert call(m.quantise_problem(1 << 30, 1 << 16, block_rows=128)) == unsup
    assert call(m.quantise_problem(0, 200), x=None, q=None, scale=None) == m.MOE_OK


def test_fp8_refusals(m):
    bad, unsup, e = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED, m.MOE_DTYPE_E4M3
    names, gnames = ["x", "x_scale", "w", "w_scale", "bias", "residual", "y"], ["x", "x_scale", "w", "w_scale", "bias", "h", "h_scale"]

    def lin(p, ws=FAKE, nb=256, **kw):
        given = dict(x=FAKE, x_scale=FAKE, w=FAKE, w_scale=FAKE, y=FAKE) | kw
        return m.raw_status("moe_linear_fp8", p, *[given.get(n) for n in names], ws, nb, None)

    def gat(p, ws=FAKE, nb=256, **kw):
        given = dict(x=FAKE, x_scale=FAKE, w=FAKE, w_scale=FAKE, h=FAKE) | kw
        return m.raw_status("moe_gated_fp8", p, *[given.get(n) for n in gnames], ws, nb, None)

    L, G = m.linear_problem, m.gated_problem
    ok, okg, okc = L(4, 24, 64, e), G(4, 24, 64, e), G(4, 32, 64, e, e)
    for kw in (dict(x=None), dict(w=None), dict(x_scale=None), dict(w_scale=None), dict(x=FAKE + 8), dict(w=FAKE + 4),
               dict(x_scale=FAKE + 2), dict(w_scale=FAKE + 1), dict(bias=FAKE + 2)):
        assert lin(ok, **kw) == bad and gat(okg, **kw) == bad and gat(okc, h_scale=FAKE, **kw) == bad, kw
    assert lin(ok, y=None) == bad and lin(ok, y=FAKE + 1) == bad and lin(ok, residual=FAKE + 1) == bad
    assert gat(okg, h=None) == bad and gat(okg, h=FAKE + 1) == bad and gat(okg, h_scale=FAKE) == bad
    assert gat(okc) == bad and gat(okc, h_scale=FAKE, h=FAKE + 8) == bad and gat(okc, h_scale=FAKE + 2) == bad
    for kw in (dict(M=-1), dict(N=-1), dict(K=0), dict(dtype=m.MOE_DTYPE_BF16), dict(out_dtype=4), dict(out_dtype=-1),
               dict(bias_dtype=e), dict(act=5), dict(ld_x=48), dict(ld_w=48)):
        a = dict(M=4, N=24, K=64, dtype=e) | kw
        for p, f, size in ((L(**a), lin, m.moe_linear_fp8_workspace_size), (G(**a), gat, m.moe_gated_fp8_workspace_size)):
            assert f(p) == bad and size(p) == 0, kw
    assert lin(L(4, 24, 64, e, e)) == bad and lin(L(4, 24, 64, e, ld_y=23)) == bad and gat(G(4, 24, 64, e, ld_h=23)) == bad
    assert lin(L(4, 24, 64, e, alpha=float("nan"))) == bad
    for kw in (dict(K=60), dict(ld_x=72), dict(ld_w=72), dict(M=1 << 30, N=1 << 29)):
        a = dict(M=4, N=24, K=64, dtype=e) | kw
        assert lin(L(**a)) == unsup and gat(G(**a)) == unsup, kw
    assert gat(G(4, 24, 64, e, e), h_scale=FAKE) == unsup  # codes in rows of no whole 16 bytes
    assert gat(G(4, 32, 64, e, e, ld_h=40), h_scale=FAKE) == unsup
    assert lin(None) == bad and gat(None) == bad
    for f, p, kw in ((lin, ok, {}), (gat, okg, {}), (gat, okc, dict(h_scale=FAKE))):
        assert f(p, ws=None, **kw) == m.MOE_ERR_WORKSPACE
        assert f(p, ws=FAKE + 16, **kw) == m.MOE_ERR_WORKSPACE
        assert f(p, nb=255, **kw) == m.MOE_ERR_WORKSPACE
    assert lin(L(0, 24, 64, e), x=None, w=None, y=None, ws=None, nb=0) == m.MOE_OK
    # the 16-bit entry points take no codes
    assert m.moe_linear_workspace_size(ok) == 0 and m.moe_gated_workspace_size(okg) == 0


class Device:
    """A CPU tensor that says it is on the GPU: its layout is looked at, its memory is not."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_rows_that_the_descriptor_does_not_name(m, monkeypatch):
    torch = pytest.importorskip("torch")
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or m.MOE_OK

    monkeypatch.setattr(m, "lib", lambda: Lib())

    def dev(rows, cols, ld=None, dtype=torch.float32):
        return Device(torch.zeros(rows, ld or cols, dtype=dtype)[:, :cols])

    M, N, K, ld = 4, 24, 64, 80
    x, w, h, z = dev(M, K), dev(2 * N, K), dev(M, N), dev(M, 2 * N)
    p = m.gated_problem(M, N, K)
    m.moe_gated(p, x, w, None, h, z, FAKE, 256, stream=0)
    m.moe_gated_backward(p, h, x, w, z, x, w, None, FAKE, 256, stream=0)
    wide = {"x": dev(M, K, ld), "w": dev(2 * N, K, ld), "h": dev(M, N, ld)}
    for name in wide:
        a = {"x": x, "w": w, "h": h} | {name: wide[name]}
        with pytest.raises(ValueError, match="elements apart"):
            m.moe_gated(p, a["x"], a["w"], None, a["h"], None, FAKE, 256, stream=0)
        with pytest.raises(ValueError, match="elements apart"):
            m.moe_gated_backward(p, a["h"], a["x"], a["w"], z, None, None, None, FAKE, 256, stream=0)
        with pytest.raises(ValueError, match="elements apart"):
            m.moe_gated_fp8(p, a["x"], FAKE, a["w"], FAKE, None, a["h"], None, FAKE, 256, stream=0)
    q = m.gated_problem(M, N, K, ld_x=ld, ld_w=ld, ld_h=ld)
    m.moe_gated(q, wide["x"], wide["w"], None, wide["h"], None, FAKE, 256, stream=0)
    l, y, wl = m.linear_problem(M, N, K, m.MOE_DTYPE_E4M3), dev(M, N), dev(N, K)
    m.moe_linear_fp8(l, x, FAKE, wl, FAKE, None, y, y, FAKE, 256, stream=0)
    for a in ((wide["x"], wl, y, y), (x, dev(N, K, ld), y, y), (x, wl, wide["h"], y), (x, wl, y, wide["h"])):
        with pytest.raises(ValueError, match="elements apart"):
            m.moe_linear_fp8(l, a[0], FAKE, a[1], FAKE, None, a[2], a[3], FAKE, 256, stream=0)
    k = m.quantise_problem(M, K, ld_q=ld)
    m.moe_quantise(k, x, dev(M, K, ld, torch.uint8), FAKE, stream=0)
    for a in ((wide["x"], dev(M, K, ld, torch.uint8)), (x, dev(M, K, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="elements apart"):
            m.moe_quantise(k, *a, FAKE, stream=0)
    assert len(seen) == 5
