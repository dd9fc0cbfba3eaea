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
