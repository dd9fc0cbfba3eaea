"""Refusals of the operators around the routed FFN: every bad argument is turned down
on the host, before anything is launched (no GPU is needed)."""
import ctypes

import pytest

FAKE = 1 << 20  # an aligned, never-dereferenced address
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def m():
    import __graft_entry__

    __graft_entry__.build()
    import mixture_experts_layer_index_gb300 as mod

    return mod


def _rule(m, **kw):
    """Options of moe_route_ex with fields set by name, the bias as an address."""
    bias = kw.pop("bias", None)
    o = m.route_options()
    for k, v in kw.items():
        setattr(o, k, v)
    o.bias = bias
    return o


def test_route_refusals(m):
    def fwd(o, T=4, E=8, k=2, s=FAKE, ids=FAKE, w=FAKE):
        a = m.raw_status("moe_route_ex", o, s, T, E, k, ids, w, None)
        b = m.raw_status("moe_route_backward", o, s, T, E, k, ids, w, FAKE, None)
        assert a == b
        return a

    ok = _rule(m)
    bad = m.MOE_ERR_INVALID_ARG
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(s=None), dict(ids=None), dict(w=None), dict(s=FAKE + 2),
               dict(ids=FAKE + 1), dict(w=FAKE + 2)):
        assert fwd(ok, **kw) == bad, kw
    for kw in (dict(score_fn=2), dict(renormalise=2), dict(scale=0.0), dict(scale=INF), dict(scale=NAN), dict(dtype=3),
               dict(n_group=0), dict(n_group=3), dict(topk_group=0), dict(n_group=2, topk_group=3), dict(group_best=0),
               dict(group_best=3), dict(ld=7), dict(ld_grad=7), dict(bias=FAKE + 2), dict(n_group=8, topk_group=1)):
        assert fwd(_rule(m, **kw)) == bad, kw
    assert fwd(None) == bad
    assert fwd(ok, E=513) == m.MOE_ERR_UNSUPPORTED
    assert fwd(ok, E=64, k=33) == m.MOE_ERR_UNSUPPORTED
    assert fwd(_rule(m, n_group=64, topk_group=64), E=128) == m.MOE_ERR_UNSUPPORTED
    assert fwd(ok, T=1 << 30, k=2) == m.MOE_ERR_UNSUPPORTED
    assert fwd(_rule(m, dtype=m.MOE_DTYPE_BF16), s=FAKE + 1) == bad
    assert fwd(ok, T=0, s=None, ids=None, w=None) == m.MOE_OK
    assert m.raw_status("moe_route_backward", ok, FAKE, 4, 8, 2, FAKE, FAKE, None, None) == bad


def test_norm_refusals(m):
    bad = m.MOE_ERR_INVALID_ARG
    names = ["h", "o", "gate", "w_post", "b_post", "w_pre", "b_pre", "h_out", "x_out"]

    def fwd(p, **kw):
        given = dict(h=FAKE, o=FAKE, h_out=FAKE, x_out=FAKE)
        given.update(kw)
        return m.raw_status("moe_norm_forward", p, *[given.get(n) for n in names], None)

    ok = m.norm_problem(4, 64)
    for kw in (dict(h=None), dict(o=None), dict(h_out=None), dict(x_out=None), dict(gate=FAKE), dict(h=FAKE + 1),
               dict(w_pre=FAKE + 2), dict(b_post=FAKE + 1)):
        assert fwd(ok, **kw) == bad, kw
    for p in (m.norm_problem(-1, 64), m.norm_problem(4, 0), m.norm_problem(4, 64, post_norm=3),
              m.norm_problem(4, 64, pre_norm=-1), m.norm_problem(4, 64, gate=4), m.norm_problem(4, 64, h_dtype=3),
              m.norm_problem(4, 64, eps=-1.0), m.norm_problem(4, 64, eps=NAN), m.norm_problem(4, 64, alpha=INF),
              m.norm_problem(4, 64, beta=NAN), m.norm_problem(4, 64, ld_h=63), m.norm_problem(4, 64, ld_o=1),
              m.norm_problem(4, 64, gate=m.MOE_GATE_TOKEN)):
        assert fwd(p) == bad
    assert fwd(m.norm_problem(4, 64, pre_norm=m.MOE_NORM_NONE)) == bad                  # x_out without a pre norm
    assert fwd(m.norm_problem(4, 64, post_norm=m.MOE_NORM_NONE), w_post=FAKE) == bad    # a weight without its norm
    assert fwd(m.norm_problem(4, 64, gate=m.MOE_GATE_TOKEN), gate=FAKE + 2) == bad
    assert fwd(m.norm_problem(4, 16385)) == m.MOE_ERR_UNSUPPORTED
    assert fwd(m.norm_problem(4, 64, o_dtype=m.MOE_DTYPE_F16)) == m.MOE_ERR_UNSUPPORTED
    assert m.raw_status("moe_norm_forward", None, *[FAKE] * 9, None) == bad

    bnames = ["dh_out", "dx_out", "h_out", "o", "gate", "w_post", "b_post", "w_pre", "dh", "d_o", "dgate", "dw_post",
              "db_post", "dw_pre", "db_pre"]

    def bwd(p, ws=FAKE, nb=1 << 40, **kw):
        given = dict(dh_out=FAKE, dx_out=FAKE, h_out=FAKE, o=FAKE, dh=FAKE, d_o=FAKE)
        given.update(kw)
        return m.raw_status("moe_norm_backward", p, *[given.get(n) for n in bnames], ws, nb, None)

    for kw in (dict(dx_out=None), dict(h_out=None), dict(o=None), dict(dgate=FAKE), dict(dw_pre=FAKE + 2), dict(dh=FAKE + 1)):
        assert bwd(ok, **kw) == bad, kw
    assert bwd(m.norm_problem(4, 64, pre_norm=m.MOE_NORM_NONE)) == bad
    assert bwd(m.norm_problem(4, 64, post_norm=m.MOE_NORM_NONE), dw_post=FAKE) == bad
    need = m.moe_norm_backward_workspace_size(ok)
    assert need > 0
    assert bwd(ok, ws=None) == m.MOE_ERR_WORKSPACE
    assert bwd(ok, nb=need - 1) == m.MOE_ERR_WORKSPACE
    assert bwd(ok, ws=FAKE + 8) == m.MOE_ERR_WORKSPACE
    assert m.moe_norm_backward_workspace_size(m.norm_problem(4, 16385)) == 0


def test_linear_refusals(m):
    bad, unsup = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED
    names = ["x", "w", "bias", "residual", "y", "z"]

    def fwd(p, ws=FAKE, nb=256, **kw):
        given = dict(x=FAKE, w=FAKE, y=FAKE)
        given.update(kw)
        return m.raw_status("moe_linear", p, *[given.get(n) for n in names], ws, nb, None)

    bnames = ["dy", "x", "w", "z", "dx", "dw", "dbias"]

    def bwd(p, ws=FAKE, nb=1 << 40, **kw):
        given = dict(dy=FAKE, x=FAKE, w=FAKE, dx=FAKE, dw=FAKE)
        given.update(kw)
        return m.raw_status("moe_linear_backward", p, *[given.get(n) for n in bnames], ws, nb, None)

    ok = m.linear_problem(4, 24, 64)
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=FAKE + 8), dict(w=FAKE + 2), dict(y=FAKE + 1),
               dict(bias=FAKE + 2), dict(residual=FAKE + 1), dict(z=FAKE + 1)):
        assert fwd(ok, **kw) == bad, kw
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(z=FAKE), dict(x=FAKE + 8), dict(dx=FAKE + 1),
               dict(dbias=FAKE + 2)):
        assert bwd(ok, **kw) == bad, kw
    for p in (m.linear_problem(-1, 24, 64), m.linear_problem(4, -1, 64), m.linear_problem(4, 24, 0),
              m.linear_problem(4, 24, 64, dtype=3), m.linear_problem(4, 24, 64, out_dtype=-1),
              m.linear_problem(4, 24, 64, bias_dtype=9), m.linear_problem(4, 24, 64, act=5),
              m.linear_problem(4, 24, 64, alpha=NAN), m.linear_problem(4, 24, 64, ld_x=56),
              m.linear_problem(4, 24, 64, ld_w=56), m.linear_problem(4, 24, 64, ld_y=23)):
        assert fwd(p) == bad and bwd(p) == bad
    for p in (m.linear_problem(4, 24, 64, dtype=m.MOE_DTYPE_F32), m.linear_problem(4, 24, 60),
              m.linear_problem(4, 24, 64, ld_x=68), m.linear_problem(4, 24, 64, ld_w=65)):
        assert fwd(p) == unsup and bwd(p) == unsup
        assert m.moe_linear_workspace_size(p) == 0 and m.moe_linear_backward_workspace_size(p) == 0
    assert fwd(None) == bad
    for f, need in ((fwd, m.moe_linear_workspace_size(ok)), (bwd, m.moe_linear_backward_workspace_size(ok))):
        assert need >= 256
        assert f(ok, ws=None) == m.MOE_ERR_WORKSPACE
        assert f(ok, ws=FAKE + 16) == m.MOE_ERR_WORKSPACE
        assert f(ok, nb=need - 1) == m.MOE_ERR_WORKSPACE
    q = m.linear_problem(4, 24, 64, act=m.MOE_ACT_SILU)
    assert bwd(q) == bad                                                                # an activation needs z
    assert fwd(m.linear_problem(0, 24, 64), x=None, w=None, y=None, ws=None, nb=0) == m.MOE_OK


def test_forward_routed_refusals(m):
    def fwd(p, opt=None, x=FAKE, ids=FAKE, w=FAKE, w1=FAKE, w2=FAKE, s1=None, s2=None, y=FAKE, ws=FAKE, nb=1 << 40):
        return m.raw_status("moe_forward_routed", ctypes.byref(p) if p else None, ctypes.byref(opt) if opt else None, x,
                            ids, w, w1, w2, s1, s2, y, ws, nb, None)

    bad = m.MOE_ERR_INVALID_ARG
    ok = m.problem(16, 8, 2, 256, 128)
    for kw in (dict(x=None), dict(ids=None), dict(w=None), dict(w1=None), dict(w2=None), dict(y=None), dict(ids=FAKE + 2),
               dict(w=FAKE + 1), dict(x=FAKE + 8), dict(y=FAKE + 2), dict(s1=FAKE)):
        assert fwd(ok, **kw) == bad, kw
    assert fwd(None) == bad
    assert fwd(ok, ws=None) == m.MOE_ERR_WORKSPACE
    assert fwd(ok, nb=m.moe_workspace_size(ok) - 1) == m.MOE_ERR_WORKSPACE
    assert fwd(m.problem(16, 8, 9, 256, 128)) == bad
    assert fwd(m.problem(16, 1000, 2, 256, 128)) == m.MOE_ERR_UNSUPPORTED
    assert fwd(m.problem(2, 32, 8, 512, 192, "fp8_tensor")) == bad  # no scales
    opt = m.moe_forward_options()
    opt.y_fp32 = 2
    assert fwd(ok, opt=opt) == bad
    assert fwd(m.problem(0, 8, 2, 256, 128), x=None, ids=None, w=None, y=None, ws=None, nb=0) == m.MOE_OK


def test_binding_checks_tensors(m):
    torch = pytest.importorskip("torch")
    p = m.linear_problem(4, 24, 64)
    with pytest.raises(ValueError, match="device tensor"):
        m.moe_linear(p, torch.zeros(4, 64), FAKE, None, None, FAKE, None, FAKE, 256, stream=0)
    with pytest.raises(m.MoeError) as e:
        m.moe_linear(p, FAKE, None, None, None, FAKE, None, FAKE, 256, stream=0)
    assert e.value.status == m.MOE_ERR_INVALID_ARG
