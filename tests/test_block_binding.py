"""What the Python binding of the operators around the routed FFN checks of its tensors'
layout, before the library is called (no GPU is needed)."""
import pytest

torch = pytest.importorskip("torch")


class Device:
    """A CPU tensor that says it is on the GPU: its layout is looked at, its memory is not."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture(scope="module")
def m():
    import __graft_entry__

    __graft_entry__.build()
    import mixture_experts_layer_index_gb300 as mod

    return mod


@pytest.fixture()
def calls(m, monkeypatch):
    """Status of a library whose entry points only note that they were reached."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or m.MOE_OK

    monkeypatch.setattr(m, "lib", lambda: Lib())
    return seen


def dev(*shape, dtype=torch.float32):
    return Device(torch.zeros(*shape, dtype=dtype))


def sliced(T, W, ld, dtype=torch.float32):
    return Device(torch.zeros(T, ld, dtype=dtype)[:, :W])


WRONG = "elements apart"


def refused(f, *args, match=WRONG, **kw):
    with pytest.raises(ValueError, match=match):
        f(*args, stream=0, **kw)


def test_rows_that_the_descriptor_does_not_name(m, calls):
    T, W, ld = 4, 50, 53
    wrong = [sliced(T, W, ld), Device(torch.zeros(1, W).expand(T, W)), Device(torch.zeros(2, T, 64)[:, :2, :W])]
    for t in wrong:  # the descriptor says contiguous rows
        with pytest.raises(ValueError, match=WRONG):
            m._rows(t, "t", W)
    with pytest.raises(ValueError, match=WRONG):
        m._rows(dev(T, W), "t", W, ld)
    with pytest.raises(ValueError, match="must be contiguous"):
        m._rows(Device(torch.zeros(W, T).t()), "t", W)
    with pytest.raises(ValueError, match="must be contiguous"):
        m._rows(Device(torch.zeros(2 * W)[::2]), "t", W)
    with pytest.raises(ValueError, match="device tensor"):
        m._rows(torch.zeros(T, W), "t", W)


def test_rows_as_the_descriptor_says(m):
    T, W, ld = 4, 50, 53
    for t, l in ((dev(T, W), 0), (dev(T, W), W), (sliced(T, W, ld), ld), (dev(T, ld), ld), (sliced(1, W, ld), 0),
                 (dev(T * ld), ld), (dev(2, T, W), 0), (Device(torch.zeros(2, T, ld)[:, :, :W]), ld), (dev(0, W), ld),
                 (Device(torch.zeros(T, ld)[:, :1]), ld)):
        assert m._rows(t, "t", W, l) == t.data_ptr()
    assert m._rows(None, "t", W) is None and m._rows(4096, "t", W, ld) == 4096


def test_every_array_of_rows_is_looked_at(m, calls):
    T, E, k, H = 6, 16, 4, 32
    opt, wide = m.route_options(), m.route_options(ld=20, ld_grad=24)
    ids, w = dev(T, k, dtype=torch.int32), dev(T, k)
    refused(m.moe_route_ex, opt, sliced(T, E, 20), T, E, k, ids, w)
    refused(m.moe_route_ex, wide, dev(T, E), T, E, k, ids, w)
    refused(m.moe_route_backward, wide, sliced(T, E, 20), T, E, k, ids, w, sliced(T, E, 20))
    m.moe_route_ex(wide, sliced(T, E, 20), T, E, k, ids, w, stream=0)
    m.moe_route_backward(wide, sliced(T, E, 20), T, E, k, ids, w, sliced(T, E, 24), stream=0)
    assert calls == ["moe_route_ex", "moe_route_backward"]
    calls.clear()

    b = torch.bfloat16
    p = m.norm_problem(T, H, gate=m.MOE_GATE_FULL, ld_h=40, ld_o=48)
    fwd = dict(h=sliced(T, H, 40, b), o=sliced(T, H, 48, b), gate=sliced(T, H, 48, b), w_post=dev(H), b_post=None,
               w_pre=dev(H), b_pre=None, h_out=sliced(T, H, 40, b), x_out=sliced(T, H, 48, b))
    for name in ("h", "o", "gate", "h_out", "x_out"):
        refused(m.moe_norm_forward, p, **{**fwd, name: dev(T, H, dtype=b)}, match=name + ": rows lie")
    m.moe_norm_forward(p, **fwd, stream=0)
    bwd = dict(dh_out=sliced(T, H, 40, b), dx_out=sliced(T, H, 48, b), h_out=sliced(T, H, 40, b), o=sliced(T, H, 48, b),
               gate=sliced(T, H, 48, b), w_post=dev(H), b_post=None, w_pre=dev(H), dh=sliced(T, H, 40, b),
               d_o=sliced(T, H, 48, b), dgate=sliced(T, H, 48, b), dw_post=dev(H), db_post=None, dw_pre=dev(H), db_pre=None,
               ws=dev(1 << 16))
    for name in ("dh_out", "dx_out", "h_out", "o", "gate", "dh", "d_o", "dgate"):
        refused(m.moe_norm_backward, p, **{**bwd, name: dev(T, H, dtype=b)}, match=name + ": rows lie")
    m.moe_norm_backward(p, **bwd, stream=0)
    token = m.norm_problem(T, H, gate=m.MOE_GATE_TOKEN, ld_h=40, ld_o=48)
    m.moe_norm_forward(token, **{**fwd, "gate": dev(T)}, stream=0)
    refused(m.moe_norm_forward, token, **{**fwd, "gate": Device(torch.zeros(T, 3)[:, 0])}, match="contiguous")
    assert calls == ["moe_norm_forward", "moe_norm_backward", "moe_norm_forward"]
    calls.clear()

    M, N, K = 6, 24, 64
    p = m.linear_problem(M, N, K, ld_x=72, ld_w=80, ld_y=25)
    fwd = dict(x=sliced(M, K, 72, b), w=sliced(N, K, 80, b), bias=None, residual=sliced(M, N, 25, b),
               y=sliced(M, N, 25, b), z=dev(M, N, dtype=b), ws=dev(256))
    for name, n in (("x", (M, K)), ("w", (N, K)), ("residual", (M, N)), ("y", (M, N))):
        refused(m.moe_linear, p, **{**fwd, name: dev(*n, dtype=b)}, match=name + ": rows lie")
    refused(m.moe_linear, p, **{**fwd, "z": sliced(M, N, 25, b)}, match="contiguous")
    m.moe_linear(p, **fwd, stream=0)
    bwd = dict(dy=sliced(M, N, 25, b), x=sliced(M, K, 72, b), w=sliced(N, K, 80, b), z=None, dx=dev(M, K, dtype=b),
               dw=dev(N, K, dtype=b), dbias=dev(N), ws=dev(1 << 16))
    for name, n in (("dy", (M, N)), ("x", (M, K)), ("w", (N, K))):
        refused(m.moe_linear_backward, p, **{**bwd, name: dev(*n, dtype=b)}, match=name + ": rows lie")
    m.moe_linear_backward(p, **bwd, stream=0)
    assert calls == ["moe_linear", "moe_linear_backward"]
