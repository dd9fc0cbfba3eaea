"""Pins of oracle/blocks.py on the CPU: gradients against central differences of the
forward, selection against brute force, closed forms."""
import itertools

import numpy as np
import pytest

from oracle import blocks as B


def _differences(f, v, step=1e-5):
    """Central differences of the scalar f along every element of v (float64, in place)."""
    out = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        keep = v[i]
        v[i] = keep + step
        up = f()
        v[i] = keep - step
        down = f()
        v[i] = keep
        out[i] = (up - down) / (2 * step)
    return out


def _close(a, b):
    # central differences: truncation step^2 times third derivatives, rounding 1e-16 / step
    assert np.max(np.abs(a - b)) <= 1e-6 * max(1.0, np.max(np.abs(b))), np.max(np.abs(a - b))


@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [True, False])))
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    s, dw = rng.standard_normal((4, 7)), rng.standard_normal((4, 3))
    s[1, 4] = -np.inf
    ids, _, _ = B.route(s, 3, score, renormalise=renorm, scale=1.7)

    def loss():
        p = B.probabilities(s, score)
        w = np.take_along_axis(p, ids.astype(np.int64), 1)
        if renorm:
            w = w / w.sum(axis=1, keepdims=True)
        return 1.7 * (w * dw).sum()

    live = np.isfinite(s)
    s0 = s.copy()
    d = _differences(loss, s)
    d[~live] = 0.0  # a masked score has no difference
    _close(B.route_backward(s0, ids, dw, score, renorm, 1.7), d)


def test_route_by_hand():
    s = np.array([[0.0, 2.0, 2.0, -np.inf, 1.0, 3.0, np.nan, -0.0]])
    assert B.route(s, 3)[0].tolist() == [[5, 1, 2]]               # a tie goes to the lower id
    assert B.route(s, 8)[0].tolist() == [[5, 1, 2, 4, 0, 7, 3, 6]]  # signed zeros tie, masked last
    ids, w, _ = B.route(s, 8, scale=2.0)
    assert w[0, 6:].tolist() == [0.0, 0.0] and abs(w.sum() - 2.0) < 1e-12
    # groups {0,1}, {2,3}, {4,5}, {6,7}: best keys 2, 2, 3, 0; sums of sigmoids in this order: 2, 0, 1, 3
    assert sorted(B.route(s, 2, n_group=4, topk_group=2)[0][0].tolist()) == [1, 5]
    assert B.route(s, 2, "sigmoid", n_group=4, topk_group=1, group_best=2)[0].tolist() == [[5, 4]]
    # the bias moves the selection, not the weight
    ids, w, _ = B.route(s, 1, "sigmoid", bias=np.array([9.0] + [0.0] * 7), renormalise=False)
    assert ids.tolist() == [[0]] and w.tolist() == [[0.5]]
    dead = np.full((1, 8), -np.inf)
    ids, w, _ = B.route(dead, 3, n_group=4, topk_group=2)
    assert ids.tolist() == [[0, 1, 2]] and w.tolist() == [[0.0, 0.0, 0.0]]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
def test_norm_gradient_against_differences(kind, gate, post, pre):
    rng = np.random.default_rng(5)
    T, H = 3, 6
    h, o = rng.standard_normal((T, H)), rng.standard_normal((T, H)) + 0.3
    wp, bp, wq, bq = (rng.standard_normal(H) for _ in range(4))
    dh, dx = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    g = None if gate is None else {"kind": gate,
                                   "values": rng.standard_normal({"channel": (H,), "token": (T,), "full": (T, H)}[gate])}
    post, pre = (kind if post else None), (kind if pre else None)

    def forward():
        return B.norm(h, o, g, wp, bp, wq, bq, post, pre, 1e-3, 0.7, 0.9)

    def loss():
        out, x, _, _ = forward()
        return (out * dh).sum() + ((x * dx).sum() if pre else 0.0)

    got = B.norm_backward(dh, dx if pre else None, forward()[0], o, g, wp, bp, wq, post, pre, 1e-3, 0.7, 0.9)
    _close(got["dh"][0], _differences(loss, h))
    _close(got["do"][0], _differences(loss, o))
    if post:
        _close(got["dw_post"][0], _differences(loss, wp))
        _close(got["db_post"][0], _differences(loss, bp))
    if pre:
        _close(got["dw_pre"][0], _differences(loss, wq))
        _close(got["db_pre"][0], _differences(loss, bq))
    if g:
        _close(got["dgate"][0], _differences(loss, g["values"]))


def test_norm_by_hand():
    h, o = np.zeros((1, 2)), np.array([[3.0, 4.0]])
    out, x, _, _ = B.norm(h, o, None, None, None, np.array([2.0, 1.0]), None, "rms", "layer", 0.0, 1.0, 1.0)
    r = np.sqrt(12.5)
    assert np.allclose(out, [[3 / r, 4 / r]]) and np.allclose(x, [[-2.0, 1.0]])


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_linear_gradient_against_differences(name):
    rng = np.random.default_rng(7)
    x, w, b, dy = (rng.standard_normal(s) for s in ((3, 4), (5, 4), (5,), (3, 5)))

    def loss():
        return (B.linear(x, w, b, None, name, 1.3)[0] * dy).sum()

    z = B.linear(x, w, b, None, name, 1.3)[1]
    got = B.linear_backward(dy, x, w, z, name, 1.3)
    _close(got["dx"][0], _differences(loss, x))
    _close(got["dw"][0], _differences(loss, w))
    _close(got["dbias"][0], _differences(loss, b))
