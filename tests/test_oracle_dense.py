"""Pins of oracle/dense.py on the CPU: the gated layer against torch and its gradient against
differences, the quantiser against torch's float8 conversion and values worked out by hand."""
import numpy as np
import pytest
import torch

from oracle import dense as D
from tests.test_oracle_blocks import _close, _differences

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.mark.parametrize("name", ACTS)
def test_gated_against_torch(name):
    rng = np.random.default_rng(3)
    x, w, b = (rng.standard_normal(s) for s in ((4, 6), (10, 6), (10,)))
    t = torch.nn.functional
    f = {"none": lambda v: v, "relu": t.relu, "silu": t.silu, "gelu": t.gelu,
         "gelu_tanh": lambda v: t.gelu(v, approximate="tanh")}[name]
    z = torch.from_numpy(x) @ torch.from_numpy(w).T + torch.from_numpy(b)
    want = f(z[:, :5]) * z[:, 5:]
    h, got, mag = D.gated(x, w, b, name)
    assert np.allclose(h, want.numpy(), atol=1e-12) and np.allclose(got, z.numpy(), atol=1e-12)
    assert np.all(mag >= np.abs(got) - 1e-12)


@pytest.mark.parametrize("name", ACTS)
def test_gated_gradient_against_differences(name):
    rng = np.random.default_rng(4)
    x, w, b, dh = (rng.standard_normal(s) for s in ((3, 4), (10, 4), (10,), (3, 5)))

    def loss():
        return (D.gated(x, w, b, name)[0] * dh).sum()

    got = D.gated_backward(dh, x, w, D.gated(x, w, b, name)[1], name)
    _close(got["dx"][0], _differences(loss, x))
    _close(got["dw"][0], _differences(loss, w))
    _close(got["dbias"][0], _differences(loss, b))


@pytest.mark.parametrize("M,K,rows", [(3, 128, 1), (5, 300, 1), (130, 257, 128), (1, 1, 128)])
def test_quantise_against_torch(M, K, rows):
    rng = np.random.default_rng(M + K)
    v = (rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))).astype(np.float32)
    codes, s = D.quantise(v, rows)
    assert s.shape == (-(-M // rows), -(-K // 128))
    full = s.repeat(rows, 0)[:M].repeat(128, 1)[:, :K]
    want = torch.from_numpy(v / full).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    assert np.max(np.abs(D.dequantise(codes, s, rows) - v) / full) <= 16.0  # half a step at 448


def test_quantise_by_hand():
    v = np.zeros((2, 129), np.float32)
    v[0, 0], v[0, 1], v[0, 128] = 896.0, -1.0, 7.0
    codes, s = D.quantise(v, 1)
    assert s.tolist() == [[2.0, 7.0 / 448.0], [1.0, 1.0]]
    assert codes[0, 0] == 0x7e and codes[0, 1] == 0xb0 and codes[0, 128] == 0x7e and not codes[1].any()  # 448, -0.5
    v[0, 1], v[1, 0] = np.nan, np.inf
    codes, s = D.quantise(v, 1)
    assert s[0, 0] == 2.0 and codes[0, 1] & 0x7f == 0x7f and np.isinf(s[1, 0]) and codes[1, 0] & 0x7f == 0x7f and codes[1, 1] == 0
