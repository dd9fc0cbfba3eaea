"""A dense block of a model end to end (block.DenseBlock), in bf16 with its gradient and on e4m3
weights, each step against the oracle's from the values that the step before it left."""
import numpy as np
import pytest
import torch

from oracle import blocks as B
from oracle import dense as D
from tests.test_block_ops import DEV, STEP, check, f64, gen, m  # noqa: F401  (m: a fixture)
from tests.test_dense_ops import acts, gated_mag

pytestmark = pytest.mark.gpu


def inputs(T, H, N, gate, seed=3):
    g = gen(seed)
    wg = (torch.randn(2 * N, H, generator=g, device=DEV) * H ** -0.5).to(torch.bfloat16)
    wd = (torch.randn(H, N, generator=g, device=DEV) * N ** -0.5).to(torch.bfloat16)
    norms = [1 + 0.2 * torch.randn(H, generator=g, device=DEV) for _ in range(2)] + [
        0.5 + 0.2 * torch.randn(H, generator=g, device=DEV) if gate else None]
    h, o = (torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    return wg, wd, norms, h, o


def check_norms(b, h, o):
    post, pre, gate = b.norms
    ref_h, ref_x, mag_h, mag_x = B.norm(f64(h), f64(o), None if gate is None else {"kind": "channel", "values": f64(gate)},
                                        f64(post), None, f64(pre), None, "rms", "rms", 1e-6, 1.0, 1.0)
    check(b.h_out, ref_h, mag_h, 32, "h")
    check(b.x, ref_x, mag_x, 64, "x")


@pytest.mark.parametrize("T,H,N", [(1, 256, 512), (7, 264, 200), (300, 512, 1024), (1500, 256, 1032)])
@pytest.mark.parametrize("act,gate", [("silu", True), ("gelu", False)])
def test_dense_block(m, T, H, N, act, gate):  # noqa: F811
    from mixture_experts_layer_index_gb300.block import DenseBlock

    wg, wd, norms, h, o = inputs(T, H, N, gate)
    b = DenseBlock(T, H, N, (wg, wd), norms, act=acts(m, act), train=True)
    assert b.status() == m.MOE_OK
    h1, o1 = b.forward(h, o)
    assert b.status() == m.MOE_OK
    check_norms(b, h, o)
    ref, z, mag = D.gated(f64(b.x), f64(wg), None, act)
    steps = H / 8 + 16
    check(b.z, z, mag, steps, "z")
    check(b.a, ref, gated_mag(z, mag, act, steps), steps, "a")
    y, _, mag = B.linear(f64(b.a), f64(wd), None, None, "none", 1.0)
    check(o1, y, mag, N / 8 + 16, "o")
    # the gradient, step by step from what the block kept
    g = gen(T)
    do, dh = (torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    r = b.gradient(o, do, dh)
    lin = B.linear_backward(f64(do), f64(b.a), f64(wd), None, "none", 1.0)
    check(r.down_weight, *lin["dw"], T / 8 + 16, "down")
    _, da, dx, _ = b._grad
    check(da, *lin["dx"], H / 8 + 16, "da")
    ref = D.gated_backward(f64(da), f64(b.x), f64(wg), f64(b.z), act)
    u = 2.0 ** -8 * 1.01  # dz is rounded to bf16 before its products
    for got, n, terms in ((dx, "dx", 2 * N / 8 + 16), (r.gated_weight, "dw", T / 8 + 16)):
        v, mag, soft = ref[n]
        check(got, v, mag + 16 * STEP * soft / (terms * STEP + u), terms, n, u)
    post, pre, gv = b.norms
    ref = B.norm_backward(f64(dh), f64(dx), f64(b.h_out), f64(o), None if gv is None else {"kind": "channel", "values": f64(gv)},
                          f64(post), None, f64(pre), "rms", "rms", 1e-6, 1.0, 1.0)
    check(r.dh, *ref["dh"], 128, "dh")
    check(r.d_o, *ref["do"], 256, "do")
    for got, n in ((r.post_weight, "dw_post"), (r.pre_weight, "dw_pre")) + (((r.gate, "dgate"),) if gv is not None else ()):
        check(got, *ref[n], 256 + T / 16, n)


@pytest.mark.parametrize("T,H,N", [(1, 256, 512), (8, 272, 208), (14, 256, 512), (300, 512, 1040), (4000, 256, 1024)])
def test_fp8_dense_block(m, T, H, N):  # noqa: F811
    from mixture_experts_layer_index_gb300.block import DenseBlock, quantise_dense

    wg, wd, norms, h, o = inputs(T, H, N, True)
    q = quantise_dense(wg, wd)
    for codes, scale, w in ((q[0][:N], q[1][0], wg[:N]), (q[0][N:], q[1][1], wg[N:]), (q[2], q[3], wd)):
        rc, rs = D.quantise(w.float().cpu().numpy(), 128)
        assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scale.cpu().numpy(), rs)
    b = DenseBlock(T, H, N, q, norms, "fp8_block")
    assert b.status() == m.MOE_OK
    h1, o1 = b.forward(h, o)
    assert b.status() == m.MOE_OK
    check_norms(b, h, o)
    codes, scales = D.quantise(b.x.float().cpu().numpy(), 1)
    assert np.array_equal(b.x_codes.cpu().numpy(), codes) and np.array_equal(b.x_scale.cpu().numpy(), scales)
    w = np.concatenate([D.dequantise(q[0][i * N:(i + 1) * N].cpu().numpy(), q[1][i].cpu().numpy(), 128) for i in range(2)])
    ref, z, mag = D.gated(D.dequantise(codes, scales, 1), w, None, "silu")
    steps = H / 8 + 16
    off = steps * STEP * gated_mag(z, mag, "silu", steps)
    a = D.dequantise(b.a.cpu().numpy(), b.a_scale.cpu().numpy(), 1)
    full = f64(b.a_scale).repeat(128, 1)[:, :N]
    worst = np.pad(off, [(0, 0), (0, -N % 128)]).reshape(T, -1, 128).max(2).repeat(128, 1)[:, :N]
    # half an e4m3 step, and a value's own error as often as it can carry it over a midpoint
    bound = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * full) * (1 + 4 * STEP) + 1.07 * off + 2.0 ** -4 * worst
    assert np.all(np.abs(a - ref) <= bound)
    wv = D.dequantise(q[2].cpu().numpy(), q[3].cpu().numpy(), 128)
    check(o1, a @ wv.T, np.abs(a) @ np.abs(wv).T, N / 8 + 16, "o")


@pytest.mark.parametrize("quant", ["bf16", "fp8_block"])
def test_dense_and_routed_blocks_in_a_graph(m, quant):  # noqa: F811
    """A dense block, a routed one and a dense one again in one captured step, replayed with other inputs."""
    from mixture_experts_layer_index_gb300.block import DenseBlock, quantise_dense
    from tests.test_block import _block

    T, H, N = 70, 256, 384
    routed, _, _, _ = _block(m, quant, T, 16, 4, H, 128, dict())
    blocks = []
    for seed in (1, 2):
        wg, wd, norms, h, o = inputs(T, H, N, True, seed)
        blocks.append(DenseBlock(T, H, N, (wg, wd) if quant == "bf16" else quantise_dense(wg, wd), norms, quant))

    def step():
        state = blocks[0].forward(h, o)
        state = routed.forward(*state)
        return blocks[1].forward(*state)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (5, 6):
        _, _, _, h2, o2 = inputs(T, H, N, True, seed)
        h.copy_(h2)
        o.copy_(o2)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for t in (blocks[0].h_out, blocks[0].o_out, routed.h_out, routed.o_out, *out):
            t.zero_()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(b.status() == m.MOE_OK for b in (*blocks, routed))


def test_dense_block_refusals(m):  # noqa: F811
    from mixture_experts_layer_index_gb300.block import DenseBlock, quantise_dense

    wg, wd, norms, h, o = inputs(4, 64, 128, False)
    with pytest.raises(ValueError):
        DenseBlock(4, 64, 128, (wg, wd), norms, "fp8_tensor")
    with pytest.raises(ValueError):
        DenseBlock(4, 64, 128, quantise_dense(wg, wd), norms, "fp8_block", train=True)
    with pytest.raises(ValueError):
        DenseBlock(4, 60, 128, (wg, wd), norms)
    b = DenseBlock(4, 64, 128, (wg, wd), norms)
    b.forward(h, o)
    with pytest.raises(ValueError):
        b.gradient(o, o)


def test_status_covers_the_gradient(m):  # noqa: F811
    """A status that one of the gradient's calls left is read after the gradient, and the next gradient clears it."""
    from mixture_experts_layer_index_gb300.block import DenseBlock

    T, H, N = 40, 256, 200
    wg, wd, norms, h, o = inputs(T, H, N, True)
    b = DenseBlock(T, H, N, (wg, wd), norms, train=True)
    made = b._grad  # before the first gradient: no call allocates
    b.forward(h, o)
    b.gradient(o, h)
    assert b.status() == m.MOE_OK and b._grad is made
    for ws in made[3][:2]:
        ws[:256] = 255  # a status word that nobody else writes
        assert b.status() != m.MOE_OK
        b.gradient(o, h)
        assert b.status() == m.MOE_OK


def test_training_step_in_a_graph(m):  # noqa: F811
    """A captured forward and gradient on another stream, replayed with other inputs: what the calls give."""
    from mixture_experts_layer_index_gb300.block import DenseBlock

    T, H, N = 300, 256, 200
    wg, wd, norms, h, o = inputs(T, H, N, True)
    do = inputs(T, H, N, True, 9)[3]
    b = DenseBlock(T, H, N, (wg, wd), norms, train=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        b.forward(h, o)
        out = b.gradient(o, do, do)
    for seed in (5, 6):
        _, _, _, h2, o2 = inputs(T, H, N, True, seed)
        h.copy_(h2)
        o.copy_(o2)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for t in out:
            t.zero_()
        b.forward(h, o)
        b.gradient(o, do, do)
        assert b.status() == m.MOE_OK
        assert all(torch.equal(x, y) for x, y in zip(got, out))


@pytest.mark.parametrize("handle", [False, True])
def test_quantise_dense_on_a_busy_stream(m, handle):  # noqa: F811
    """On a stream that is not the current one and has other work ahead; the memory that the codes get was
    another tensor's, which the current stream still reads."""
    from mixture_experts_layer_index_gb300.block import quantise_dense

    N, H = 1024, 512
    wg, wd, _, _, _ = inputs(4, H, N, False)
    want = quantise_dense(wg, wd)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    before = [torch.full_like(t, 7) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    copies = [t.clone() for t in before]
    del before  # its memory is free on the current stream, which has not read it yet
    with torch.cuda.stream(stream):
        torch.cuda._sleep(5_000_000)
    got = quantise_dense(wg, wd, stream=stream.cuda_stream if handle else stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in copies)
