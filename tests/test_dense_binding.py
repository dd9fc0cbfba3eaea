"""What block.py's functions for dense blocks do around the library's calls (no GPU is needed: the calls
are noted, and done later on the CPU, as a stream does them)."""
import pytest

torch = pytest.importorskip("torch")

from mixture_experts_layer_index_gb300 import block  # noqa: E402


@pytest.fixture()
def later(monkeypatch):
    """moe_quantise as a stream does it: some time after the call has returned."""
    queue = []

    def quantise(p, x, q, scale, stream=None):
        assert (p.M, p.K, p.block_rows) == (*x.shape, 128)
        assert q.shape == x.shape and q.is_contiguous() and scale.is_contiguous()
        assert scale.shape == (-(-p.M // 128), -(-p.K // 128))

        def work():
            q.copy_(x.to(torch.uint8))
            scale.fill_(float(x[0, 0]))

        queue.append((stream, work))

    monkeypatch.setattr(block, "moe_quantise", quantise)
    return queue


@pytest.mark.parametrize("N,H", [(128, 64), (200, 144), (16, 272)])
def test_quantise_dense_reads_nothing_that_its_calls_write(later, N, H):
    """The codes are the calls' own outputs: nothing is copied before the stream has come to them."""
    g = torch.Generator().manual_seed(N)
    wg, wd = (torch.randint(0, 256, s, generator=g).float() for s in ((2 * N, H), (H, N)))
    codes, scales, down, down_scales = block.quantise_dense(wg, wd)
    assert codes.shape == (2 * N, H) and scales.shape == (2, -(-N // 128), -(-H // 128))
    assert down.shape == (H, N) and down_scales.shape == (-(-H // 128), -(-N // 128))
    for _, work in later:
        work()
    assert torch.equal(codes, wg.to(torch.uint8)) and torch.equal(down, wd.to(torch.uint8))
    assert (scales[0] == wg[0, 0]).all() and (scales[1] == wg[N, 0]).all() and (down_scales == wd[0, 0]).all()
