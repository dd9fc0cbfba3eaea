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


@pytest.mark.parametrize("gated,down", [((33, 64), (64, 16)), ((32, 64), (64, 15)), ((32, 64), (48, 16)), ((32,), (64, 16))])
def test_quantise_dense_refuses_weights_that_are_no_block(later, gated, down):
    """Halves of unequal rows, and a down projection of other sizes."""
    with pytest.raises(ValueError, match="w_gated"):
        block.quantise_dense(torch.zeros(gated), torch.zeros(down))
    assert not later


def test_quantise_dense_refuses_types(later):
    for gated, down in ((torch.float64, torch.float32), (torch.bfloat16, torch.uint8)):
        with pytest.raises(ValueError, match="16 or 32 bits"):
            block.quantise_dense(torch.zeros(32, 64, dtype=gated), torch.zeros(64, 16, dtype=down))
    assert not later


T, H, N = 4, 64, 144


def weights(quant, **other):
    """A block's weights and norms, with some of them replaced by zeros of (shape, dtype)."""
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    if quant == "bf16":
        given = dict(gated=((2 * N, H), bf16), down=((H, N), bf16))
    else:
        given = dict(gated=((2 * N, H), u8), gated_scale=((2, 2, 1), f32), down=((H, N), u8), down_scale=((1, 2), f32))
    norms = dict(post=((H,), f32), pre=((H,), f32), gate=((H,), f32))
    made = {k: None if v is None else torch.zeros(v[0], dtype=v[1]) for k, v in (given | norms | other).items()}
    return tuple(made[k] for k in given), tuple(made[k] for k in norms)


def make(quant, **other):
    w, norms = weights(quant, **other)
    return block.DenseBlock(T, H, N, w, norms, quant)


@pytest.mark.parametrize("quant,name,shape,dtype", [
    ("bf16", "gated", (2 * N - 1, H), torch.bfloat16), ("bf16", "gated", (N, H), torch.bfloat16),
    ("bf16", "gated", (2 * N, H + 8), torch.bfloat16), ("bf16", "gated", (2 * N, H), torch.float16),
    ("bf16", "down", (N, H), torch.bfloat16), ("bf16", "down", (H, N), torch.float32),
    ("fp8_block", "gated", (N, H), torch.uint8), ("fp8_block", "gated", (2 * N, H), torch.bfloat16),
    ("fp8_block", "gated_scale", (3, 1), torch.float32), ("fp8_block", "gated_scale", (2, 1, 1), torch.float32),
    ("fp8_block", "gated_scale", (2, 2, 1), torch.bfloat16), ("fp8_block", "down", (H, N - 16), torch.uint8),
    ("fp8_block", "down_scale", (2, 1), torch.float32), ("fp8_block", "down_scale", (1, 2), torch.float64),
    ("bf16", "post", (H - 1,), torch.float32), ("bf16", "pre", (H,), torch.bfloat16), ("fp8_block", "gate", (T, H), torch.float32)])
def test_dense_block_refuses_what_its_kernels_would_read_past(quant, name, shape, dtype):
    with pytest.raises(ValueError, match=name):
        make(quant, **{name: (shape, dtype)})


def test_dense_block_refuses_another_number_of_weights():
    w, norms = weights("bf16")
    with pytest.raises(ValueError, match="weights"):
        block.DenseBlock(T, H, N, w, norms, "fp8_block")
    w, norms = weights("fp8_block")
    with pytest.raises(ValueError, match="weights"):
        block.DenseBlock(T, H, N, w, norms, "bf16")


def test_dense_block_takes_what_quantise_dense_makes():
    make("bf16")
    make("bf16", gate=None)
    make("fp8_block")
    make("fp8_block", gated=((2 * N, H), torch.float8_e4m3fn), down=((H, N), torch.float8_e4m3fn))
