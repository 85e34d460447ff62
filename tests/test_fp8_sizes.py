"""Sizes past 31 bits, which the C calls cannot take, are refused by the binding before they are cut
to 32 bits (without a GPU: tensors without memory, and a library that must not be called)."""
import pytest
import torch

BIG = 2 ** 32 + 16                       # cut to 32 bits: 16


@pytest.fixture
def d(monkeypatch):
    from block_diffusion_speculative_02_gb300 import dflash

    class Library:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    monkeypatch.setattr(dflash, "load_library", lambda: Library())
    monkeypatch.setattr(dflash, "_here", lambda stream: (-1, None))
    return dflash


def new(dtype, *shape):
    return torch.empty(*shape, dtype=dtype, device="meta")


def rows(m, k):
    return new(torch.float8_e4m3fn, m, k), new(torch.float32, -(-k // 128), m)


def weight(*shape):
    *g, n, k = shape
    return (new(torch.float8_e4m3fn, *shape), new(torch.float32, *g, -(-n // 128), -(-k // 128)))


BF = torch.bfloat16


@pytest.mark.parametrize("m", [2 ** 31, 2 ** 32, BIG])
def test_rows_past_31_bits(d, m):
    ws = new(torch.uint8, 256)
    x = new(BF, m, 16)
    with pytest.raises(ValueError, match="2\\^31"):
        d.dflash_fp8_norm_rows(x, None, None, 1e-6, None, *rows(m, 16))
    with pytest.raises(ValueError, match="2\\^31"):
        d.dflash_fp8_silu_mul(new(BF, m, 32), *rows(m, 16))
    with pytest.raises(ValueError, match="2\\^31"):
        d.dflash_fp8_linear(*rows(m, 16), *weight(8, 16), new(BF, m, 8), ws)
    start = new(torch.int32, 2)
    with pytest.raises(ValueError, match="2\\^31"):
        d.dflash_fp8_grouped(*rows(m, 16), *weight(1, 8, 16), start, None, new(BF, m, 8), ws)
    with pytest.raises(ValueError, match="2\\^31"):            # rows of out alone
        d.dflash_fp8_grouped(*rows(5, 16), *weight(1, 8, 16), start, new(torch.int32, m),
                             new(BF, m, 8), ws)
    with pytest.raises(ValueError, match="2\\^31"):            # rows of x alone
        d.dflash_fp8_grouped(*rows(m, 16), *weight(1, 8, 16), start, new(torch.int32, 5),
                             new(BF, 5, 8), ws)


def test_features_and_columns_past_31_bits(d):
    ws = new(torch.uint8, 256)
    for shape in ((BIG, 16), (16, BIG), (2, BIG, 16), (BIG, 2, 16), (2, 16, BIG)):
        with pytest.raises(ValueError, match="2\\^31"):
            d.dflash_fp8_weight(new(BF, *shape), *weight(*shape))
    with pytest.raises(ValueError, match="2\\^31"):
        d.dflash_fp8_norm_rows(new(BF, 1, BIG), None, None, 1e-6, None, *rows(1, BIG))
    with pytest.raises(ValueError, match="2\\^31"):
        d.dflash_fp8_silu_mul(new(BF, 1, 2 * BIG), *rows(1, BIG))
    with pytest.raises(ValueError, match="2\\^31"):
        d.dflash_fp8_linear(*rows(1, 16), *weight(BIG, 16), new(BF, 1, BIG), ws)
    with pytest.raises(ValueError, match="2\\^31"):
        d.dflash_fp8_linear(*rows(1, BIG), *weight(8, BIG), new(BF, 1, 8), ws)
    with pytest.raises(ValueError, match="2\\^31"):
        d.dflash_fp8_grouped(*rows(1, 16), *weight(BIG, 1, 16), new(torch.int32, BIG + 1), None,
                             new(BF, 1, 1), ws)


def test_sizes_within_31_bits_reach_the_library(d):
    with pytest.raises(AssertionError, match="dflash_fp8_linear was called"):
        d.dflash_fp8_linear(*rows(2 ** 31 - 1, 16), *weight(8, 16), new(BF, 2 ** 31 - 1, 8),
                            new(torch.uint8, 256))
