"""Pins of the oracle of the linear layers in 8-bit floating point."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O


def test_decode_matches_every_code():
    c = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.decode(c), t, equal_nan=True)
    assert O.decode([0x7E])[0] == 448 and O.decode([0x08])[0] == 2.0 ** -6
    assert O.decode([0x01])[0] == 2.0 ** -9 and O.decode([0xB8])[0] == -1


def test_encode_is_the_nearest_code_with_ties_to_even():
    c = np.array([b for b in range(256) if (b & 127) != 127], np.uint8)
    assert np.array_equal(O.encode(O.decode(c)), c)
    pos = O.decode(np.arange(127, dtype=np.uint8))
    mid = (pos[:-1] + pos[1:]) / 2
    assert np.array_equal(O.encode(mid) % 2, np.zeros(126))          # the even neighbour
    y = np.random.default_rng(0).normal(size=100_000) * 100
    y = y[np.abs(y) <= 448]
    t = torch.from_numpy(y).float()
    assert np.array_equal(O.encode(t.double().numpy()),
                          t.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert np.array_equal(O.encode([1e9, -1e9, np.nan, -0.0]), [0x7E, 0xFE, 0x7F, 0x80])
    near = np.abs(O.decode(O.encode(y))[:, None] - y[:, None])
    assert (near <= np.abs(pos[None, :] - np.abs(y)[:, None]).min(axis=1, keepdims=True)).all()


def test_round_rows_worked_case():
    h = np.zeros((2, 130))
    h[0, 3], h[0, 127], h[0, 128], h[1, 129] = 896.0, -2.0, 7.0, -0.5
    q, s = O.round_rows(h)
    assert s.shape == (2, 2) and s[0, 0] == 2 and s[1, 0] == 7 / 448 and s[1, 1] == 0.5 / 448
    assert s[0, 1] == 2.0 ** -117 / 448
    v = O.rows_value(q, s)
    assert np.allclose(v, h, rtol=1e-15, atol=0)


def test_round_weight_has_a_scale_for_each_square():
    w = np.ones((2, 130, 144))
    w[1, 129, 143] = 4
    q, s = O.round_weight(w)
    assert s.shape == (2, 2, 2) and (s[0] == 1 / 448).all() and s[1, 1, 1] == 4 / 448
    assert np.allclose(O.weight_value(q, s), w, rtol=1e-15)


def test_norm_and_activation_closed_forms():
    x = np.full((1, 8), 3.0)
    s, h = O.norm_rows(x, residual=-x / 3, norm_w=np.arange(8.0), eps=0.0)
    assert (s == 2).all() and np.allclose(h, np.arange(8.0))
    _, h = O.norm_rows(np.random.default_rng(1).normal(size=(3, 16)), norm_w=np.ones(16), eps=0.0)
    assert np.allclose((h * h).mean(1), 1)
    g = np.linspace(-900, 900, 7)[None]
    a, b = O.silu_mul(np.hstack([g, np.ones_like(g)])), O.silu_mul(np.hstack([-g, np.ones_like(g)]))
    assert np.allclose(a - b, g)                                      # silu(x) - silu(-x) = x


@pytest.mark.parametrize("gather", [False, True])
def test_grouped_by_brute_force(gather):
    rng = np.random.default_rng(2)
    x, w = rng.normal(size=(5, 16)), rng.normal(size=(3, 4, 16))
    start = [1, 3, 3, 5]
    rows = [4, 2, 9, 0, 2, 1, 1] if gather else None
    out = np.full((7 if gather else 5, 4), 7.0)
    got = O.grouped(x, w, start, rows, out)
    want = out.copy()
    for e, (a, b) in enumerate(zip(start[:-1], start[1:])):
        for n in range(a, b):
            src = n if rows is None else rows[n]
            for j in range(4):
                want[n, j] = sum(w[e, j, k] * x[src, k] for k in range(16)) if src < 5 else 0
    assert np.allclose(got, want) and (got[0] == 7).all()
    assert (O.grouped(x, w, [2, 1, 9, 5], rows, out)[:1] == 7).all()   # bad groups left out


def test_grouped_rows_have_one_owner():
    x, w = np.ones((6, 2)), np.arange(1.0, 5.0)[:, None, None] * np.ones((4, 1, 2))
    got = O.grouped(x, w, [0, 4, 2, 5, 6], None, np.zeros((6, 1)))
    assert got[:, 0].tolist() == [2, 2, 2, 2, 0, 8]                   # 0 .. 3, not 2 .. 4, then 5
