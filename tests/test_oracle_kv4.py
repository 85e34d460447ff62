"""The 4-bit oracle against what its definitions fix."""
import numpy as np
import pytest

from oracle import kv4_oracle as O


def test_every_code_is_its_own_quantisation():
    """Rows whose largest element is 6 scale come back as they were, for every scale."""
    for s in range(1, 127):
        x = O.E2M1[[7, 0, 1, 2, 3, 4, 5, 6, 15, 9, 10, 11, 12, 13, 14, 7]] * O.E4M3[s]
        code, scale = O.quantise(x[None], [0])
        assert scale[0, 0] == s
        np.testing.assert_array_equal(O.values(code, scale, [0])[0], x)


@pytest.mark.parametrize("x,code", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4),
                                    (3.5, 6), (5.0, 6), (0.26, 1), (5.1, 7), (-0.75, 10)])
def test_halfway_cases_go_to_the_even_code(x, code):
    row = np.zeros(16)
    row[0], row[3] = 6.0, x
    assert O.quantise(row[None], [0])[0][0, 3] == code


def test_saturation_zero_and_gain():
    big = np.full((1, 16), 1e6)
    code, scale = O.quantise(big, [0])
    assert scale[0, 0] == 126 and (code == 7).all()                  # 448 * 6
    tiny = np.full((1, 16), 6 * 2.0 ** -11)                          # scale rounds to 0
    assert (O.quantise(tiny, [0])[0] == 0).all()
    code, scale = O.quantise(tiny, [-11])
    np.testing.assert_array_equal(O.values(code, scale, [-11]), tiny)


@pytest.mark.parametrize("d", [64, 128])
def test_cell_rows_do_not_touch_each_other(d):
    rng = np.random.default_rng(d)
    cell = np.zeros(18 * d, np.uint8)
    rows = []
    for r in range(16):
        rows.append((rng.integers(0, 16, d), rng.integers(0, 127, d // 16),
                     rng.integers(0, 16, d), rng.integers(0, 127, d // 16)))
        O.put_row(cell, r, *rows[-1])
    for r in range(16):
        for a, b in zip(O.get_row(cell, r), rows[r]):
            np.testing.assert_array_equal(a, b)


def test_reserve_worked_case():
    """Three sequences: one grows inside its page, one takes two pages, one does not fit."""
    table = np.array([[5, -1, -1], [-1, -1, -1], [7, -1, -1]])
    got = O.reserve([3, 0, 16], [4, 17, 20], table, np.array([9, 8, 6]), 3, 16, 50, 64, 48)
    assert got["start"].tolist() == [0, 4, 21, 41]
    assert got["table"].tolist() == [[5, -1, -1], [6, 8, -1], [7, -1, -1]]
    assert got["free_count"] == 1 and got["status"] == {"pool_empty"}
    assert got["new_len"].tolist() == [7, 17, 16]
    assert got["slot"][:4].tolist() == [83, 84, 85, 86]
    assert got["slot"][4:21].tolist() == list(range(96, 112)) + [128]
    assert (got["slot"][21:] == -1).all() and (got["pos"][21:] == -1).all()


def test_attention_is_a_brute_force_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(2, 4, 8)), rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 2, 8))
    out, _, _ = O.attention(q, k, v, [0, 3], 0.5)
    assert (out[0] == 0).all()
    w = np.exp([0.5 * sum(q[1, 3, i] * k[j, 1, i] for i in range(8)) for j in range(3)])
    np.testing.assert_allclose(out[1, 3], sum(w[j] * v[j, 1] for j in range(3)) / w.sum())


def test_rotation_keeps_norms_and_depends_on_distance():
    rng = np.random.default_rng(2)
    x, y = rng.normal(size=(1, 1, 64)), rng.normal(size=(1, 1, 64))
    r = lambda z, p: O.norm_rope(z, None, [p], 1e6, 0.0)[0, 0]  # noqa: E731
    np.testing.assert_allclose(np.linalg.norm(r(x, 12345)), np.linalg.norm(x))
    np.testing.assert_allclose(r(x, 105) @ r(y, 100), r(x, 9005) @ r(y, 9000), rtol=1e-9)
