"""Norms of rows whose squares leave the range of fp32, against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.gpu_helpers import Guarded
from tests.test_gpu_fp8 import BF, F8, NORM_EPS, bf16, check_codes, check_scales, codes, f64

pytestmark = pytest.mark.gpu

# Rows are multiplied by a power of two first, which is exact; eps times its square is rounded
# twice, and halved by the root like the sum.
RANGE_EPS = NORM_EPS + 2 * 2.0 ** -24


def norm(x, r, w, eps):
    """Codes, scales and sums of the call, checked against the oracle where that is finite."""
    import block_diffusion_speculative_02_gb300 as dfl
    m, k = x.shape
    q, s, total = Guarded((m, k), F8), Guarded((O.blocks(k), m), torch.float32), Guarded((m, k), BF)
    dfl.dflash_fp8_norm_rows(x, r, w, eps, total.t, q.t, s.t)
    add, h = O.norm_rows(f64(x), None if r is None else f64(r), f64(w), float(np.float32(eps)))
    scale = s.t.cpu().numpy().astype(np.float64)
    check_scales(scale, O._maxima(np.abs(h), (1,)).T, RANGE_EPS)
    check_codes(codes(q.t), O.spread(scale.T, k, 1), h, RANGE_EPS)
    assert (np.abs(f64(total.t) - add) <= 2.0 ** -8 * np.abs(add) + 2.0 ** -133).all()
    for g in (q, s, total):
        g.check()
    return h


# a row to a warp, to a CTA in one, two and four pieces a thread
@pytest.mark.parametrize("k", [16, 144, 512, 4096, 16384, 32768])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_whose_squares_overflow(k, residual):
    rng = np.random.default_rng(k)
    top = [1e18, 3e19, 1e25, 1e30, 1e38, 3.3e38]
    x = rng.normal(size=(2 * len(top), k))
    for i, t in enumerate(top):
        x[2 * i, rng.integers(k)] = -t                    # one large element
        x[2 * i + 1] *= t / 8                             # a row of them (4.1 sigma at the end)
    x = np.clip(x, -3.3e38, 3.3e38)
    r = bf16(np.roll(x, 1, axis=1) * 0.01) if residual else None
    h = norm(bf16(x), r, bf16(1 + 0.1 * rng.normal(size=k)), 1e-6)
    assert (np.abs(h).max(1) > 0.4).all()                 # (no row of zeros is expected)


@pytest.mark.parametrize("k", [16, 144, 4096, 32768])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-36, 1e-31])
def test_rows_whose_squares_underflow(k, eps):
    rng = np.random.default_rng(k)
    x = rng.normal(size=(9, k)) * np.ldexp(1.0, [-126, -110, -80, -63, -60, -52, -48, -40, 0])[:, None]
    x[0, 0] = 2.0 ** -133                                 # (bf16's smallest)
    norm(bf16(x), None, bf16(1 + 0.1 * rng.normal(size=k)), eps)


@pytest.mark.parametrize("k", [144, 4096])
def test_rows_of_zeros_and_bad_values_stay_what_they_were(k):
    """Zeros over eps are zeros, over nothing NaN; an infinity marks its own block, the finite rest
    of its row is zero; a NaN marks the row."""
    import block_diffusion_speculative_02_gb300 as dfl
    x = torch.full((5, k), 1e30, dtype=BF, device="cuda")
    x[0] = 0
    x[1, 3], x[2, 3] = float("inf"), float("nan")
    x[3, 3] = x[4, 3] = 3.0e38
    r = torch.zeros_like(x)
    r[3, 3] = 3.0e38                                      # the sum is an infinity
    w = torch.ones(k, dtype=BF, device="cuda")
    for eps in (1e-6, 0.0):
        q, s = dfl.alloc_fp8_rows(5, k)
        dfl.dflash_fp8_norm_rows(x, r, w, eps, None, q, s)
        v = O.rows_value(codes(q), s.cpu().numpy())
        assert np.isnan(v[0]).all() if eps == 0 else (v[0] == 0).all()
        for i in (1, 3):
            assert np.isnan(v[i, :128]).all() and (v[i, 128:] == 0).all()
        assert np.isnan(v[2]).all() and np.isfinite(v[4]).all()
        assert np.isclose(v[4, 3], np.sqrt(k), rtol=2.0 ** -4)
