"""GPU parity of the linear layers in 8-bit floating point against the float64 oracle.

Tolerances.  A code is the nearest to what the kernel rounds, so it is off by half a step
of e4m3 at that value, and by the error eps of the fp32 arithmetic before it, relative to the
value.  A product's fp32 sum over K is off by at most
    (2^-19 + 2^-23 K/128) S,   S = sum of |x| |w|:
32 products meet in one step of the tensor cores, aligned to the largest with at least 24 bits
(32 2^-24 = 2^-19 of it), and one rounded addition for each block; then 2^-8 of the value for the
rounding to bf16."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.gpu_helpers import Guarded

pytestmark = pytest.mark.gpu

BF, F8, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32


def _dfl():
    import block_diffusion_speculative_02_gb300 as dfl
    return dfl


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.float32))).to(BF).cuda()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def codes(t):
    return t.detach().view(torch.uint8).cpu().numpy()


def strided(rows, cols, pitch, fill=None):
    """A bf16 matrix whose rows lie pitch elements apart."""
    t = torch.zeros(max(rows, 1), pitch, dtype=BF, device="cuda")[:rows, :cols]
    if fill is not None:
        t.copy_(fill)
    return t


def check_codes(q, scale, h, eps):
    """q, scale of rows (or, given [N, K] scales spread already, of weights) against h."""
    q, scale = np.asarray(q), np.asarray(scale, np.float64)
    y = h / scale
    near = O.half_step(np.minimum(np.abs(y) * (1 + eps), 448.0))
    # past 448 only by rounding: the largest is a (1 + eps) / (a / 448)
    off = np.abs(O.decode(q) - y)
    assert (off <= near + (eps + 2.0 ** -22) * np.abs(y)).all(), float((off - near).max())


def check_scales(scale, a, eps):
    want = np.maximum(a, O.TINY) / 448
    assert (np.abs(scale - want) <= (eps + 2.0 ** -22) * want).all()


def make_rows(rng, m, k, outliers=True):
    x = rng.normal(size=(m, k))
    if outliers:
        x *= np.where(rng.random(k) < 0.02, 20.0, 1.0)
    return x


def random_x(rng, m, k):
    """8-bit rows as tensors and as float64 values."""
    q, s = O.round_rows(make_rows(rng, m, k))
    s = s.astype(np.float32)
    return (torch.from_numpy(q).cuda().view(F8), torch.from_numpy(s).cuda(), O.rows_value(q, s))


def random_w(rng, *shape):
    q, s = O.round_weight(0.02 * rng.normal(size=shape))
    s = s.astype(np.float32)
    return (torch.from_numpy(q).cuda().view(F8), torch.from_numpy(s).cuda(), O.weight_value(q, s))


def product_bound(x, w, ref):
    kb = O.blocks(x.shape[1])
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -19 + kb * 2.0 ** -23) * (np.abs(x) @ np.abs(w).T)


def check_product(got, x, w):
    ref = O.linear(x, w)
    off = np.abs(got - ref)
    bound = product_bound(x, w, ref)
    assert (off <= bound).all(), (int((off > bound).sum()), np.argwhere(off > bound)[:5])


# --------------------------------------------------------------------------------------------
# rows and weights to 8 bits
# --------------------------------------------------------------------------------------------
# eps of the norm: the sum of squares has at most 16 x 4 products a thread and 10 levels of
# a tree (74 2^-24, halved by the root), the root 2 units, four more roundings
NORM_EPS = 45 * 2.0 ** -24


@pytest.mark.parametrize("m,k", [(1, 16), (1, 128), (3, 144), (17, 512), (9, 528), (16, 4096),
                                 (5, 8192), (3, 8208), (2, 16400), (2, 32768), (300, 1008)])
@pytest.mark.parametrize("residual,norm", [(True, True), (False, True), (True, False),
                                           (False, False)])
def test_norm_rows(m, k, residual, norm):
    dfl = _dfl()
    rng = np.random.default_rng(m * 100003 + k)
    x, r = bf16(make_rows(rng, m, k)), bf16(make_rows(rng, m, k)) if residual else None
    w = bf16(1 + 0.1 * rng.normal(size=k)) if norm else None
    total = Guarded((m, k), BF)
    q, s = Guarded((m, k), F8), Guarded((O.blocks(k), m), torch.float32)
    dfl.dflash_fp8_norm_rows(x, r, w, 1e-6, total.t if residual else None, q.t, s.t)
    add, h = O.norm_rows(f64(x), None if r is None else f64(r), None if w is None else f64(w))
    eps = NORM_EPS if norm else 2.0 ** -23
    scale = s.t.cpu().numpy().astype(np.float64)
    check_scales(scale, O._maxima(np.abs(h), (1,)).T, eps)
    check_codes(codes(q.t), O.spread(scale.T, k, 1), h, eps)
    if residual:
        assert (np.abs(f64(total.t) - add) <= 2.0 ** -8 * np.abs(add) + 2.0 ** -24).all()
    for g in (total, q, s):
        g.check()


def test_norm_rows_strided_and_in_place():
    dfl = _dfl()
    rng = np.random.default_rng(5)
    m, k = 33, 640
    x, r = strided(m, k, 1288, bf16(make_rows(rng, m, k))), strided(m, k, 648)
    r.copy_(bf16(make_rows(rng, m, k)))
    w = bf16(1 + 0.1 * rng.normal(size=k))
    want_sum = strided(m, k, 704)
    q0, s0 = dfl.alloc_fp8_rows(m, k)
    dfl.dflash_fp8_norm_rows(x, r, w, 1e-6, want_sum, q0, s0)
    dense = torch.empty(m, k, dtype=BF, device="cuda")
    q1, s1 = dfl.alloc_fp8_rows(m, k)
    dfl.dflash_fp8_norm_rows(x.contiguous(), r.contiguous(), w, 1e-6, dense, q1, s1)
    assert torch.equal(dense, want_sum)
    for target in ("x", "residual"):
        xx, rr = x.clone(), r.clone()
        q2, s2 = dfl.alloc_fp8_rows(m, k)
        dfl.dflash_fp8_norm_rows(xx, rr, w, 1e-6, xx if target == "x" else rr, q2, s2)
        assert torch.equal(xx if target == "x" else rr, dense)
        for q, s in ((q1, s1), (q2, s2)):
            assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)


def test_rows_with_zeros_tiny_and_bad_values():
    """Blocks of zeros and of subnormal numbers are finite; an infinity or NaN marks its block."""
    dfl = _dfl()
    x = torch.ones(6, 384, dtype=BF, device="cuda")
    x[0] = 0
    x[1, :128] = 2.0 ** -130
    x[2, 200] = float("inf")
    x[3, 5] = float("nan")
    x[4, 300] = 3.0e38
    q, s = dfl.alloc_fp8_rows(6, 384)
    dfl.dflash_fp8_norm_rows(x, None, None, 0.0, None, q, s)
    v = O.rows_value(codes(q), s.cpu().numpy())
    assert (v[0] == 0).all() and (codes(q)[0] == 0).all() and (s[:, 0] > 0).all()
    assert np.isfinite(v[1]).all()
    assert np.abs(v[1, :128] - 2.0 ** -130).max() <= 2.0 ** -10 * 2.0 ** -117 / 448 + 2.0 ** -149
    bad = np.zeros((6, 3), bool)
    bad[2, 1] = bad[3, 0] = True
    assert np.array_equal(np.isnan(s.cpu().numpy().T), bad)
    assert np.array_equal(np.isnan(v).reshape(6, 3, 128).all(-1), bad)
    assert np.array_equal(np.isnan(v).reshape(6, 3, 128).any(-1), bad)
    assert np.isclose(v[4, 300], float(x[4, 300]), rtol=1e-6)


@pytest.mark.parametrize("m,f", [(1, 16), (1, 128), (2, 144), (16, 12288), (300, 272), (67, 1024)])
def test_silu_mul(m, f):
    dfl = _dfl()
    rng = np.random.default_rng(m + f)
    x = rng.normal(size=(m, 2 * f)) * 3
    x[:, 0] = -90.0                                   # the exponential is past the largest number
    gu = strided(m, 2 * f, 2 * f + 24, bf16(x))
    q, s = Guarded((m, f), F8), Guarded((O.blocks(f), m), torch.float32)
    dfl.dflash_fp8_silu_mul(gu, q.t, s.t)
    h = O.silu_mul(f64(gu))
    # __expf: 2 + 1.173 |g| units of 2^-23; the division 2, the product and the sum 1 each
    g = np.abs(f64(gu)[:, :f])
    eps = (6 + 1.2 * g) * 2.0 ** -23
    scale = s.t.cpu().numpy().astype(np.float64)
    check_scales(scale, O._maxima(np.abs(h), (1,)).T, eps[:, 1:].max() if f > 1 else eps.max())
    check_codes(codes(q.t), O.spread(scale.T, f, 1), np.where(g > 80, 0.0, h), eps)
    q.check()
    s.check()


def test_silu_mul_of_gates_near_the_end_of_the_exponential():
    """exp(-g) from 2^120 to past the largest number, alone in blocks with large u."""
    dfl = _dfl()
    g = np.repeat([-83.0, -86.5, -87.5, -88.0, -88.5, 88.0, 100.0, 3e38], 128)[None]
    x = np.concatenate([g, np.full_like(g, 2.0 ** 100)], axis=1)
    x[:, 128 * 14:] = 0.5                             # (h of the last two within fp32)
    gu = bf16(x)
    q, s = dfl.alloc_fp8_rows(1, 1024)
    dfl.dflash_fp8_silu_mul(gu, q, s)
    h = O.silu_mul(f64(gu))
    # the exponential: 2 + 1.173 |g| units of 2^-23; the division 2, two products and the sum 1 each
    g = np.minimum(np.abs(f64(gu)[:, :1024]), 104.0)
    eps = (7 + 1.2 * g) * 2.0 ** -23
    scale = s.cpu().numpy().astype(np.float64)
    check_scales(scale, O._maxima(np.abs(h), (1,)).T, eps.max())
    check_codes(codes(q), O.spread(scale.T, 1024, 1), h, eps)


@pytest.mark.parametrize("shape", [(1, 16), (128, 128), (129, 144), (1000, 272), (3, 130, 400)])
def test_weight(shape):
    dfl = _dfl()
    rng = np.random.default_rng(sum(shape))
    w = bf16(0.02 * rng.normal(size=shape))
    q, s = dfl.alloc_fp8_weight(*shape)
    gq = Guarded(q.shape, F8)
    dfl.dflash_fp8_weight(w, gq.t, s)
    h = f64(w)
    scale = s.cpu().numpy().astype(np.float64)
    ax = h.ndim - 2
    check_scales(scale, O._maxima(np.abs(h), (ax, ax + 1)), 0.0)
    check_codes(codes(gq.t), O.spread(O.spread(scale, shape[-2], ax), shape[-1], ax + 1), h, 0.0)
    gq.check()


# --------------------------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------------------------
SHAPES = [(1, 1, 16), (1, 128, 128), (1, 4096, 4096), (2, 130, 144), (7, 257, 400), (16, 512, 4096),
          (17, 384, 1024), (31, 129, 272), (33, 1000, 2048), (63, 640, 784), (64, 256, 12288),
          (65, 255, 512), (100, 1537, 640), (128, 128, 128), (129, 511, 2560), (255, 2567, 256),
          (256, 1024, 1024), (257, 768, 4000), (513, 520, 128), (1000, 136, 1040), (700, 2056, 16),
          (2048, 2048, 512), (128, 20000, 144), (2148, 2048, 256), (2200, 1500, 272),
          (1, 24576, 128), (24, 8192, 640), (50, 20000, 384), (2500, 387, 144), (200, 5003, 2064),
          (900, 2600, 144), (1500, 1537, 656), (1000, 2600, 1168), (4000, 1029, 656),
          (500, 387, 2064), (700, 1300, 4000), (300, 2051, 144), (150, 4096, 8192),
          (700, 5003, 4112), (600, 8200, 4096)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(m, n, k):
    dfl = _dfl()
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    x, xs, xv = random_x(rng, m, k)
    w, wscale, wv = random_w(rng, n, k)
    out, ws = Guarded((m, n), BF), dfl.alloc_fp8_workspace()
    dfl.dflash_fp8_linear(x, xs, w, wscale, out.t, ws)
    check_product(f64(out.t), xv, wv)
    out.check()
    assert dfl.dflash_read_status(ws) == 0 and not bool(ws.any())


# (of 387 features: streamed, and tiles of 128 x 128; of 1537 tiles of 128 x 256, and pairs)
@pytest.mark.parametrize("m,n,k", [(5, 387, 320), (40, 387, 320), (200, 387, 320), (600, 387, 320),
                                   (2500, 387, 144), (1500, 1537, 144), (1500, 1537, 656),
                                   (1500, 1537, 4112)])
@pytest.mark.parametrize("apart,offset", [(8, 0), (9, 0), (16, 3), (16, 8)])
def test_linear_into_strided_rows(m, n, k, apart, offset):
    """Rows of out that lie apart, also unaligned: nothing between them is touched."""
    dfl = _dfl()
    pitch = (n + 7) // 8 * 8 + apart
    rng = np.random.default_rng(m + pitch)
    x, xs, xv = random_x(rng, m, k)
    w, wscale, wv = random_w(rng, n, k)
    buf = torch.full((m * pitch + 64,), 7.0, dtype=BF, device="cuda")
    out = buf[offset:offset + m * pitch].view(m, pitch)[:, :n]
    dfl.dflash_fp8_linear(x, xs, w, wscale, out, dfl.alloc_fp8_workspace())
    check_product(f64(out), xv, wv)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[offset:offset + m * pitch].view(m, pitch)[:, :n] = False
    assert bool((buf[keep] == 7).all())


@pytest.mark.parametrize("m", [3, 60, 300])
def test_linear_bad_values_stay_in_their_rows(m):
    dfl = _dfl()
    rng = np.random.default_rng(m)
    n, k = 300, 512
    x, xs, xv = random_x(rng, m, k)
    w, wscale, wv = random_w(rng, n, k)
    out, ws = torch.empty(m, n, dtype=BF, device="cuda"), dfl.alloc_fp8_workspace()
    xs[2, 1] = float("nan")
    w.view(torch.uint8)[7, 100] = 0x7F
    dfl.dflash_fp8_linear(x, xs, w, wscale, out, ws)
    got = f64(out)
    nan = np.zeros((m, n), bool)
    nan[1], nan[:, 7] = True, True
    assert np.array_equal(np.isnan(got), nan)
    keep_r, keep_c = [i for i in range(m) if i != 1], [j for j in range(n) if j != 7]
    check_product(got[np.ix_(keep_r, keep_c)], xv[keep_r], wv[keep_c])


@pytest.mark.parametrize("m", [1, 16, 50, 256, 1024])
def test_linear_gives_the_same_bits_again(m):
    dfl = _dfl()
    rng = np.random.default_rng(m)
    x, xs, _ = random_x(rng, m, 4096)
    w, wscale, _ = random_w(rng, 1024, 4096)
    ws = dfl.alloc_fp8_workspace()
    first = torch.empty(m, 1024, dtype=BF, device="cuda")
    dfl.dflash_fp8_linear(x, xs, w, wscale, first, ws)
    for _ in range(5):
        again = torch.empty_like(first)
        dfl.dflash_fp8_linear(x, xs, w, wscale, again, ws)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))


# --------------------------------------------------------------------------------------------
# products by expert
# --------------------------------------------------------------------------------------------
def counts_of(kind, e, m, rng):
    if kind == "even":
        return [m // e + (i < m % e) for i in range(e)]
    if kind == "one":
        return [m if i == e // 2 else 0 for i in range(e)]
    share = rng.random(e) ** 3
    return rng.multinomial(m, share / share.sum()).tolist()


GROUPED = [("even", 4, 4, 130, 144), ("skew", 128, 128, 256, 512), ("skew", 128, 900, 200, 256),
           ("one", 7, 90, 300, 640), ("skew", 9, 1500, 520, 384), ("even", 3, 700, 513, 1040),
           ("one", 1, 50, 128, 128), ("skew", 1024, 700, 16, 128), ("skew", 33, 300, 129, 2048),
           ("even", 64, 4096, 128, 256), ("even", 2, 3000, 2000, 256),
           ("even", 2, 1300, 2816, 144), ("even", 2, 1300, 300, 400), ("skew", 40, 800, 5000, 144),
           ("skew", 3, 200, 1200, 2304), ("skew", 5, 2800, 4096, 16), ("one", 1000, 1500, 512, 272),
           ("even", 2, 1300, 2816, 656), ("skew", 16, 2900, 1500, 1040),
           ("even", 4, 330, 1536, 2048),
           ("skew", 64, 12000, 400, 656), ("even", 6, 2600, 900, 1040), ("skew", 8, 560, 2050, 784),
           ("skew", 4, 8000, 1050, 656), ("skew", 300, 20000, 140, 144),
           ("skew", 1024, 40000, 300, 144), ("skew", 1024, 120000, 140, 272),
           ("skew", 5, 2900, 1030, 4112)]


@pytest.mark.parametrize("kind,e,m,n,k", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(kind, e, m, n, k, gather):
    dfl = _dfl()
    rng = np.random.default_rng(e * 31 + m)
    before, behind = 3, 5
    counts = counts_of(kind, e, m, rng)
    start = np.cumsum([before] + counts)
    total = before + m + behind
    n_src = 37 if gather else total
    x, xs, xv = random_x(rng, n_src, k)
    w, wscale, wv = random_w(rng, e, n, k)
    rows = rng.integers(0, n_src, total) if gather else np.arange(total)
    out, ws = Guarded((total, n), BF, fill=3.0), dfl.alloc_fp8_workspace()
    dfl.dflash_fp8_grouped(x, xs, w, wscale, i32(start), i32(rows) if gather else None, out.t, ws)
    got = f64(out.t)
    for g in range(e):
        a, b = start[g], start[g + 1]
        if b > a:
            check_product(got[a:b], xv[rows[a:b]], wv[g])
    assert (got[:before] == 3).all() and (got[before + m:] == 3).all()
    out.check()
    assert dfl.dflash_read_status(ws) == 0


@pytest.mark.parametrize("m", [40, 700])
def test_grouped_bad_groups_and_rows(m):
    """What the host cannot see: starts out of order or out of range, rows outside x."""
    dfl = _dfl()
    rng = np.random.default_rng(m)
    n, k, bits = 200, 256, dfl.dflash.STATUS_BITS["capacity"]
    x, xs, xv = random_x(rng, 20, k)
    w, wscale, wv = random_w(rng, 4, n, k)
    ws = dfl.alloc_fp8_workspace()
    rows = rng.integers(0, 20, m)
    bad = rows.copy()
    bad[[3, m - 1]] = 20, -1
    for start, rws in (([0, 10, 5, 20, m], rows), ([0, 10, 20, m + 1, m + 9], rows),
                       ([-4, 10, 20, 30, m], rows), ([0, 10, 20, 30, m], bad),
                       ([2 ** 31 - 1, -2 ** 31, 5, 9, 30], rows)):
        out = torch.full((m, n), 3.0, dtype=BF, device="cuda")
        dfl.dflash_fp8_grouped(x, xs, w, wscale, i32(start), i32(rws), out, ws)
        assert dfl.dflash_read_status(ws) == bits
        got, seen = f64(out), np.zeros(m, bool)
        for e in range(4):
            a, b = start[e], start[e + 1]
            if not 0 <= a <= b <= m or seen[a:b].any():
                continue
            ok = (rws[a:b] >= 0) & (rws[a:b] < 20)
            vals = np.where(ok[:, None], xv[np.where(ok, rws[a:b], 0)], 0.0)
            overlap = any(0 <= start[f] <= start[f + 1] <= m and start[f] < b and start[f + 1] > a
                          for f in range(4) if f != e)
            if not overlap:
                check_product(got[a:b], vals, wv[e])
                assert (got[a:b][~ok] == 0).all()
            seen[a:b] = True
        covered = np.zeros(m, bool)
        for e in range(4):
            if 0 <= start[e] <= start[e + 1] <= m:
                covered[start[e]:start[e + 1]] = True
        assert (got[~covered] == 3).all()
    assert dfl.dflash_read_status(ws) == 0


@pytest.mark.parametrize("e,m,n,k", [(64, 384, 300, 2048), (6, 500, 260, 256), (4, 2600, 260, 256)])
def test_grouped_rows_have_one_owner(e, m, n, k):
    """Experts that claim rows of one before them are left out."""
    dfl = _dfl()
    rng = np.random.default_rng(e)
    x, xs, xv = random_x(rng, m, k)
    w, wscale, wv = random_w(rng, e, n, k)
    last = m - m // 4
    start = [0] + [last, 0] * (e // 2 - 1) + [m - 40, m]       # the last of 40 rows does not
    out, ws = Guarded((m, n), BF, fill=3.0), dfl.alloc_fp8_workspace()
    dfl.dflash_fp8_grouped(x, xs, w, wscale, i32(start), None, out.t, ws)
    assert dfl.dflash_read_status(ws) == dfl.dflash.STATUS_BITS["capacity"]
    got = f64(out.t)
    check_product(got[:last], xv[:last], wv[0])
    assert (got[last:m - 40] == 3).all()
    check_product(got[m - 40:], xv[m - 40:], wv[-1])
    out.check()


def test_grouped_equals_linear():
    """One expert with all rows: the same bits as the plain product."""
    dfl = _dfl()
    rng = np.random.default_rng(11)
    for m in (1, 16, 64, 300):
        x, xs, _ = random_x(rng, m, 1024)
        w, wscale, _ = random_w(rng, 640, 1024)
        ws = dfl.alloc_fp8_workspace()
        a, b = (torch.empty(m, 640, dtype=BF, device="cuda") for _ in range(2))
        dfl.dflash_fp8_linear(x, xs, w, wscale, a, ws)
        dfl.dflash_fp8_grouped(x, xs, w[None], wscale[None], i32([0, m]), None, b, ws)
        assert torch.equal(a, b)


# --------------------------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------------------------
def test_empty_calls_launch_nothing():
    dfl = _dfl()
    ws = dfl.alloc_fp8_workspace()
    x = torch.empty(0, 256, dtype=BF, device="cuda")
    q, s = dfl.alloc_fp8_rows(0, 256)
    dfl.dflash_fp8_norm_rows(x, None, None, 1e-6, None, q, s)
    dfl.dflash_fp8_silu_mul(torch.empty(0, 512, dtype=BF, device="cuda"), q, s)
    w, wscale = dfl.alloc_fp8_weight(2, 64, 256)
    out = torch.empty(0, 64, dtype=BF, device="cuda")
    dfl.dflash_fp8_linear(q, s, w[0], wscale[0], out, ws)
    dfl.dflash_fp8_grouped(q, s, w, wscale, i32([0, 0, 0]), None, out, ws)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0


def mlp(dfl, x, residual, norm_w, w1, w2, ws, buf):
    """One MLP of a target in 8 bits: norm, gate and up, activation, down."""
    dfl.dflash_fp8_norm_rows(x, residual, norm_w, 1e-6, buf["sum"], buf["q"], buf["s"])
    dfl.dflash_fp8_linear(buf["q"], buf["s"], *w1, buf["gu"], ws)
    dfl.dflash_fp8_silu_mul(buf["gu"], buf["qa"], buf["sa"])
    dfl.dflash_fp8_linear(buf["qa"], buf["sa"], *w2, buf["y"], ws)


def mlp_buffers(dfl, m, h, f):
    (q, s), (qa, sa) = dfl.alloc_fp8_rows(m, h), dfl.alloc_fp8_rows(m, f)
    new = lambda n: torch.empty(m, n, dtype=BF, device="cuda")  # noqa: E731
    return dict(q=q, s=s, qa=qa, sa=sa, sum=new(h), gu=new(2 * f), y=new(h))


@pytest.mark.parametrize("m", [1, 16, 130, 600])
def test_mlp_in_8_bits(m):
    """The calls one after the other, each against the oracle on what the one before left, and
    the whole against the bf16 weights: three roundings of operands to 8 bits (2^-4 each) on
    sums of independent terms."""
    dfl = _dfl()
    rng = np.random.default_rng(m)
    h, f = 512, 1408
    w1, w2 = bf16(0.05 * rng.normal(size=(2 * f, h))), bf16(0.05 * rng.normal(size=(h, f)))
    q1, q2 = dfl.alloc_fp8_weight(2 * f, h), dfl.alloc_fp8_weight(h, f)
    dfl.dflash_fp8_weight(w1, *q1)
    dfl.dflash_fp8_weight(w2, *q2)
    x, r = bf16(rng.normal(size=(m, h))), bf16(rng.normal(size=(m, h)))
    g = bf16(1 + 0.1 * rng.normal(size=h))
    ws, buf = dfl.alloc_fp8_workspace(), mlp_buffers(dfl, m, h, f)
    mlp(dfl, x, r, g, q1, q2, ws, buf)
    v = lambda q, s: O.rows_value(codes(q), s.cpu().numpy())  # noqa: E731
    wv = lambda t: O.weight_value(codes(t[0]), t[1].cpu().numpy())  # noqa: E731
    check_product(f64(buf["gu"]), v(buf["q"], buf["s"]), wv(q1))
    check_product(f64(buf["y"]), v(buf["qa"], buf["sa"]), wv(q2))
    _, hn = O.norm_rows(f64(x), f64(r), f64(g))
    ref = O.silu_mul(hn @ f64(w1).T) @ f64(w2).T
    assert np.linalg.norm(f64(buf["y"]) - ref) <= 3 * 2.0 ** -4 * np.linalg.norm(ref)
    assert dfl.dflash_read_status(ws) == 0


def test_mlp_captured_and_replayed_with_other_inputs():
    dfl = _dfl()
    rng = np.random.default_rng(3)
    m, h, f = 48, 256, 384
    q1, q2 = random_w(rng, 2 * f, h)[:2], random_w(rng, h, f)[:2]
    x, r, g = bf16(rng.normal(size=(m, h))), bf16(rng.normal(size=(m, h))), bf16(np.ones(h))
    ws, buf = dfl.alloc_fp8_workspace(), mlp_buffers(dfl, m, h, f)
    mlp(dfl, x, r, g, q1, q2, ws, buf)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mlp(dfl, x, r, g, q1, q2, ws, buf)
    for _ in range(3):
        x.copy_(bf16(rng.normal(size=(m, h))))
        graph.replay()
        other = mlp_buffers(dfl, m, h, f)
        mlp(dfl, x, r, g, q1, q2, ws, other)
        torch.cuda.synchronize()
        for name in buf:
            assert torch.equal(buf[name].view(torch.uint8), other[name].view(torch.uint8)), name
    assert dfl.dflash_read_status(ws) == 0


@pytest.mark.parametrize("m", [48, 400, 2600])
def test_grouped_captured_and_replayed_with_other_experts(m):
    """start and rows change between replays; rows of the padding name no row of x."""
    dfl = _dfl()
    rng = np.random.default_rng(m)
    e, n, k, pad = 6, 300, 400, 9
    x, xs, xv = random_x(rng, 50, k)
    w, wscale, wv = random_w(rng, e, n, k)
    start, rows = torch.zeros(e + 1, dtype=torch.int32, device="cuda"), i32(np.full(m + pad, -1))
    out, ws = torch.zeros(m + pad, n, dtype=BF, device="cuda"), dfl.alloc_fp8_workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dfl.dflash_fp8_grouped(x, xs, w, wscale, start, rows, out, ws)
    for kind in ("even", "one", "skew", "none"):
        counts = [0] * e if kind == "none" else counts_of(kind, e, m, rng)
        edge, index = np.cumsum([0] + counts), rng.integers(0, 50, m + pad)
        index[edge[-1]:] = -1
        start.copy_(i32(edge))
        rows.copy_(i32(index))
        out.fill_(3)
        graph.replay()
        got = f64(out)
        for g in range(e):
            check_product(got[edge[g]:edge[g + 1]], xv[index[edge[g]:edge[g + 1]]], wv[g])
        assert (got[edge[-1]:] == 3).all()
    assert dfl.dflash_read_status(ws) == 0


def test_two_streams_share_a_workspace():
    """Products on two streams at once, with one workspace (it is only their status)."""
    dfl = _dfl()
    rng = np.random.default_rng(4)
    ws = dfl.alloc_fp8_workspace()
    jobs = []
    for m in (16, 700):
        x, xs, xv = random_x(rng, m, 2048)
        w, wscale, wv = random_w(rng, 1000, 2048)
        jobs.append((x, xs, w, wscale, torch.empty(m, 1000, dtype=BF, device="cuda"), xv, wv))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (x, xs, w, wscale, out, _, _) in zip(streams, jobs):
            dfl.dflash_fp8_linear(x, xs, w, wscale, out, ws, stream=st)
    torch.cuda.synchronize()
    for _, _, _, _, out, xv, wv in jobs:
        check_product(f64(out), xv, wv)
    assert dfl.dflash_read_status(ws) == 0


@pytest.mark.parametrize("tokens", [1, 16, 200])
def test_experts_of_a_layer(tokens):
    """A layer with experts: rows in 8 bits once, each token through two of them, and back."""
    dfl = _dfl()
    rng = np.random.default_rng(tokens)
    e, top, h, f = 8, 2, 256, 192
    x = bf16(rng.normal(size=(tokens, h)))
    g = bf16(np.ones(h))
    w1, w2 = random_w(rng, e, 2 * f, h), random_w(rng, e, h, f)
    pick = torch.from_numpy(np.stack([rng.permutation(e)[:top] for _ in range(tokens)])).cuda()
    order = pick.flatten().argsort(stable=True)
    rows = (order // top).int()
    start = torch.zeros(e + 1, dtype=I32, device="cuda")
    start[1:] = torch.bincount(pick.flatten(), minlength=e).cumsum(0)
    m = tokens * top
    q, s = dfl.alloc_fp8_rows(tokens, h)
    qa, sa = dfl.alloc_fp8_rows(m, f)
    gu, y = (torch.empty(m, n, dtype=BF, device="cuda") for n in (2 * f, h))
    ws = dfl.alloc_fp8_workspace()
    dfl.dflash_fp8_norm_rows(x, None, g, 1e-6, None, q, s)
    dfl.dflash_fp8_grouped(q, s, w1[0], w1[1], start, rows, gu, ws)
    dfl.dflash_fp8_silu_mul(gu, qa, sa)
    dfl.dflash_fp8_grouped(qa, sa, w2[0], w2[1], start, None, y, ws)
    out = torch.zeros(tokens, h, device="cuda").index_add_(0, rows.long(), y.float())
    assert dfl.dflash_read_status(ws) == 0
    _, hn = O.norm_rows(f64(x), None, f64(g))
    ref = np.zeros((tokens, h))
    for t in range(tokens):
        for k in pick[t].tolist():
            ref[t] += w2[2][k] @ O.silu_mul((w1[2][k] @ hn[t])[None])[0]
    assert np.linalg.norm(f64(out) - ref) <= 2 * 2.0 ** -4 * np.linalg.norm(ref)


def test_large_offsets():
    """Elements of out and of the scales' array past 2^31 bytes and elements."""
    dfl = _dfl()
    m, n, k = 70000, 32768, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, k, generator=g, device="cuda").to(BF)
    q, s = dfl.alloc_fp8_rows(m, k)
    dfl.dflash_fp8_norm_rows(x, None, None, 0.0, None, q, s)
    w, wscale = dfl.alloc_fp8_weight(n, k)
    dfl.dflash_fp8_weight(torch.randn(n, k, generator=g, device="cuda").to(BF), w, wscale)
    out = torch.zeros(m, n, dtype=BF, device="cuda")
    dfl.dflash_fp8_linear(q, s, w, wscale, out, dfl.alloc_fp8_workspace())
    for lo in (0, 65500, m - 40):
        xv = O.rows_value(codes(q[lo:lo + 40]), s[:, lo:lo + 40].cpu().numpy())
        wv = O.weight_value(codes(w), wscale.cpu().numpy())
        check_product(f64(out[lo:lo + 40]), xv, wv)
    assert bool((out.abs().amax(1) > 0).all())


@pytest.mark.parametrize("m", [24, 3000])
def test_weights_past_2_to_the_32_bytes(m):
    dfl = _dfl()
    e, n, k = 36, 15000, 8192                          # 4.4 GB
    g = torch.Generator(device="cuda").manual_seed(2)
    w, wscale = dfl.alloc_fp8_weight(e, n, k)
    for i in range(e):
        part = torch.randn(n, k, generator=g, device="cuda").to(BF)
        dfl.dflash_fp8_weight(part, w[i], wscale[i])
    whole, whole_scale = dfl.alloc_fp8_weight(e, n, k)
    big = torch.zeros(e, n, k, dtype=BF, device="cuda")
    big[-1] = part
    dfl.dflash_fp8_weight(big, whole, whole_scale)     # the last past 2^32 of codes and of bf16
    assert torch.equal(whole[-1].view(torch.uint8), w[-1].view(torch.uint8))
    assert torch.equal(whole_scale[-1], wscale[-1])
    del big, whole
    rng = np.random.default_rng(m)
    x, xs, xv = random_x(rng, m, k)
    out, ws = torch.zeros(m, n, dtype=BF, device="cuda"), dfl.alloc_fp8_workspace()
    start = [0, m // 2] + [m // 2] * (e - 2) + [m]
    dfl.dflash_fp8_grouped(x, xs, w, wscale, i32(start), None, out, ws)
    for at, expert in ((0, 0), (m // 2, e - 1)):
        for col in (0, n - 100):
            wv = O.weight_value(codes(w[expert]), wscale[expert].cpu().numpy())[col:col + 100]
            check_product(f64(out[at:at + 12, col:col + 100]), xv[at:at + 12], wv)
    assert dfl.dflash_read_status(ws) == 0


@pytest.mark.parametrize("n", [300, 1400, 2300])
def test_more_rows_than_a_band(n):
    """Row tiles past a band of 64, with feature tiles that fill no chunk of four."""
    dfl = _dfl()
    rng = np.random.default_rng(n)
    m, k = 17111, 144
    x, xs, xv = random_x(rng, m, k)
    w, wscale, wv = random_w(rng, 2, n, k)
    out, ws = Guarded((m, n), BF), dfl.alloc_fp8_workspace()
    dfl.dflash_fp8_linear(x, xs, w[0], wscale[0], out.t, ws)
    check_product(f64(out.t), xv, wv[0])
    rows = rng.permutation(m)
    for index in (None, rows):
        dfl.dflash_fp8_grouped(x, xs, w, wscale, i32([0, 200, m]),
                               None if index is None else i32(index), out.t, ws)
        got, vals = f64(out.t), xv if index is None else xv[index]
        check_product(got[:200], vals[:200], wv[0])
        check_product(got[200:], vals[200:], wv[1])
    out.check()
    assert dfl.dflash_read_status(ws) == 0


# --------------------------------------------------------------------------------------------
# refusals of the binding
# --------------------------------------------------------------------------------------------
def test_binding_refuses_and_touches_nothing():
    dfl = _dfl()
    m, n, k, e = 8, 96, 256, 3
    x = torch.zeros(m, k, dtype=BF, device="cuda")
    q, s = dfl.alloc_fp8_rows(m, k)
    w, wscale = dfl.alloc_fp8_weight(e, n, k)
    out, ws = torch.full((m, n), 3.0, dtype=BF, device="cuda"), dfl.alloc_fp8_workspace()
    start = i32([0, 2, 2, m])
    linear = lambda **c: dfl.dflash_fp8_linear(*{**dict(  # noqa: E731
        x=q, x_scale=s, w=w[0], w_scale=wscale[0], out=out, ws=ws), **c}.values())
    grouped = lambda **c: dfl.dflash_fp8_grouped(*{**dict(  # noqa: E731
        x=q, x_scale=s, w=w, w_scale=wscale, start=start, rows=None, out=out, ws=ws), **c}.values())
    norm = lambda **c: dfl.dflash_fp8_norm_rows(*{**dict(  # noqa: E731
        x=x, residual=None, norm_w=None, rms_eps=1e-6, sum_out=None, q=q, scale=s), **c}.values())
    for f, bad in ((linear, dict(x=x)), (linear, dict(x=q.t())), (linear, dict(x_scale=s.t())),
                   (linear, dict(w=w)), (linear, dict(w_scale=wscale)), (linear, dict(out=out.t())),
                   (linear, dict(out=out.float())), (linear, dict(ws=ws.int())),
                   (linear, dict(w=w[0, :, :128])), (linear, dict(x=q.cpu())),
                   (linear, dict(x=None)), (linear, dict(out=out[:, :95])),
                   (grouped, dict(start=start.long())), (grouped, dict(start=start[:3])),
                   (grouped, dict(rows=start)), (grouped, dict(out=out[:4])),
                   (grouped, dict(w=w[0])), (grouped, dict(out=None)),
                   (norm, dict(x=x[:, ::2])), (norm, dict(residual=x[:4])),
                   (norm, dict(norm_w=x[0, :128])), (norm, dict(q=x)), (norm, dict(scale=s[:1])),
                   (norm, dict(x=x.cpu())), (norm, dict(sum_out=x.float()))):
        with pytest.raises(ValueError):
            f(**bad)
    for f, bad in ((linear, dict(ws=ws[:32])), (norm, dict(rms_eps=-1.0))):
        with pytest.raises(dfl.DFlashError):
            f(**bad)
    odd = torch.zeros(4, 200, dtype=BF, device="cuda")               # 200 is no multiple of 16
    with pytest.raises(dfl.DFlashError):
        dfl.dflash_fp8_norm_rows(odd, None, None, 0.0, None, *dfl.alloc_fp8_rows(4, 200))
    with pytest.raises(dfl.DFlashError):                             # a pitch of no multiple of 8
        dfl.dflash_fp8_norm_rows(torch.zeros(4, 250, dtype=BF, device="cuda")[:, :240], None, None,
                                 0.0, None, *dfl.alloc_fp8_rows(4, 240))
    with pytest.raises(ValueError):
        dfl.dflash_fp8_silu_mul(torch.zeros(4, 33, dtype=BF, device="cuda"), q, s)
    torch.cuda.synchronize()
    assert bool((out == 3).all()) and dfl.dflash_read_status(ws) == 0


@pytest.mark.parametrize("m", [16, 300])
def test_first_use_inside_a_capture(m):
    """A graph that holds the calls alone, replayed on a stream of its own."""
    dfl = _dfl()
    rng = np.random.default_rng(m)
    x, xs, xv = random_x(rng, m, 512)
    w, wscale, wv = random_w(rng, 640, 512)
    out, ws = torch.zeros(m, 640, dtype=BF, device="cuda"), dfl.alloc_fp8_workspace()
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        dfl.dflash_fp8_linear(x, xs, w, wscale, out, ws)
        dfl.dflash_fp8_linear(x, xs, w, wscale, out, ws)
    with torch.cuda.stream(stream):
        graph.replay()
    stream.synchronize()
    check_product(f64(out), xv, wv)


FIRST_USE = """
import sys, torch
import block_diffusion_speculative_02_gb300 as dfl
m, n, k, index = map(int, sys.argv[1:])
x, xs = dfl.alloc_fp8_rows(m, k)
w, ws = dfl.alloc_fp8_weight(1, n, k)
x.copy_(torch.eye(m, k))
xs.fill_(1)
ws.fill_(1)
w.copy_((torch.arange(n * k) % 17).view(1, n, k).float())
out, space = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda"), dfl.alloc_fp8_workspace()
start = torch.tensor([0, m], dtype=torch.int32, device="cuda")
rows = torch.arange(m, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    if index:
        dfl.dflash_fp8_grouped(x, xs, w, ws, start, rows, out, space)
    else:
        dfl.dflash_fp8_linear(x, xs, w[0], ws[0], out, space)
graph.replay()
torch.cuda.synchronize()
assert dfl.dflash_read_status(space) == 0
assert torch.equal(out[:k].float(), w[0].float().T[:m]) and not bool(out[k:].any())
"""


@pytest.mark.parametrize("m,n,k,index", [(2500, 387, 144, 0), (1500, 1537, 144, 0),
                                         (1500, 1537, 656, 0), (2500, 387, 144, 1),
                                         (40, 4096, 1024, 1)])
def test_first_use_of_a_process_inside_a_capture(m, n, k, index):
    """Each kernel of the products for the first time, while a graph is captured."""
    done = subprocess.run([sys.executable, "-c", FIRST_USE, str(m), str(n), str(k), str(index)],
                          capture_output=True, text=True, timeout=120,
                          cwd=Path(__file__).resolve().parents[1])
    assert done.returncode == 0, done.stderr[-2000:]


def test_rows_of_x_given_many_times():
    """One row of x for every row of out, and each expert with its own number of them."""
    dfl = _dfl()
    rng = np.random.default_rng(8)
    for m in (64, 2000):
        x, xs, xv = random_x(rng, 3, 384)
        w, wscale, wv = random_w(rng, 2, 260, 384)
        out = torch.zeros(m, 260, dtype=BF, device="cuda")
        dfl.dflash_fp8_grouped(x, xs, w, wscale, i32([0, m // 3, m]), i32(np.full(m, 2)), out,
                               dfl.alloc_fp8_workspace())
        got = f64(out)
        assert (got[:m // 3] == got[0]).all() and (got[m // 3:] == got[-1]).all()
        check_product(got[:1], xv[2:], wv[0])
        check_product(got[-1:], xv[2:], wv[1])


def test_neighbours_of_a_small_row_range_stay():
    """x of fewer rows than a tile, inside a larger array whose other rows hold NaN."""
    dfl = _dfl()
    rng = np.random.default_rng(9)
    for m in (1, 5, 33, 70, 100):
        x, xs, xv = random_x(rng, m, 256)
        big = torch.full((m + 300, 256), 0x7F, dtype=torch.uint8, device="cuda")
        big[:m] = x.view(torch.uint8)
        w, wscale, wv = random_w(rng, 1300, 256)
        out = torch.zeros(m, 1300, dtype=BF, device="cuda")
        dfl.dflash_fp8_linear(big.view(F8)[:m], xs, w, wscale, out, dfl.alloc_fp8_workspace())
        check_product(f64(out), xv, wv)
