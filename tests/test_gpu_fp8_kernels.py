"""Every kernel of the 8-bit products on what the host cannot see: starts out of order, rows outside
x, bad values, replays with other experts.  Each case says which kernel it is for, and fails if
the sizes go to another one."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.gpu_helpers import Guarded
from tests.test_gpu_fp8 import BF, check_product, counts_of, f64, i32, random_w, random_x

pytestmark = pytest.mark.gpu

# (tile rows, features, shares of K), e, m, n, k, by index
TILES = [((128, 256, 1), 4, 2600, 2816, 144, True), ((128, 256, 1), 8, 6000, 1500, 656, True),
         ((128, 256, 1), 4, 6000, 1500, 400, False), ((128, 128, 1), 4, 2600, 700, 400, False),
         ((256, 256, 1), 4, 2600, 2816, 656, False), ((256, 256, 1), 8, 6000, 1000, 1040, False)]
STREAMS = [((16, 128, 8), 4, 8, 512, 2048, True), ((16, 128, 8), 4, 12, 130, 1024, False),
           ((16, 128, 4), 8, 64, 130, 2320, True), ((16, 128, 2), 32, 20, 130, 2048, False),
           ((16, 128, 2), 16, 20, 260, 2048, True), ((32, 128, 8), 4, 64, 260, 2320, True),
           ((32, 128, 4), 4, 260, 260, 2320, False), ((32, 128, 2), 16, 130, 130, 2048, True),
           ((32, 128, 8), 4, 40, 130, 2048, False), ((64, 128, 2), 8, 200, 512, 2048, True),
           ((64, 128, 4), 4, 700, 130, 2320, True), ((64, 128, 4), 8, 260, 130, 4096, False),
           ((64, 128, 8), 4, 300, 130, 4096, True)]
WHOLE = [((16, 128, 1), 8, 64, 512, 400, True), ((16, 128, 1), 8, 60, 512, 400, False),
         ((32, 128, 1), 4, 120, 700, 400, True), ((32, 128, 1), 8, 300, 1000, 1024, False),
         ((64, 128, 1), 8, 6000, 130, 400, True), ((64, 128, 1), 16, 260, 1500, 2048, False)]


def goes_to(plan, e, m, n, k, index):
    import block_diffusion_speculative_02_gb300 as dfl
    assert dfl.dflash_fp8_plan(m, n, k, e, index) == plan
    return dfl


def owners(start, m):
    """The expert that each row of out belongs to, or -1, and whether an expert was left out."""
    own, end, bad = np.full(m, -1), 0, False
    for e in range(len(start) - 1):
        a, b = int(start[e]), int(start[e + 1])
        if not 0 <= a <= b <= m:
            bad = True
        elif a < b:
            if a < end:
                bad = True
            else:
                own[a:b], end = e, b
    return own, bad


def check_rows(got, own, x, w, index, before=3.0):
    """Rows of every expert against the oracle (zeros where the index names no row), others as
    they were."""
    ok = (index >= 0) & (index < len(x))
    vals = np.where(ok[:, None], x[np.where(ok, index, 0)], 0.0)
    for e in range(len(w)):
        mine = own == e
        if mine.any():
            check_product(got[mine], vals[mine], w[e])
    assert (got[own < 0] == before).all()
    assert (got[(own >= 0) & ~ok] == 0).all()


@pytest.mark.parametrize("plan,e,m,n,k,index", TILES + STREAMS + WHOLE)
def test_bad_starts_and_rows(plan, e, m, n, k, index):
    dfl = goes_to(plan, e, m, n, k, index)
    rng = np.random.default_rng(m + n + k)
    n_src = 37 if index else m
    x, xs, xv = random_x(rng, n_src, k)
    w, wscale, wv = random_w(rng, e, n, k)
    ws, out = dfl.alloc_fp8_workspace(), Guarded((m, n), BF, fill=3.0)
    good = np.cumsum([0] + counts_of("even", e, m, rng))
    good[-1] = m
    skew = np.cumsum([0] + counts_of("skew", e, m, rng))
    down, past, below, wild = good.copy(), good.copy(), good.copy(), good.copy()
    down[e // 2] = max(int(good[e // 2 - 1]) - 3, 0) if good[e // 2 - 1] else m
    down[e // 2 + 1] = good[e // 2 - 1]                      # (claims rows of one before it)
    past[-1] = m + 1
    below[0] = -4
    wild[:2] = 2 ** 31 - 1, -2 ** 31
    rows = rng.integers(0, n_src, m) if index else np.arange(m)
    bad_rows = rows.copy()
    bad_rows[[0, m // 2, m - 1]] = n_src, -1, 2 ** 31 - 1
    for start, idx in ((good, rows), (skew, rows), (down, rows), (past, rows), (below, rows),
                       (wild, rows), (good, bad_rows), (past, bad_rows)):
        if idx is bad_rows and not index:
            continue
        out.t.fill_(3.0)
        dfl.dflash_fp8_grouped(x, xs, w, wscale, i32(start), i32(idx) if index else None, out.t, ws)
        own, bad = owners(start, m)
        bad = bad or bool(((idx < 0) | (idx >= n_src))[own >= 0].any())
        assert dfl.dflash_read_status(ws) == (dfl.dflash.STATUS_BITS["capacity"] if bad else 0)
        check_rows(f64(out.t), own, xv, wv, idx)
        out.check()


@pytest.mark.parametrize("plan,e,m,n,k,index", TILES + STREAMS)
@pytest.mark.parametrize("kind", ["skew", "one"])
def test_uneven_experts(plan, e, m, n, k, index, kind):
    """Experts without rows, and one with all of them, between rows that are no expert's."""
    dfl = goes_to(plan, e, m, n, k, index)
    rng = np.random.default_rng(m * 3 + n + k)
    before, behind = 2, 1 + m // 50
    start = np.cumsum([before] + counts_of(kind, e, m - before - behind, rng))
    n_src = 41 if index else m
    x, xs, xv = random_x(rng, n_src, k)
    w, wscale, wv = random_w(rng, e, n, k)
    rows = rng.integers(0, n_src, m) if index else np.arange(m)
    out, ws = Guarded((m, n), BF, fill=3.0), dfl.alloc_fp8_workspace()
    dfl.dflash_fp8_grouped(x, xs, w, wscale, i32(start), i32(rows) if index else None, out.t, ws)
    check_rows(f64(out.t), owners(start, m)[0], xv, wv, rows)
    out.check()
    assert dfl.dflash_read_status(ws) == 0


@pytest.mark.parametrize("plan,e,m,n,k,index", TILES + STREAMS[::3])
def test_replayed_with_other_experts(plan, e, m, n, k, index):
    """start and rows change between replays, to bad ones and back; twice in one graph."""
    dfl = goes_to(plan, e, m, n, k, index)
    rng = np.random.default_rng(m * 5 + n + k)
    n_src = 29 if index else m
    x, xs, xv = random_x(rng, n_src, k)
    w, wscale, wv = random_w(rng, e, n, k)
    start, rows = i32(np.zeros(e + 1)), i32(np.full(m, -1))
    outs = [torch.zeros(m, n, dtype=BF, device="cuda") for _ in range(2)]
    ws, graph = dfl.alloc_fp8_workspace(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for out in outs:
            dfl.dflash_fp8_grouped(x, xs, w, wscale, start, rows if index else None, out, ws)
    for kind in ("even", "bad", "skew", "none", "one"):
        edge = np.cumsum([0] + ([0] * e if kind == "none" else
                                counts_of("even" if kind == "bad" else kind, e, m - 3, rng)))
        idx = rng.integers(0, n_src, m) if index else np.arange(m)
        if kind == "bad":
            edge[e // 2] = m + 5
        start.copy_(i32(edge)), rows.copy_(i32(idx))
        for out in outs:
            out.fill_(3)
        graph.replay()
        own, bad = owners(edge, m)
        assert bad == (kind == "bad")
        check_rows(f64(outs[0]), own, xv, wv, idx)
        assert torch.equal(outs[0], outs[1])
        assert dfl.dflash_read_status(ws) == (dfl.dflash.STATUS_BITS["capacity"] if bad else 0)


# (tile rows, features, shares of K), m, n, k
LINEAR = [((16, 128, 8), 3, 300, 2064), ((32, 128, 8), 20, 387, 2064), ((32, 128, 1), 200, 300, 512),
          ((64, 128, 4), 140, 1000, 2064), ((64, 128, 1), 1100, 700, 144),
          ((128, 128, 1), 500, 2816, 512), ((128, 256, 1), 1500, 2816, 512),
          ((256, 256, 1), 1100, 2816, 656), ((256, 256, 1), 700, 5003, 4112)]


@pytest.mark.parametrize("plan,m,n,k", LINEAR)
def test_bad_values_stay_in_their_rows(plan, m, n, k):
    """A row with a scale of NaN and one with a code of NaN, a feature with a code of NaN and a block
    of features with an infinite scale."""
    dfl = goes_to(plan, 0, m, n, k, False)
    rng = np.random.default_rng(m + k)
    x, xs, xv = random_x(rng, m, k)
    w, wscale, wv = random_w(rng, n, k)
    out, ws = Guarded((m, n), BF), dfl.alloc_fp8_workspace()
    r, c = m // 2, n // 2
    xs[1, r] = float("nan")
    x.view(torch.uint8)[m - 1, k - 1] = 0xFF
    w.view(torch.uint8)[c, 100] = 0x7F
    last = (n - 1) // 128
    wscale[last, 0] = float("inf")
    dfl.dflash_fp8_linear(x, xs, w, wscale, out.t, ws)
    got = f64(out.t)
    inf = np.arange(n) >= last * 128
    assert np.isnan(got[[r, m - 1]]).all() and np.isnan(got[:, c]).all()
    assert not np.isfinite(got[:, inf]).any()
    keep_r = [i for i in range(m) if i not in (r, m - 1)]
    keep_c = [j for j in range(n) if j != c and not inf[j]]
    check_product(got[np.ix_(keep_r, keep_c)], xv[keep_r], wv[keep_c])
    out.check()


@pytest.mark.parametrize("plan,m,n,k", LINEAR)
def test_the_same_bits_again(plan, m, n, k):
    """Also as one expert's, where its rows in order go to the same kernel."""
    dfl = goes_to(plan, 0, m, n, k, False)
    rng = np.random.default_rng(m)
    x, xs, _ = random_x(rng, m, k)
    w, wscale, _ = random_w(rng, n, k)
    ws = dfl.alloc_fp8_workspace()
    first = torch.empty(m, n, dtype=BF, device="cuda")
    dfl.dflash_fp8_linear(x, xs, w, wscale, first, ws)
    for _ in range(5):
        again = torch.empty_like(first)
        dfl.dflash_fp8_linear(x, xs, w, wscale, again, ws)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))
    if dfl.dflash_fp8_plan(m, n, k, 1, False) == plan:
        dfl.dflash_fp8_grouped(x, xs, w[None], wscale[None], i32([0, m]), None, again, ws)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))
    assert dfl.dflash_read_status(ws) == 0


@pytest.mark.parametrize("m", [1, 5, 40, 300])
def test_buffers_for_the_most_rows_serve_fewer(m):
    """Codes cut to their first rows, scales from a flat buffer; and some of the rows by an index."""
    import block_diffusion_speculative_02_gb300 as dfl
    rng = np.random.default_rng(m)
    most, n, k = 320, 384, 400
    h = torch.from_numpy(rng.normal(size=(most, k))).to(BF).cuda()
    w, wscale, wv = random_w(rng, n, k)
    x_all, s_all = dfl.alloc_fp8_rows(most, k)
    x, xs = x_all[:m], s_all.view(-1)[:O.blocks(k) * m].view(O.blocks(k), m)
    dfl.dflash_fp8_norm_rows(h[:m], None, None, 0.0, None, x, xs)
    out, ws = Guarded((m, n), BF), dfl.alloc_fp8_workspace()
    dfl.dflash_fp8_linear(x, xs, w, wscale, out.t, ws)
    xv = O.rows_value(x.view(torch.uint8).cpu().numpy(), xs.cpu().numpy())
    check_product(f64(out.t), xv, wv)
    out.check()
    rows = np.arange(m // 2, m)
    part = torch.empty(len(rows), n, dtype=BF, device="cuda")
    dfl.dflash_fp8_grouped(x, xs, w[None], wscale[None], i32([0, len(rows)]), i32(rows), part, ws)
    check_product(f64(part), xv[rows], wv)
    assert dfl.dflash_read_status(ws) == 0
