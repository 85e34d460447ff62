"""GPU parity of the serving calls over a 4-bit KV cache against the float64
oracle, through the public binding."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as O

pytestmark = pytest.mark.gpu

I32, BF, U8 = torch.int32, torch.bfloat16, torch.uint8


def _dfl():
    import block_diffusion_speculative_02_gb300 as dfl
    return dfl


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.float32))).to(BF).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def status(ws):
    return _dfl().dflash_read_status(ws)


def bits(*names):
    return sum(_dfl().dflash.STATUS_BITS[n] for n in names)


class Cache:
    """A 4-bit cache with its float64 image: lengths, shuffled pages, random rows.

    Cell bytes no row was written to hold 0xFF (NaN scales, code -6)."""

    def __init__(self, rng, lens, hkv, d, page_size=16, spare=3, exps=True, extra_rows=0,
                 contiguous=0):
        dfl = _dfl()
        B = len(lens)
        self.hkv, self.d, self.page, self.lens = hkv, d, page_size, list(lens)
        self.k_exp = rng.integers(-3, 4, hkv) if exps else np.zeros(hkv, int)
        self.v_exp = rng.integers(-8, 2, hkv) if exps else np.zeros(hkv, int)
        self.k = [np.zeros((n, hkv, d)) for n in lens]
        self.v = [np.zeros((n, hkv, d)) for n in lens]
        if contiguous:
            self.table = None
            slabs, rows, cap = B, contiguous, contiguous
            slot = lambda b, i: (b, i)  # noqa: E731
        else:
            per = [-(-n // page_size) for n in lens]
            width = max(-(-(n + extra_rows) // page_size) for n in lens) + 1
            n_pages = sum(per) + B * -(-extra_rows // page_size) + spare
            order = rng.permutation(n_pages)
            self.table = np.full((B, width), -1)
            at = 0
            for b in range(B):
                self.table[b, :per[b]] = order[at:at + per[b]]
                at += per[b]
            self.free = np.concatenate([order[at:], order[:at]])
            self.count = n_pages - at
            slabs, rows, cap = n_pages, page_size, width * page_size
            slot = lambda b, i: (self.table[b, i // page_size], i % page_size)  # noqa: E731
        cells = np.full((slabs, hkv, rows // 16, 18 * d), 0xFF, np.uint8)
        for b, n in enumerate(lens):
            kx = np.ldexp(rng.normal(size=(n, hkv, d)), self.k_exp[:, None])
            vx = np.ldexp(rng.normal(size=(n, hkv, d)), self.v_exp[:, None])
            kc, ks = O.quantise(kx, self.k_exp)
            vc, vs = O.quantise(vx, self.v_exp)
            self.k[b], self.v[b] = O.values(kc, ks, self.k_exp), O.values(vc, vs, self.v_exp)
            for i in range(n):
                s, r = slot(b, i)
                for h in range(hkv):
                    O.put_row(cells[s, h, r // 16], r % 16, kc[i, h], ks[i, h], vc[i, h], vs[i, h])
        self.view = dfl.KV4View(
            torch.from_numpy(cells).cuda(), i32(lens), cap,
            None if contiguous else i32(self.table), None if contiguous else i32(self.free),
            None if contiguous else i32([self.count]), page_size,
            i32(self.k_exp) if exps else None, i32(self.v_exp) if exps else None)


def bound(ref, avg, e, v):
    """Element by element, with A = avg = sum p |v| / sum p and e = scale max sum |q||k| (the
    oracle's), n keys:
      2^-8 |ref|     the rounding to bf16 (half a step)
      A 2^-11 * 2    probabilities kept in fp16 for the second product, in numerator and
                     weight
      n 2^-32 max|v|  and small ones of them in steps of 2^-24, half a step each, where the
                     largest is at least 2^7 (so the weights' sum is too): a probability
                     below 2^-21 of the largest has no relative bound.  It shows where the
                     keys that matter have v = 0 in a dim.
      A 2^-22 * 4    exponentials (2^-22 relative)
      A e 2^-16      scores: 128 products summed in 32 bits (128 * 2^-24 of their
                     absolute sum) and one more rounding each of scale and subtraction
      A 2^-16        the same for the sums of the second product
    """
    return (2.0 ** -8 * np.abs(ref) + avg * (2.0 ** -10 + 2.0 ** -20 + (e + 1) * 2.0 ** -16)
            + len(v) * 2.0 ** -32 * np.abs(v).max(initial=0.0))


def check_attention(rng, cache, new, hq, causal, pad=0, scale=None, q_gain=1.0, q=None):
    """Runs the call on fresh queries and compares every row.

    See bound()."""
    dfl = _dfl()
    B, d, hkv = len(new), cache.d, cache.hkv
    n = sum(new) + pad
    scale = 1 / np.sqrt(d) if scale is None else scale
    dims = dfl.make_kv4_dims(B, n, max(max(new), 1), hq, hkv, d)
    ws = dfl.alloc_kv4_workspace(dims)
    if q is None:
        gain = np.ldexp(q_gain, -np.repeat(cache.k_exp, hq // hkv))[:, None]
        q = bf16(rng.normal(size=(n, hq, d)) * gain)
    start = np.concatenate([[0], np.cumsum(new)])
    out = torch.full((n, hq, d), -7.0, dtype=BF, device="cuda")
    dfl.dflash_kv4_attention(dims, q, i32(start), cache.view, float(scale), causal, out, ws)
    torch.cuda.synchronize()
    assert status(ws) == 0
    got, qd = f64(out), f64(q)
    for b, T in enumerate(new):
        lo, L = start[b], cache.lens[b]
        seen = [min(L, L - T + t + 1) if causal else L for t in range(T)]
        ref, avg, e = O.attention(qd[lo:lo + T], cache.k[b], cache.v[b], seen, scale)
        tol = bound(ref, avg, e, cache.v[b])
        err = np.abs(got[lo:lo + T] - ref)
        assert (err <= tol).all(), (b, np.argwhere(err > tol)[:5], (err - tol).max())
    assert (got[start[-1]:] == -7).all()                # padding rows are left
    return out


# ---------------------------------------------------------------------------
# page reservation
# ---------------------------------------------------------------------------
def run_reserve(lens, new, table, free, count, page, n_tokens, max_tokens, limit, alias=False):
    dfl = _dfl()
    B = len(lens)
    dims = dfl.make_kv4_dims(B, n_tokens, max_tokens, 1, 1, 64)
    ws = dfl.alloc_kv4_workspace(dims)
    seq = i32(lens)
    view = dfl.KVView(None, None, seq, limit, None if table is None else i32(table),
                      None if table is None else i32(free),
                      None if table is None else i32([count]), page)
    start, pos, slot = (torch.full((m,), -9, dtype=I32, device="cuda")
                        for m in (B + 1, n_tokens, n_tokens))
    new_len = seq if alias else torch.full((B,), -9, dtype=I32, device="cuda")
    dfl.dflash_kv_reserve(dims, view, i32(new), start, pos, slot, new_len, ws)
    torch.cuda.synchronize()
    ref = O.reserve(lens, new, None if table is None else np.array(table), np.array(free), count,
                    page, n_tokens, max_tokens, limit)
    assert status(ws) == bits(*ref["status"])
    for name, t in (("start", start), ("pos", pos), ("slot", slot), ("new_len", new_len)):
        np.testing.assert_array_equal(t.cpu().numpy(), ref[name], err_msg=name)
    if table is not None:
        np.testing.assert_array_equal(view.page_table.cpu().numpy(), ref["table"])
        assert int(view.free_count) == ref["free_count"]
    return ref


@pytest.mark.parametrize("B,page,new_hi,pad", [(1, 16, 1, 0), (1, 16, 900, 5), (5, 16, 40, 0),
                                               (33, 32, 17, 9), (300, 16, 3, 2), (70, 1, 9, 0),
                                               (40, 16, 700, 0), (1100, 16, 2, 0)])
def test_reserve(B, page, new_hi, pad):
    rng = np.random.default_rng(B + page)
    lens = rng.integers(0, 200, B)
    new = rng.integers(0, new_hi + 1, B)
    new[0] = new_hi
    width = int((lens + new).max()) // page + 2
    per = -(-lens // page)
    n_pages = int(per.sum() + (new // page + 2).sum())
    order = rng.permutation(n_pages)
    table, at = np.full((B, width), -1), 0
    for b in range(B):
        table[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
        if rng.random() < 0.3 and per[b] < width:       # a page mapped ahead of the rows
            table[b, min(per[b] + 1, width - 1)] = order[at]
            at += 1
    run_reserve(lens, new, table, np.concatenate([order[at:], order[:at]]), n_pages - at, page,
                int(new.sum()) + pad, new_hi, width * page, alias=B == 5)


@pytest.mark.parametrize("count", [0, 1, 2, 3, 5, 6])
def test_reserve_short_pool(count):
    """What fits is served in order; a sequence that lacks pages is left as it was."""
    lens, new = [3, 0, 16, 40, 15, 8], [4, 33, 20, 8, 2, 0]
    table = np.full((6, 5), -1)
    table[0, 0], table[2, 0], table[3, :3], table[4, 0], table[5, 0] = 20, 21, (22, 23, 24), 25, 26
    run_reserve(lens, new, table, np.arange(30), count, 16, 67, 64, 80)


def test_reserve_refuses_bad_sequences():
    """Negative counts and lengths, rows past the capacity, the array and max_tokens."""
    lens, new = [0, -1, 70, 5, 81, 0, 10], [2, 3, 11, -4, 1, 17, 6]
    table = np.full((7, 5), -1)
    ref = run_reserve(lens, new, table, np.arange(40), 40, 16, 36, 16, 80)
    assert ref["new_len"].tolist() == [2, -1, 70, 5, 81, 0, 10]


def test_reserve_contiguous_and_again():
    run_reserve([0, 7, 30], [4, 16, 2], None, [], 0, 0, 24, 16, 32)
    dfl = _dfl()
    table = np.full((2, 4), -1)
    dims = dfl.make_kv4_dims(2, 20, 16, 1, 1, 64)
    ws = dfl.alloc_kv4_workspace(dims)
    view = dfl.KVView(None, None, i32([0, 3]), 64, i32(table), i32(np.arange(9)), i32([9]), 16)
    got = []
    for _ in range(2):                                  # the same lengths: nothing changes
        o = [torch.zeros(m, dtype=I32, device="cuda") for m in (3, 20, 20, 2)]
        dfl.dflash_kv_reserve(dims, view, i32([4, 16]), *o, ws)
        got.append([x.tolist() for x in o] + [view.page_table.tolist(), int(view.free_count)])
    assert got[0] == got[1]


# ---------------------------------------------------------------------------
# norms and rotation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,hq,hkv,d", [(1, 4, 2, 64), (3, 5, 5, 128), (17, 32, 8, 128),
                                        (130, 7, 1, 64), (40, 64, 8, 128)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("place", ["own", "fused", "inplace"])
def test_qk_norm_rope(n, hq, hkv, d, norm, place):
    dfl = _dfl()
    rng = np.random.default_rng(n * d + hq)
    qkv = bf16(rng.normal(size=(n, (hq + 2 * hkv) * d)))
    q = qkv[:, :hq * d].unflatten(1, (hq, d))
    k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    if place == "own":
        q, k = q.contiguous(), k.contiguous()
    q0, k0, rest = f64(q), f64(k), f64(qkv[:, (hq + hkv) * d:])
    qw, kw = (bf16(1 + 0.2 * rng.normal(size=d)) for _ in range(2)) if norm else (None, None)
    pos = rng.integers(0, 300000, n)
    pos[0] = 2 ** 31 - 1 if n == 17 else 0
    pos[n // 2::7] = -1
    if place == "inplace":
        q_out, k_out = q, k
    else:
        q_out = torch.full((n, hq, d), 3.0, dtype=BF, device="cuda")
        k_out = torch.full((n, hkv, d), 3.0, dtype=BF, device="cuda")
    dims = dfl.make_kv4_dims(1, n, n, hq, hkv, d)
    dfl.dflash_qk_norm_rope(dims, q, k, qw, kw, i32(pos), 1e6, 1e-6, q_out, k_out)
    torch.cuda.synchronize()
    for x, w, y in ((q0, qw, q_out), (k0, kw, k_out)):
        ref = O.norm_rope(x, None if w is None else f64(w), pos, 1e6, 1e-6)
        # half a bf16 step, and for the arithmetic in 32 bits 2^-16 of the rotated pair:
        # (D + 8) roundings of 2^-24 in the norm, 2^-21 in the angle and its sine; the float64
        # angle itself is off by pos 2^-53
        pair = np.abs(ref) + np.abs(np.roll(ref, d // 2, axis=-1))
        tol = 2.0 ** -8 * np.abs(ref) + pair * (2.0 ** -16 + np.abs(pos)[:, None, None] * 2.0 ** -52)
        got = f64(y)
        keep = pos < 0
        assert (np.abs(got - ref) <= tol)[~keep].all()
        same = x if place == "inplace" else np.full_like(x, 3.0)
        np.testing.assert_array_equal(got[keep], same[keep])
    np.testing.assert_array_equal(f64(qkv[:, (hq + hkv) * d:]), rest)


# ---------------------------------------------------------------------------
# append and gather
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("hkv,d,page,contiguous", [(2, 64, 16, 0), (8, 128, 16, 0), (3, 128, 48, 0),
                                                   (1, 64, 0, 80)])
@pytest.mark.parametrize("n", [1, 15, 16, 100])
def test_append_and_gather(hkv, d, page, contiguous, n):
    """Rows at scattered slots, whole cells in order among them: the values are the oracle's
    exactly, other rows' bytes stay, and what is gathered goes in again."""
    dfl = _dfl()
    rng = np.random.default_rng(n + d + page)
    lens = [160] if not contiguous else [80, 80]
    cache = Cache(rng, lens, hkv, d, page or 16, spare=2, contiguous=contiguous)
    before = cache.view.cells.cpu().numpy().copy()
    rows = 160 if contiguous else int(cache.free.size) * page
    slot = rng.permutation(rows)[:n]
    if n == 100:
        slot = np.concatenate([np.arange(32, 80), np.setdiff1d(rng.permutation(rows), np.arange(
            32, 80), assume_unique=True)[:52]])
        slot[[50, 99]] = -1
    live = slot >= 0
    scale = np.exp2(rng.integers(-12, 13, (n, hkv, 1)))          # past both ends of the scales
    qkv = bf16(np.concatenate([rng.normal(size=(n, hkv, d)) * scale] * 3, 1))
    qkv[:, hkv:] *= 0.5
    k, v = qkv[:, :hkv], qkv[:, hkv:2 * hkv]
    if n > 1:
        k[1] = 0
    dims = dfl.make_kv4_dims(len(lens), n, n, hkv, hkv, d)
    ws = dfl.alloc_kv4_workspace(dims)
    dfl.dflash_kv4_append(dims, k, v, i32(slot), cache.view, ws)
    ko = torch.full((n, hkv, d), 5.0, dtype=BF, device="cuda")
    vo = torch.full((n, hkv, d), 5.0, dtype=BF, device="cuda")
    dfl.dflash_kv4_gather(dims, i32(slot), cache.view, ko, vo, ws)
    torch.cuda.synchronize()
    assert status(ws) == 0
    kc, ks = O.quantise(f64(k), cache.k_exp)
    vc, vs = O.quantise(f64(v), cache.v_exp)
    np.testing.assert_array_equal(f64(ko)[live], O.values(kc, ks, cache.k_exp)[live])
    np.testing.assert_array_equal(f64(vo)[live], O.values(vc, vs, cache.v_exp)[live])
    assert (f64(ko)[~live] == 5).all() and (f64(vo)[~live] == 5).all()
    # the bytes: the oracle's cells, up to the sign of zero codes
    slab_rows = contiguous or page
    for i in np.nonzero(live)[0]:
        s, r = divmod(int(slot[i]), slab_rows)
        for h in range(hkv):
            O.put_row(before[s, h, r // 16], r % 16, kc[i, h], ks[i, h], vc[i, h], vs[i, h])
    after = cache.view.cells.cpu().numpy()
    codes = lambda x: np.stack([x & 15, x >> 4])  # noqa: E731
    a, b = codes(after[..., :16 * d]), codes(before[..., :16 * d])
    assert ((a == b) | ((a & 7 == 0) & (b & 7 == 0))).all()
    np.testing.assert_array_equal(after[..., 16 * d:], before[..., 16 * d:])
    dfl.dflash_kv4_append(dims, ko, vo, i32(slot), cache.view, ws)
    k2, v2 = torch.zeros_like(ko), torch.zeros_like(vo)
    dfl.dflash_kv4_gather(dims, i32(slot), cache.view, k2, v2, ws)
    # again the same values where the scale is normal (code 8 and up) or 0.  A normal scale is
    # within 2^-4 of max / 6, so max / scale >= 6 / (1 + 2^-4) > 5.6 has code 6, the values'
    # maximum is 6 scale, and the same scale and codes follow.  A subnormal scale (a multiple
    # of 2^-9) may be up to half larger than max / 6: the largest code may be 4.
    for a, b, sc in ((k2, ko, ks), (v2, vo, vs)):
        sure = np.repeat((sc >= 8) | (sc == 0), 16, axis=-1) & live[:, None, None]
        assert sure.any() or n == 1
        np.testing.assert_array_equal(f64(a)[sure], f64(b)[sure])


def test_append_halfway_cases_and_every_scale():
    """Each row's largest element is 6 times a scale; the others lie halfway between codes."""
    dfl = _dfl()
    d, rows = 64, []
    for s in range(8, 127):                                       # normal scales
        row = np.zeros(d)
        for g in range(4):
            half = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
            row[16 * g:16 * g + 8] = np.array([6.0] + half) * O.E4M3[s] * (-1) ** g
            row[16 * g + 8] = O.E4M3[s] * 3
        rows.append(row)
    # and rows whose scale itself is halfway between two
    for s in range(8, 126):
        row = np.zeros(d)
        row[0], row[5] = 3 * (O.E4M3[s] + O.E4M3[s + 1]), 1.0
        rows.append(row)
    x = np.array(rows)[:, None, :]
    n = len(x)
    assert (f64(bf16(x)) == x).all()                              # bf16 holds them
    cache = Cache(np.random.default_rng(0), [n + 20], 1, d, exps=False)
    slot = np.array([cache.table[0, i // 16] * 16 + i % 16 for i in range(n)])
    dims = dfl.make_kv4_dims(1, n, n, 1, 1, d)
    ws = dfl.alloc_kv4_workspace(dims)
    ko, vo = (torch.zeros(n, 1, d, dtype=BF, device="cuda") for _ in range(2))
    dfl.dflash_kv4_append(dims, bf16(x), bf16(-x), i32(slot), cache.view, ws)
    dfl.dflash_kv4_gather(dims, i32(slot), cache.view, ko, vo, ws)
    ref = O.values(*O.quantise(x, [0]), [0])
    np.testing.assert_array_equal(f64(ko), ref)
    np.testing.assert_array_equal(f64(vo), -ref)
    assert status(ws) == 0


def test_append_bad_values_and_slots():
    dfl = _dfl()
    d = 64
    cache = Cache(np.random.default_rng(0), [16], 1, d, exps=False, spare=1)
    k = np.ones((4, 1, d))
    k[0, 0, 3], k[1, 0, 20], k[1, 0, 21] = np.nan, np.inf, -np.inf
    dims = dfl.make_kv4_dims(1, 4, 4, 1, 1, d)
    ws = dfl.alloc_kv4_workspace(dims)
    base = int(cache.table[0, 0]) * 16
    slot = i32([base, base + 1, 10 ** 6, base + 2])
    ko, vo = (torch.full((4, 1, d), 9.0, dtype=BF, device="cuda") for _ in range(2))
    dfl.dflash_kv4_append(dims, bf16(k), bf16(np.ones((4, 1, d))), slot, cache.view, ws)
    assert status(ws) == bits("bad_value", "capacity")
    dfl.dflash_kv4_gather(dims, slot, cache.view, ko, vo, ws)
    assert status(ws) == bits("capacity")
    got = f64(ko)[:, 0]
    one = O.values(*O.quantise(np.ones((1, 16)), [0]), [0])[0]
    assert got[0, 3] == 0 and (got[0, :3] == one[0]).all()
    assert got[1, 20] == 2688 and got[1, 21] == -2688 and (got[1, 32:] == one[0]).all()
    assert (got[2] == 9).all() and (got[3] == one[0]).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 2, 128), (8, 1, 128), (3, 3, 64),
                                      (16, 1, 128), (64, 1, 64)])
@pytest.mark.parametrize("T", [1, 2, 5, 16])
def test_attention_lengths(causal, hq, hkv, d, T):
    """Lengths around the edges of cells, tiles of keys and pages; a length below T."""
    rng = np.random.default_rng(d * T + hq)
    lens = [T, 1, 15, 17, 64, 127, 128, 130, 257, 0]
    cache = Cache(rng, lens, hkv, d)
    check_attention(rng, cache, [T] * len(lens), hq, causal, pad=2)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (16, 4, 128)])
def test_attention_ragged(causal, hq, hkv, d):
    """Rows per sequence from none to more than one tile of query rows."""
    rng = np.random.default_rng(hq)
    new = [0, 70, 1, 0, 16, 33, 3, 0]
    lens = [40, 70, 300, 0, 500, 90, 3, 12]
    check_attention(rng, Cache(rng, lens, hkv, d), new, hq, causal, pad=3)


@pytest.mark.parametrize("page", [32, 48, 128])
def test_attention_larger_pages(page):
    rng = np.random.default_rng(page)
    check_attention(rng, Cache(rng, [1, 200, 333], 2, 128, page_size=page), [1, 4, 9], 8, True)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_contiguous(causal):
    rng = np.random.default_rng(5)
    check_attention(rng, Cache(rng, [3, 272, 150], 2, 128, contiguous=272, exps=False),
                    [2, 16, 1], 8, causal)


def test_attention_many_sequences():
    """More sequences than there are SMs, most of them short."""
    rng = np.random.default_rng(11)
    lens = rng.integers(1, 40, 170)
    lens[7] = 700
    check_attention(rng, Cache(rng, lens, 1, 64), [1] * 170, 2, True)


@pytest.mark.parametrize("q_gain", [40.0, 1e-3])
def test_attention_sharp_and_flat(q_gain):
    """Scores of a few hundred (one key takes all) and of next to nothing."""
    rng = np.random.default_rng(3)
    check_attention(rng, Cache(rng, [700, 1, 129], 2, 128), [16, 1, 16], 8, True, q_gain=q_gain)


def test_attention_rows_of_unlike_size():
    """Queries of one call a factor 2^30 apart, and rows of zeros."""
    rng = np.random.default_rng(4)
    cache = Cache(rng, [300], 1, 128, exps=False)
    q = rng.normal(size=(16, 4, 128)) * np.exp2(rng.integers(-15, 16, (16, 4, 1)))
    q[3] = 0
    check_attention(rng, cache, [16], 4, True, q=bf16(q), scale=2.0 ** -14)


def test_attention_rising_scores():
    """Keys ordered so that the running maximum moves again and again, and falls."""
    rng = np.random.default_rng(6)
    cache = Cache(rng, [2000], 1, 128, exps=False)
    q = rng.normal(size=(16, 4, 128)) * 8
    for order in (1, -1):
        rank = np.argsort(order * (cache.k[0][:, 0] @ q[5, 2]))
        kk, vv = cache.k[0][rank], cache.v[0][rank]
        again = Cache(rng, [2000], 1, 128, exps=False)
        dfl = _dfl()
        dims = dfl.make_kv4_dims(1, 2000, 2000, 1, 1, 128)
        ws = dfl.alloc_kv4_workspace(dims)
        slot = [again.table[0, i // 16] * 16 + i % 16 for i in range(2000)]
        dfl.dflash_kv4_append(dims, bf16(kk), bf16(vv), i32(slot), again.view, ws)
        again.k[0], again.v[0] = kk, vv
        check_attention(rng, again, [16], 4, False, q=bf16(q))


def test_attention_nan_query_stays_in_its_row():
    rng = np.random.default_rng(8)
    cache = Cache(rng, [200], 1, 64)
    dfl = _dfl()
    q = bf16(rng.normal(size=(16, 4, 64)))
    clean = check_attention(rng, cache, [16], 4, True, q=q)
    bad = q.clone()
    bad[5, 2, 7] = float("nan")
    out = torch.zeros_like(q)
    dims = dfl.make_kv4_dims(1, 16, 16, 4, 1, 64)
    dfl.dflash_kv4_attention(dims, bad, i32([0, 16]), cache.view, 0.125, True, out,
                             dfl.alloc_kv4_workspace(dims))
    got, ref = f64(out), f64(clean)
    assert np.isnan(got[5, 2]).all()
    got[5, 2] = ref[5, 2]
    np.testing.assert_array_equal(got, ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("group,T", [(1, 1), (4, 1), (8, 1), (3, 5), (16, 1), (7, 4), (4, 16), (5, 12),
                                     (8, 16), (16, 13)])
def test_attention_long_and_uneven(group, T, causal, d):
    """Contexts that many CTAs share beside short ones: units cut at any tile, CTAs with
    several units, at every number of query rows to a unit."""
    rng = np.random.default_rng(group * T)
    lens = [int(x) for x in rng.integers(1, 900, 12)] + [6000, 1, 129, 2500]
    new = [min(T, n) if i % 5 else 0 for i, n in enumerate(lens)]
    check_attention(rng, Cache(rng, lens, 1, d), new, group, causal, pad=1)


@pytest.mark.parametrize("group,T", [(2, 1), (4, 4), (8, 4), (4, 16), (4, 30)])
def test_attention_scale_zero_and_negative(group, T):
    """Scale 0 weighs every row alike; a negative one turns the order round."""
    rng = np.random.default_rng(T)
    cache = Cache(rng, [300, 40], 2, 64)
    for scale in (0.0, -0.125):
        check_attention(rng, cache, [T, T], 2 * group, True, scale=scale)


@pytest.mark.parametrize("group,T", [(2, 1), (4, 4), (8, 4), (4, 16), (4, 30)])
def test_attention_zero_rows_at_the_smallest_gain(group, T):
    """Factors of a score below 2^-149: rows past the length and masked ones still count nothing."""
    rng = np.random.default_rng(T)
    cache = Cache(rng, [37, 200], 1, 128)
    cache.k = [np.ldexp(k, -64 - cache.k_exp[:, None]) for k in cache.k]
    cache.view.k_exp = i32([-64])
    q = torch.zeros(2 * T, group, 128, dtype=BF, device="cuda")
    check_attention(rng, cache, [T, T], group, True, q=q)


@pytest.mark.parametrize("T", [1, 4, 16])
def test_attention_infinite_and_nan_queries_stay_in_their_rows(T):
    dfl = _dfl()
    rng = np.random.default_rng(T)
    cache = Cache(rng, [200, 31], 1, 64)
    q = bf16(rng.normal(size=(2 * T, 4, 64)))
    clean = f64(check_attention(rng, cache, [T, T], 4, True, q=q))
    bad = q.clone()
    bad[0, 2, 7], bad[T, 1, 3], bad[T, 3, 0] = float("inf"), float("nan"), float("-inf")
    out = torch.zeros_like(q)
    dims = dfl.make_kv4_dims(2, 2 * T, T, 4, 1, 64)
    dfl.dflash_kv4_attention(dims, bad, i32([0, T, 2 * T]), cache.view, 0.125, True, out,
                             dfl.alloc_kv4_workspace(dims))
    got = f64(out)
    for row in ((0, 2), (T, 1), (T, 3)):
        assert np.isnan(got[row]).all()
        got[row] = clean[row]
    np.testing.assert_array_equal(got, clean)


def test_attention_bad_sequences_and_pages():
    """Bad lengths leave the output; pages that are missing or numbered past the pool read
    as zeros; the other sequences of the batch are right."""
    dfl = _dfl()
    rng = np.random.default_rng(9)
    cache = Cache(rng, [100, 100, 100, 40, 60], 1, 64)
    new = [2, 2, 2, 9, 2]
    start = np.concatenate([[0], np.cumsum(new)])
    cache.view.seq_len.copy_(i32([100, -1, 10 ** 6, 40, 60]))
    cache.view.page_table[0, 2] = -1
    cache.view.page_table[4, 1] = 10 ** 6
    for b, page in ((0, 2), (4, 1)):
        cache.k[b][16 * page:16 * page + 16] = cache.v[b][16 * page:16 * page + 16] = 0
    dims = dfl.make_kv4_dims(5, 17, 8, 4, 1, 64)
    ws = dfl.alloc_kv4_workspace(dims)
    q = bf16(rng.normal(size=(17, 4, 64)))
    out = torch.full_like(q, 2.0)
    dfl.dflash_kv4_attention(dims, q, i32(start), cache.view, 0.125, True, out, ws)
    assert status(ws) == bits("capacity", "page_missing")
    got = f64(out)
    assert (got[2:15] == 2).all()
    for b, lo, L in ((0, 0, 100), (4, 15, 60)):
        ref, avg, _ = O.attention(f64(q)[lo:lo + 2], cache.k[b], cache.v[b], [L - 1, L], 0.125)
        assert (np.abs(got[lo:lo + 2] - ref) <= 2.0 ** -8 * np.abs(ref) + avg * 2.0 ** -9).all()
    # row offsets outside the batch's rows
    cache.view.seq_len.copy_(i32([100, 100, 100, 40, 60]))
    for bad in ([-2, 2, 4, 6, 8, 10], [0, 2, 1, 3, 5, 30]):
        out.fill_(2.0)
        dfl.dflash_kv4_attention(dims, q, i32(bad), cache.view, 0.125, True, out, ws)
        assert status(ws) & bits("capacity")
        assert not (f64(out)[4 if bad[0] < 0 else 1] == 2).all()


@pytest.mark.parametrize("T,causal", [(1, True), (16, False), (200, True)])
def test_attention_repeats_its_bits(T, causal):
    """Split work is joined in a fixed order: two runs give the same bits."""
    dfl = _dfl()
    rng = np.random.default_rng(T)
    cache = Cache(rng, [1500, 700], 2, 128)
    dims = dfl.make_kv4_dims(2, 2 * T, T, 8, 2, 128)
    ws = dfl.alloc_kv4_workspace(dims)
    q = bf16(rng.normal(size=(2 * T, 8, 128)))
    outs = []
    for _ in range(5):
        out = torch.zeros_like(q)
        dfl.dflash_kv4_attention(dims, q, i32([0, T, 2 * T]), cache.view, 0.1, causal, out, ws)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_attention_far_pool():
    """Cells past 2^31 and 2^32 bytes of the pool, and slots written and read there."""
    dfl = _dfl()
    rng = np.random.default_rng(12)
    hkv, d = 8, 128
    small = Cache(rng, [50, 300], hkv, d)
    per = 18 * d * hkv
    n_pages = 2 ** 32 // per + 4096
    cells = torch.zeros(n_pages, hkv, 1, 18 * d, dtype=U8, device="cuda")
    far = small.table.copy()
    used = sorted(far[far >= 0])
    for i, page in enumerate(used):
        to = n_pages - 1 - 7 * i if i % 2 else 2 ** 31 // per + 3 * i
        cells[to] = small.view.cells[int(page)]
        far[small.table == page] = to
    small.view.cells = cells
    small.view.page_table = i32(far)
    small.view.free_list = torch.zeros(n_pages, dtype=I32, device="cuda")
    check_attention(rng, small, [3, 16], 32, True)
    n = 20
    dims = dfl.make_kv4_dims(2, n, n, hkv, hkv, d)
    ws = dfl.alloc_kv4_workspace(dims)
    slot = i32([int(far[1, 18 - i // 16]) * 16 + i % 16 for i in range(n)])
    ko, vo = (torch.zeros(n, hkv, d, dtype=BF, device="cuda") for _ in range(2))
    dfl.dflash_kv4_gather(dims, slot, small.view, ko, vo, ws)
    for i in range(min(n, 12)):
        np.testing.assert_array_equal(f64(ko)[i], small.k[1][18 * 16 + i])
    x = bf16(rng.normal(size=(n, hkv, d)))
    dfl.dflash_kv4_append(dims, x, x, slot, small.view, ws)
    dfl.dflash_kv4_gather(dims, slot, small.view, ko, vo, ws)
    ref = O.values(*O.quantise(f64(x), small.k_exp), small.k_exp)
    np.testing.assert_array_equal(f64(ko), ref)


# ---------------------------------------------------------------------------
# the calls together
# ---------------------------------------------------------------------------
def test_serving_steps_end_to_end():
    """Prompts of uneven lengths, a token each, blocks with a crop, a sequence that joins: each
    step reserves, norms and rotates, appends, attends and (after a block) crops, on one stream
    that is not the default one; every output against the oracle's own cache."""
    dfl = _dfl()
    rng = np.random.default_rng(21)
    B, hq, hkv, d, theta, eps = 4, 8, 2, 128, 1e6, 1e-6
    n_pages, width = 60, 20
    view = dfl.KV4View(dfl.alloc_kv4_cells(n_pages, hkv, 16, d), i32([0] * B), width * 16,
                       i32(np.full((B, width), -1)), i32(rng.permutation(n_pages)), i32([n_pages]),
                       16, i32([1, -1]), i32([-2, 0]))
    k_exp, v_exp = np.array([1, -1]), np.array([-2, 0])
    K, V = [np.zeros((0, hkv, d))] * B, [np.zeros((0, hkv, d))] * B
    qw, kw = bf16(1 + 0.1 * rng.normal(size=d)), bf16(1 + 0.1 * rng.normal(size=d))
    side = torch.cuda.Stream()
    steps = [([37, 100, 0, 16], True, None), ([1, 1, 1, 1], True, None),
             ([16, 16, 16, 16], True, [3, 16, 0, 9]), ([16, 16, 0, 16], False, [0, 0, 0, 0]),
             ([1, 0, 60, 1], True, None)]
    for new, causal, keep in steps:
        n, pad = sum(new), 3
        dims = dfl.make_kv4_dims(B, n + pad, max(new), hq, hkv, d)
        ws = dfl.alloc_kv4_workspace(dims)
        qkv = bf16(rng.normal(size=(n + pad, (hq + 2 * hkv) * d)))
        q = qkv[:, :hq * d].unflatten(1, (hq, d))
        k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        v = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        start, pos, slot = (torch.zeros(m, dtype=I32, device="cuda")
                            for m in (B + 1, n + pad, n + pad))
        q_out = torch.zeros(n + pad, hq, d, dtype=BF, device="cuda")
        out = torch.zeros_like(q_out)
        n_new, before = i32(new), view.seq_len.clone()
        side.wait_stream(torch.cuda.current_stream())
        dfl.dflash_kv_reserve(dims, view, n_new, start, pos, slot, view.seq_len, ws, stream=side)
        dfl.dflash_qk_norm_rope(dims, q, k, qw, kw, pos, theta, eps, q_out, k, stream=side)
        dfl.dflash_kv4_append(dims, k, v, slot, view, ws, stream=side)
        dfl.dflash_kv4_attention(dims, q_out, start, view, d ** -0.5, causal, out, ws, stream=side)
        kept = None
        if keep is not None:
            kept = before + i32(keep)
            side.wait_stream(torch.cuda.current_stream())
            dfl.dflash_kv_crop([view.pages()], kept, B, ws, stream=side)
        side.synchronize()
        assert status(ws) == 0
        kd, vd, qd, got, at = f64(k), f64(v), f64(q_out), f64(out), 0
        for b, T in enumerate(new):
            rows = slice(at, at + T)
            K[b] = np.concatenate([K[b], O.values(*O.quantise(kd[rows], k_exp), k_exp)])
            V[b] = np.concatenate([V[b], O.values(*O.quantise(vd[rows], v_exp), v_exp)])
            L = len(K[b])
            seen = [L - T + t + 1 if causal else L for t in range(T)]
            ref, avg, e = O.attention(qd[rows], K[b], V[b], seen, d ** -0.5)
            tol = bound(ref, avg, e, V[b])
            assert (np.abs(got[rows] - ref) <= tol).all(), (new, b)
            if keep is not None:
                K[b], V[b] = K[b][:L - T + keep[b]], V[b][:L - T + keep[b]]
            at += T
        assert view.seq_len.tolist() == [len(x) for x in K]
    held = sum(-(-len(x) // 16) for x in K)
    assert int(view.free_count) == n_pages - held


def test_captured_step_replays_with_other_lengths():
    """A decode step captured once and replayed: lengths, pages and rows are read on the
    device each time; two graphs that share a workspace, replayed in turn."""
    dfl = _dfl()
    rng = np.random.default_rng(22)
    B, hq, hkv, d, pad = 3, 4, 1, 64, 4
    view = dfl.KV4View(dfl.alloc_kv4_cells(64, hkv, 16, d), i32([0] * B), 20 * 16,
                       i32(np.full((B, 20), -1)), i32(np.arange(64)), i32([64]), 16)
    n = 3 * 16 + pad
    dims = dfl.make_kv4_dims(B, n, 16, hq, hkv, d)
    ws = dfl.alloc_kv4_workspace(dims)
    n_new = i32([1] * B)
    start, pos, slot = (torch.zeros(m, dtype=I32, device="cuda") for m in (B + 1, n, n))
    q, k, v = (torch.zeros(n, h, d, dtype=BF, device="cuda") for h in (hq, hkv, hkv))
    outs = [torch.zeros_like(q) for _ in range(2)]

    def step(out, causal):
        dfl.dflash_kv_reserve(dims, view, n_new, start, pos, slot, view.seq_len, ws)
        dfl.dflash_kv4_append(dims, k, v, slot, view, ws)
        dfl.dflash_kv4_attention(dims, q, start, view, 0.125, causal, out, ws)

    graphs = []
    for out, causal in zip(outs, (True, False)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(out, causal)
        graphs.append(g)
    assert view.seq_len.tolist() == [0] * B                       # capture runs nothing
    K, V = [np.zeros((0, hkv, d))] * B, [np.zeros((0, hkv, d))] * B
    for i, new in enumerate([[16, 3, 0], [1, 1, 1], [16, 16, 16], [0, 5, 1], [1, 1, 1]]):
        m = sum(new)
        n_new.copy_(i32(new))
        for t in (q, k, v):
            t.copy_(bf16(rng.normal(size=t.shape)))
        outs[i % 2].fill_(4.0)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert status(ws) == 0
        at = 0
        for b, T in enumerate(new):
            rows = slice(at, at + T)
            K[b] = np.concatenate([K[b], O.values(*O.quantise(f64(k)[rows], [0]), [0])])
            V[b] = np.concatenate([V[b], O.values(*O.quantise(f64(v)[rows], [0]), [0])])
            L = len(K[b])
            seen = [L - T + t + 1 if i % 2 == 0 else L for t in range(T)]
            ref, avg, e = O.attention(f64(q)[rows], K[b], V[b], seen, 0.125)
            tol = bound(ref, avg, e, V[b])
            assert (np.abs(f64(outs[i % 2])[rows] - ref) <= tol).all(), (i, b)
            at += T
        assert (f64(outs[i % 2])[m:] == 4).all()


def test_refuses_wrong_tensors():
    dfl = _dfl()
    rng = np.random.default_rng(1)
    cache = Cache(rng, [20], 1, 64)
    dims = dfl.make_kv4_dims(1, 2, 2, 2, 1, 64)
    ws = dfl.alloc_kv4_workspace(dims)
    q = torch.zeros(2, 2, 64, dtype=BF, device="cuda")
    call = lambda q, out, start, w=ws: dfl.dflash_kv4_attention(  # noqa: E731
        dims, q, start, cache.view, 1.0, True, out, w)
    s = i32([0, 2])
    for bad in (q.float(), q.cpu(), q[:1], q.transpose(0, 1)):
        with pytest.raises(ValueError):
            call(bad, q, s)
        with pytest.raises(ValueError):
            call(q, bad, s)
    with pytest.raises(ValueError):
        call(q, q, s[:1])
    with pytest.raises(dfl.DFlashError):
        call(q, torch.zeros_like(q), s, ws[:128])
    with pytest.raises(ValueError):
        dfl.dflash_kv4_append(dims, q, q, s[:2], cache.view, ws)     # two heads, one expected
    with pytest.raises(ValueError):
        cache.view.cells = cache.view.cells[:1]
        call(q, torch.zeros_like(q), s)


def test_view_follows_its_tensors():
    """A view whose tensors are exchanged, moved or resized between calls is read anew."""
    rng = np.random.default_rng(31)
    cache = Cache(rng, [40, 70], 1, 64)
    check_attention(rng, cache, [1, 1], 2, True)
    wide = torch.full((2, 12), -1, dtype=I32, device="cuda")
    wide[:, :cache.view.page_table.shape[1]] = cache.view.page_table
    old, cache.view.page_table = cache.view.page_table, wide
    check_attention(rng, cache, [1, 1], 2, True)
    width = old.shape[1]
    wide.resize_(2, width)                              # the same tensor at the same address
    wide.copy_(old)
    check_attention(rng, cache, [1, 1], 2, True)
    other = Cache(rng, [40, 70], 1, 64)
    cache.view.cells, cache.view.page_table = other.view.cells, other.view.page_table
    cache.view.k_exp, cache.view.v_exp = other.view.k_exp, other.view.v_exp
    cache.k, cache.v, cache.k_exp = other.k, other.v, other.k_exp
    check_attention(rng, cache, [1, 1], 2, True)


def test_two_streams_at_once():
    """Two attentions on two streams with a workspace each, over one cache."""
    dfl = _dfl()
    rng = np.random.default_rng(32)
    cache = Cache(rng, [900, 500, 1300], 2, 128)
    outs, refs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for T in (16, 1):
        gain = np.ldexp(1.0, -np.repeat(cache.k_exp, 4))[:, None]
        q = bf16(rng.normal(size=(3 * T, 8, 128)) * gain)
        refs.append(check_attention(rng, cache, [T] * 3, 8, True, q=q))
        outs.append((T, q, torch.zeros_like(q)))
    jobs = []
    for (T, q, out), st in zip(outs, streams):
        dims = dfl.make_kv4_dims(3, 3 * T, T, 8, 2, 128)
        jobs.append((dims, q, i32(np.arange(4) * T), out, dfl.alloc_kv4_workspace(dims), st))
    torch.cuda.synchronize()
    for _ in range(20):
        for dims, q, start, out, ws, st in jobs:
            dfl.dflash_kv4_attention(dims, q, start, cache.view, 1 / np.sqrt(128), True, out, ws,
                                     stream=st)
    torch.cuda.synchronize()
    for (dims, q, start, out, ws, st), ref in zip(jobs, refs):
        assert status(ws) == 0
        assert torch.equal(out, ref)


def test_norm_rope_follows_theta_and_head_dim():
    """Calls in turn with other bases and head dims: each has its own angles."""
    dfl = _dfl()
    rng = np.random.default_rng(33)
    for d, theta in ((64, 1e4), (128, 1e4), (128, 1e6), (64, 1e4), (64, 5e5)):
        q, k = bf16(rng.normal(size=(5, 2, d))), bf16(rng.normal(size=(5, 1, d)))
        pos = [0, 1, 77, 4095, 100000]
        qo, ko = torch.zeros_like(q), torch.zeros_like(k)
        dims = dfl.make_kv4_dims(1, 5, 5, 2, 1, d)
        dfl.dflash_qk_norm_rope(dims, q, k, None, None, i32(pos), theta, 1e-6, qo, ko)
        for x, y in ((q, qo), (k, ko)):
            a = np.array(pos)[:, None] * theta ** (-2.0 * np.arange(d // 2) / d)
            c, s = np.cos(a)[:, None], np.sin(a)[:, None]
            lo, hi = f64(x)[..., :d // 2], f64(x)[..., d // 2:]
            ref = np.concatenate([lo * c - hi * s, hi * c + lo * s], -1)
            mag = np.concatenate([np.abs(lo) + np.abs(hi)] * 2, -1)
            # half a step of bf16; angles off by 2^-23 turns, cosines and products by a few 2^-24
            assert (np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * mag).all()


@pytest.mark.parametrize("n_tokens", [40, 8300])              # one launch, and two
def test_reserve_counts_past_int32(n_tokens):
    """Counts whose sum passes 2^31 (offsets stop there): every sequence behind is refused."""
    dfl = _dfl()
    lens, new = [4, 0, 7, 3], [5, 2 ** 31 - 3, 40, 2 ** 31 - 1]
    dims = dfl.make_kv4_dims(4, n_tokens, 16, 1, 1, 64)
    ws = dfl.alloc_kv4_workspace(dims)
    view = dfl.KVView(None, None, i32(lens), 64, i32(np.full((4, 4), -1)), i32(range(9)), i32([9]),
                      16)
    guard = 4096
    start, new_len = (torch.full((m,), -9, dtype=I32, device="cuda") for m in (5, 4))
    pos, slot = (torch.full((n_tokens + 2 * guard,), -9, dtype=I32, device="cuda")
                 for _ in range(2))
    inner = slice(guard, guard + n_tokens)
    dfl.dflash_kv_reserve(dims, view, i32(new), start, pos[inner], slot[inner], new_len, ws)
    assert status(ws) == bits("capacity")
    top = 2 ** 31 - 1
    assert start.tolist() == [0, 5, top, top, top] and new_len.tolist() == [9, 0, 7, 3]
    assert pos[inner].tolist() == [4, 5, 6, 7, 8] + [-1] * (n_tokens - 5)
    assert slot[inner].tolist() == [8 * 16 + i for i in range(4, 9)] + [-1] * (n_tokens - 5)
    for t in (pos, slot):
        assert (t[:guard] == -9).all() and (t[guard + n_tokens:] == -9).all()
    assert int(view.free_count) == 8 and view.page_table[0].tolist() == [8, -1, -1, -1]


@pytest.mark.parametrize("T,group", [(1, 4), (3, 4), (8, 4), (16, 4), (32, 4)])
@pytest.mark.parametrize("page", [16, 48])
def test_attention_missing_pages_among_copies(T, group, page):
    """Missing pages throughout long contexts: the zeros that stand for them lie where copies
    landed before and land again after, at every width of a unit."""
    dfl = _dfl()
    rng = np.random.default_rng(T + page)
    lens = [6000, 900]
    cache = Cache(rng, lens, 1, 128, page_size=page)
    for b, n in enumerate(lens):
        gone = rng.random(-(-n // page)) < 0.3
        gone[-1] = False
        for i in np.nonzero(gone)[0]:
            cache.view.page_table[b, i] = -1 if i % 2 else 10 ** 6
            cache.k[b][page * i:page * (i + 1)] = cache.v[b][page * i:page * (i + 1)] = 0
    dims = dfl.make_kv4_dims(2, 2 * T, T, group, 1, 128)
    ws = dfl.alloc_kv4_workspace(dims)
    q = bf16(rng.normal(size=(2 * T, group, 128)) * np.ldexp(1.0, -cache.k_exp[0]))
    scale, outs = 128 ** -0.5, []
    for _ in range(3):
        out = torch.zeros_like(q)
        dfl.dflash_kv4_attention(dims, q, i32([0, T, 2 * T]), cache.view, scale, True, out, ws)
        assert status(ws) == bits("page_missing")
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    got = f64(outs[0])
    for b, L in enumerate(lens):
        rows = slice(b * T, b * T + T)
        ref, avg, e = O.attention(f64(q)[rows], cache.k[b], cache.v[b],
                                  [L - T + t + 1 for t in range(T)], scale)
        assert (np.abs(got[rows] - ref) <= bound(ref, avg, e, cache.v[b])).all(), b


# one launch (at most 256 sequences and 8192 rows), and the two launches of larger batches
TWO_LAUNCHES = [0, 8300]


def _grown(lens, new, table, batch):
    """The same sequences, with sequences of length 0 without new rows behind them."""
    more = batch - len(lens)
    return (list(lens) + [0] * more, list(new) + [0] * more,
            np.concatenate([table, np.full((more, table.shape[1]), -1)]))


@pytest.mark.parametrize("pad", TWO_LAUNCHES)
@pytest.mark.parametrize("batch", [6, 300])
@pytest.mark.parametrize("count", [0, 1, 2, 3, 5, 6])
def test_reserve_short_pool_both_ways(count, batch, pad):
    lens, new = [3, 0, 16, 40, 15, 8], [4, 33, 20, 8, 2, 0]
    table = np.full((6, 5), -1)
    table[0, 0], table[2, 0], table[3, :3], table[4, 0], table[5, 0] = 20, 21, (22, 23, 24), 25, 26
    lens, new, table = _grown(lens, new, table, batch)
    for alias in (False, True):
        ref = run_reserve(lens, new, table, np.arange(30), count, 16, 67 + pad, 64, 80, alias=alias)
        assert ("pool_empty" in ref["status"]) == (count < 6)


@pytest.mark.parametrize("pad", TWO_LAUNCHES)
@pytest.mark.parametrize("batch", [7, 300])
def test_reserve_refuses_bad_sequences_both_ways(batch, pad):
    lens, new = [0, -1, 70, 5, 81, 0, 10], [2, 3, 11, -4, 1, 17, 6]
    lens, new, table = _grown(lens, new, np.full((7, 5), -1), batch)
    for alias in (False, True):
        ref = run_reserve(lens, new, table, np.arange(40), 40, 16, 36 + pad, 16, 80, alias=alias)
        # (the last one's rows fit the array once it is padded)
        assert ref["new_len"][:7].tolist() == [2, -1, 70, 5, 81, 0, 16 if pad else 10]


@pytest.mark.parametrize("pad", TWO_LAUNCHES)
@pytest.mark.parametrize("batch", [3, 300])
def test_reserve_contiguous_both_ways(batch, pad):
    lens, new, _ = _grown([0, 7, 30], [4, 16, 2], np.full((3, 1), -1), batch)
    for alias in (False, True):
        run_reserve(lens, new, None, [], 0, 0, 24 + pad, 16, 32, alias=alias)


@pytest.mark.parametrize("pad", TWO_LAUNCHES)
def test_reserve_again_both_ways(pad):
    """A second call with the same lengths changes nothing; one in place goes on from there."""
    dfl = _dfl()
    n = 20 + pad
    dims = dfl.make_kv4_dims(2, n, 16, 1, 1, 64)
    ws = dfl.alloc_kv4_workspace(dims)
    view = dfl.KVView(None, None, i32([0, 3]), 64, i32(np.full((2, 4), -1)), i32(np.arange(9)),
                      i32([9]), 16)
    got = []
    for _ in range(2):
        o = [torch.zeros(m, dtype=I32, device="cuda") for m in (3, n, n, 2)]
        dfl.dflash_kv_reserve(dims, view, i32([4, 16]), *o, ws)
        got.append([x.tolist() for x in o] + [view.page_table.tolist(), int(view.free_count)])
    assert got[0] == got[1]
    for lens in ([4, 19], [8, 35], [12, 51]):
        o = [torch.zeros(m, dtype=I32, device="cuda") for m in (3, n, n)]
        dfl.dflash_kv_reserve(dims, view, i32([4, 16]), *o, view.seq_len, ws)
        assert view.seq_len.tolist() == lens
        assert o[1][:4].tolist() == list(range(lens[0] - 4, lens[0]))
    assert status(ws) == 0


@pytest.mark.parametrize("B,pad", [(20, 8300), (280, 0)])
def test_reserve_random_two_launches(B, pad):
    """Random lengths, counts (bad ones among them), tables and pools, some of them too small."""
    rng = np.random.default_rng(B)
    for _ in range(8):
        lens = rng.integers(0, 90, B)
        new = rng.integers(0, 40, B)
        new[rng.random(B) < 0.1] = -3
        lens[rng.random(B) < 0.05] = -2
        table, at = np.full((B, 7), -1), 0
        order = rng.permutation(10 * B)
        for b in range(B):
            per = -(-max(lens[b], 0) // 16)
            table[b, :per] = order[at:at + per]
            at += per
        count = int(rng.integers(0, 3 * B))
        run_reserve(lens, new, table, np.concatenate([order[at:], order[:at]]), count, 16,
                    int(np.maximum(new, 0).sum()) + pad, 38, 112, alias=rng.random() < 0.5)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("T", [1, 6, 16, 40])
def test_attention_refuses_more_tiles_than_int32(T, causal):
    """64 sequences of 2^29 rows and 8 KV heads: 2^31 tiles and more.  Nothing is written;
    with short lengths the next call over the same workspace is right."""
    dfl = _dfl()
    rng = np.random.default_rng(T)
    B, hkv, d, page = 64, 8, 64, 2 ** 16
    cells = dfl.alloc_kv4_cells(1, hkv, page, d)
    table = torch.full((B, 2 ** 13), -1, dtype=I32, device="cuda")
    view = dfl.KV4View(cells, i32([2 ** 29] * B), 2 ** 29, table, i32([0]), i32([0]), page)
    dims = dfl.make_kv4_dims(B, B * T, T, 4 * hkv, hkv, d)
    ws = dfl.alloc_kv4_workspace(dims)
    q = bf16(rng.normal(size=(B * T, 4 * hkv, d)))
    out = torch.full_like(q, 5.0)
    start = i32(np.arange(B + 1) * T)
    dfl.dflash_kv4_attention(dims, q, start, view, 0.1, causal, out, ws)
    assert status(ws) == bits("capacity")
    assert (f64(out) == 5).all()
    view.seq_len.fill_(T)
    table[:, 0] = 0
    dfl.dflash_kv4_attention(dims, q, start, view, 0.1, causal, out, ws)
    assert status(ws) == 0
    assert (f64(out) == 0).all()                       # (cells of zeros)


@pytest.mark.parametrize("T", [1, 16])
def test_step_with_a_sequence_that_was_not_served(T):
    """The chain after a reservation that ran out of pages: the other sequences' outputs are
    right, no cell of the one left out changes, its norms are skipped, and once it was served its
    step comes out as if nothing had been."""
    dfl = _dfl()
    rng = np.random.default_rng(T)
    hq, hkv, d = 4, 1, 64
    cache = Cache(rng, [32, 16, 30], hkv, d, spare=0)
    view = cache.view
    wide = torch.full((3, 6), -1, dtype=I32, device="cuda")
    wide[:, :view.page_table.shape[1]] = view.page_table
    view.page_table = wide
    lens = [32 - T, 16, 30 - T]                          # the first and last have their pages
    view.seq_len.copy_(i32(lens))
    view.free_count.zero_()
    dims = dfl.make_kv4_dims(3, 3 * T, T, hq, hkv, d)
    ws = dfl.alloc_kv4_workspace(dims)
    start, pos, slot = (torch.zeros(m, dtype=I32, device="cuda") for m in (4, 3 * T, 3 * T))
    q0, k0, v0 = (bf16(rng.normal(size=(3 * T, h, d))) for h in (hq, hkv, hkv))
    before = view.cells.clone()

    def step(q, k):
        out = torch.full_like(q, 9.0)
        dfl.dflash_kv_reserve(dims, view, i32([T] * 3), start, pos, slot, view.seq_len, ws)
        st = status(ws)
        dfl.dflash_qk_norm_rope(dims, q, k, None, None, pos, 1e6, 1e-6, q, k)
        dfl.dflash_kv4_append(dims, k, v0, slot, view, ws)
        dfl.dflash_kv4_attention(dims, q, start, view, 0.125, True, out, ws)
        assert status(ws) == 0
        return st, out

    q, k = q0.clone(), k0.clone()
    st, out = step(q, k)
    assert st == bits("pool_empty")
    assert view.seq_len.tolist() == [32, 16, 30] and pos[T] == -1 and slot[T] == -1
    mid = slice(T, 2 * T)
    assert torch.equal(q[mid], q0[mid]) and torch.equal(k[mid], k0[mid])
    page = int(cache.table[1, 0])
    assert torch.equal(view.cells[page], before[page])
    kd, vd, qd, got = f64(k), f64(v0), f64(q), f64(out)

    def check(b, rows, got, keep):
        kk = np.concatenate([cache.k[b][:keep], O.values(*O.quantise(kd[rows], cache.k_exp),
                                                         cache.k_exp)])
        vv = np.concatenate([cache.v[b][:keep], O.values(*O.quantise(vd[rows], cache.v_exp),
                                                         cache.v_exp)])
        ref, avg, e = O.attention(qd[rows], kk, vv, [keep + t + 1 for t in range(T)], 0.125)
        assert (np.abs(got[rows] - ref) <= bound(ref, avg, e, vv)).all(), b

    for b in (0, 2):
        check(b, slice(b * T, b * T + T), got, lens[b])
    # a page comes free: the crop takes the step back, and all three are served
    dfl.dflash_kv_crop([view.pages()], i32(lens), 3, ws)
    new_page = torch.zeros(1, *view.cells.shape[1:], dtype=U8, device="cuda")
    view.cells = torch.cat([view.cells, new_page])
    view.free_list = torch.cat([view.free_list, i32([0])])
    view.free_list[int(view.free_count)] = len(view.cells) - 1
    view.free_count += 1
    q, k = q0.clone(), k0.clone()
    st, out = step(q, k)
    assert st == 0 and view.seq_len.tolist() == [32, 16 + T, 30]
    kd, qd, got = f64(k), f64(q), f64(out)
    for b in range(3):
        check(b, slice(b * T, b * T + T), got, lens[b])


def test_layers_share_one_reservation():
    """Two layers' cells over one set of lengths and pages: reserved and cropped once a step, as
    the documentation has it, over three steps."""
    dfl = _dfl()
    rng = np.random.default_rng(41)
    B, hq, hkv, d, n_pages = 2, 4, 2, 64, 20
    seq, table, free, count = (i32([0] * B), i32(np.full((B, 8), -1)),
                               i32(rng.permutation(n_pages)), i32([n_pages]))
    views = [dfl.KV4View(dfl.alloc_kv4_cells(n_pages, hkv, 16, d), seq, 128, table, free, count, 16)
             for _ in range(2)]
    K, V = ([[np.zeros((0, hkv, d))] * B for _ in views] for _ in range(2))
    for new, kept in (([20, 5], [20, 5]), ([16, 16], [3, 16]), ([1, 1], [1, 1])):
        T, n = max(new), sum(new)
        dims = dfl.make_kv4_dims(B, n, T, hq, hkv, d)
        ws = dfl.alloc_kv4_workspace(dims)
        start, pos, slot = (torch.zeros(m, dtype=I32, device="cuda") for m in (B + 1, n, n))
        before = seq.clone()
        dfl.dflash_kv_reserve(dims, views[0], i32(new), start, pos, slot, seq, ws)
        for i, view in enumerate(views):
            q, k, v = (bf16(rng.normal(size=(n, h, d))) for h in (hq, hkv, hkv))
            out = torch.zeros_like(q)
            dfl.dflash_qk_norm_rope(dims, q, k, None, None, pos, 1e6, 1e-6, q, k)
            dfl.dflash_kv4_append(dims, k, v, slot, view, ws)
            dfl.dflash_kv4_attention(dims, q, start, view, 0.125, True, out, ws)
            at = 0
            for b, t in enumerate(new):
                rows = slice(at, at + t)
                K[i][b] = np.concatenate([K[i][b], O.values(*O.quantise(f64(k)[rows], [0]), [0])])
                V[i][b] = np.concatenate([V[i][b], O.values(*O.quantise(f64(v)[rows], [0]), [0])])
                L = len(K[i][b])
                ref, avg, e = O.attention(f64(q)[rows], K[i][b], V[i][b],
                                          [L - t + j + 1 for j in range(t)], 0.125)
                assert (np.abs(f64(out)[rows] - ref) <= bound(ref, avg, e, V[i][b])).all(), (i, b)
                K[i][b], V[i][b] = (x[:L - t + kept[b]] for x in (K[i][b], V[i][b]))
                at += t
        dfl.dflash_kv_crop([views[0].pages()], before + i32(kept), B, ws)
        assert status(ws) == 0
        assert seq.tolist() == [len(x) for x in K[0]]
    assert int(count) == n_pages - sum(-(-len(x) // 16) for x in K[0])


@pytest.mark.parametrize("T", [1, 4, 8, 16, 32])
def test_attention_smallest_queries_and_largest_scale(T):
    """Queries of subnormal numbers, the scale near the largest number, gains either way: the
    scores are of size 1, whatever the factors between are."""
    rng = np.random.default_rng(T)
    cache = Cache(rng, [300, 40], 4, 128)
    gain = np.array([0, 12, 1, -2])
    cache.k = [np.ldexp(k, (gain - cache.k_exp)[:, None]) for k in cache.k]
    cache.k_exp = gain
    cache.view.k_exp = i32(cache.k_exp)
    whole = rng.integers(-8, 9, (2 * T, 16, 128))
    whole[:, 4:8] = np.sign(whole[:, 4:8]) * (rng.random((2 * T, 4, 128)) < 2.0 ** -6)
    whole[0, 0] = whole[-1, -1] = 0
    q = bf16(np.ldexp(whole.astype(np.float64), -133))
    assert (f64(q) == np.ldexp(whole.astype(np.float64), -133)).all()
    check_attention(rng, cache, [T, T], 16, True, q=q, scale=2.0 ** 126)


@pytest.mark.parametrize("fine", [False, True])
@pytest.mark.parametrize("T", [1, 4, 8, 16, 32])
def test_attention_small_rows_beside_large_ones(T, fine):
    """Rows of one unit down to 2^-18 of its largest, which lies just above 2^-2 (where queries
    are left as they are), under a scale that gives the small rows scores of a few units.

    A query element is off by at most e = 2^-23 of the unit's largest, so every score of a row by
    at most s = scale sum |k| e, a weight by a factor of exp(+-2 s): added to bound() is
    A (exp(2 s) - 1).  Elements that are multiples of 2^-24 are exact (`fine`): nothing is added."""
    dfl = _dfl()
    rng = np.random.default_rng(T)
    hq, d, lens = 4, 128, [300, 77]
    cache = Cache(rng, lens, 1, d, exps=False)
    q = rng.uniform(0.25, 0.4375, (2 * T, hq, d)) * rng.choice([-1, 1], (2 * T, hq, d))
    small = rng.random((2 * T, hq)) < 0.7
    if fine:
        q[small] = rng.integers(-8, 9, (int(small.sum()), d)) * 2.0 ** -20
    else:
        q[small] *= np.exp2(rng.integers(-16, -11, (int(small.sum()), 1)))
    qt = bf16(q)
    scale = 2.0 ** 14
    dims = dfl.make_kv4_dims(2, 2 * T, T, hq, 1, d)
    ws = dfl.alloc_kv4_workspace(dims)
    out = torch.zeros_like(qt)
    dfl.dflash_kv4_attention(dims, qt, i32([0, T, 2 * T]), cache.view, scale, True, out, ws)
    assert status(ws) == 0
    qd, got = f64(qt), f64(out)
    for b, L in enumerate(lens):
        for t in range(T):
            row, m = b * T + t, L - T + t + 1
            for h in range(hq):
                ref, avg, e = O.attention(qd[row:row + 1, h:h + 1], cache.k[b], cache.v[b], [m],
                                          scale)
                tol = bound(ref, avg, e, cache.v[b])
                if not fine and small[row, h]:
                    s = scale * np.abs(cache.k[b][:m, 0]).sum(-1).max() * 2.0 ** -23 * 0.4375
                    tol = tol + avg * np.expm1(2 * s)
                assert (np.abs(got[row, h] - ref) <= tol).all(), (b, t, h, bool(small[row, h]))


def test_no_bound_on_new_rows():
    """max_tokens 2^31 - 1: every call takes it as no bound."""
    dfl = _dfl()
    rng = np.random.default_rng(51)
    cache = Cache(rng, [40, 300, 2], 2, 64, spare=8, extra_rows=20)
    view, new = cache.view, [20, 1, 7]
    n = sum(new)
    outs = []
    lens = view.seq_len.clone()
    for top in (2 ** 31 - 1, 20):
        dims = dfl.make_kv4_dims(3, n, top, 8, 2, 64)
        ws = dfl.alloc_kv4_workspace(dims)
        start, pos, slot = (torch.zeros(m, dtype=I32, device="cuda") for m in (4, n, n))
        view.seq_len.copy_(lens)
        g = np.random.default_rng(1)
        q, k, v = (bf16(g.normal(size=(n, h, 64))) for h in (8, 2, 2))
        out = torch.zeros_like(q)
        dfl.dflash_kv_reserve(dims, view, i32(new), start, pos, slot, view.seq_len, ws)
        dfl.dflash_qk_norm_rope(dims, q, k, None, None, pos, 1e6, 1e-6, q, k)
        dfl.dflash_kv4_append(dims, k, v, slot, view, ws)
        dfl.dflash_kv4_attention(dims, q, start, view, 0.125, True, out, ws)
        assert status(ws) == 0
        outs.append(out)
    # A unit takes 32 rows or 16: the same sums in other tiles.  Each run is within bound() of the
    # exact value: with A <= V, the largest |v| (a value of 4 bits is at most 1 + 2^-4 of what it stands
    # for, or half a smallest step), and e < 64 (0.125 * 64 dims * |q| |k| of 8 on the average):
    # 2^-8 of the value and V (2^-10 + 2^-20 + 65 * 2^-16) < V 2^-8 for each of the two
    V = max(1.07 * np.abs(f64(v)).max() + 2.0 ** -9, max(np.abs(x).max() for x in cache.v))
    a, b = (f64(x) for x in outs)
    assert (np.abs(a - b) <= 2.0 ** -7 * np.maximum(np.abs(a), np.abs(b)) + 2.0 ** -7 * V).all()


def test_largest_batch():
    """4096 sequences: reserved, appended and attended in one step, from a prompt's rows to none."""
    dfl = _dfl()
    rng = np.random.default_rng(61)
    B, hq, hkv, d, width = 4096, 2, 1, 64, 4
    new = rng.integers(0, 4, B)
    new[[0, 77, B - 1]] = 50, 0, 33
    n = int(new.sum()) + 5
    pages = int((-(-new // 16)).sum()) + 9
    view = dfl.KV4View(dfl.alloc_kv4_cells(pages, hkv, 16, d), i32([0] * B), width * 16,
                       i32(np.full((B, width), -1)), i32(rng.permutation(pages)), i32([pages]), 16)
    dims = dfl.make_kv4_dims(B, n, 50, hq, hkv, d)
    ws = dfl.alloc_kv4_workspace(dims)
    start, pos, slot = (torch.zeros(m, dtype=I32, device="cuda") for m in (B + 1, n, n))
    q, k, v = (bf16(rng.normal(size=(n, h, d))) for h in (hq, hkv, hkv))
    out = torch.full_like(q, 3.0)
    dfl.dflash_kv_reserve(dims, view, i32(new), start, pos, slot, view.seq_len, ws)
    dfl.dflash_kv4_append(dims, k, v, slot, view, ws)
    dfl.dflash_kv4_attention(dims, q, start, view, 0.125, True, out, ws)
    assert status(ws) == 0 and int(view.free_count) == 9
    assert (view.seq_len.cpu().numpy() == new).all()
    at = np.concatenate([[0], np.cumsum(new)])
    assert (start.cpu().numpy() == at).all()
    K, V = (O.values(*O.quantise(f64(x), [0]), [0]) for x in (k, v))
    got, qd = f64(out), f64(q)
    for b in [0, 1, 31, 32, 33, 77, 1000, 2047, 2048, *rng.integers(0, B, 200), B - 2, B - 1]:
        rows = slice(at[b], at[b + 1])
        ref, avg, e = O.attention(qd[rows], K[rows], V[rows], range(1, new[b] + 1), 0.125)
        assert (np.abs(got[rows] - ref) <= bound(ref, avg, e, V[rows])).all(), b
    assert (got[at[-1]:] == 3).all()


@pytest.mark.parametrize("T", [1, 16, 64])
def test_a_batch_without_new_rows(T):
    """Nothing but padding: nothing is taken, written or read."""
    dfl = _dfl()
    rng = np.random.default_rng(T)
    cache = Cache(rng, [40, 0, 17], 1, 64)
    dims = dfl.make_kv4_dims(3, T, T, 4, 1, 64)
    ws = dfl.alloc_kv4_workspace(dims)
    cells, table = cache.view.cells.clone(), cache.view.page_table.clone()
    start, pos, slot = (torch.full((m,), 9, dtype=I32, device="cuda") for m in (4, T, T))
    q, k = (torch.full((T, h, 64), 2.0, dtype=BF, device="cuda") for h in (4, 1))
    out = torch.full_like(q, 5.0)
    dfl.dflash_kv_reserve(dims, cache.view, i32([0, 0, 0]), start, pos, slot, cache.view.seq_len, ws)
    dfl.dflash_qk_norm_rope(dims, q, k, None, None, pos, 1e6, 1e-6, q, k)
    dfl.dflash_kv4_append(dims, k, k, slot, cache.view, ws)
    dfl.dflash_kv4_attention(dims, q, start, cache.view, 0.125, True, out, ws)
    dfl.dflash_kv4_gather(dims, slot, cache.view, k, k.clone(), ws)
    assert status(ws) == 0
    assert start.tolist() == [0] * 4 and pos.tolist() == slot.tolist() == [-1] * T
    assert torch.equal(cache.view.cells, cells) and torch.equal(cache.view.page_table, table)
    assert (out == 5).all() and (q == 2).all() and (k == 2).all()
    assert cache.view.seq_len.tolist() == [40, 0, 17]


def test_shared_pages_and_repeated_slots():
    """Two sequences over the same full pages of a prefix, each going on in pages of its own; rows
    gathered more than once."""
    dfl = _dfl()
    rng = np.random.default_rng(71)
    cache = Cache(rng, [48, 64], 2, 64, spare=6, extra_rows=20)
    view = cache.view
    view.page_table[1, :3] = view.page_table[0, :3]
    view.page_table[1, 3] = -1
    view.seq_len.fill_(48)
    cache.k[1], cache.v[1] = cache.k[0], cache.v[0]
    T, n = 5, 10
    dims = dfl.make_kv4_dims(2, n, T, 8, 2, 64)
    ws = dfl.alloc_kv4_workspace(dims)
    start, pos, slot = (torch.zeros(m, dtype=I32, device="cuda") for m in (3, n, n))
    gain = np.ldexp(1.0, -np.repeat(cache.k_exp, 4))[:, None]
    q = bf16(rng.normal(size=(n, 8, 64)) * gain)
    k, v = (bf16(rng.normal(size=(n, 2, 64)) * np.ldexp(1.0, e)[:, None])
            for e in (cache.k_exp, cache.v_exp))
    out = torch.zeros_like(q)
    dfl.dflash_kv_reserve(dims, view, i32([T, T]), start, pos, slot, view.seq_len, ws)
    dfl.dflash_kv4_append(dims, k, v, slot, view, ws)
    dfl.dflash_kv4_attention(dims, q, start, view, 0.125, True, out, ws)
    assert status(ws) == 0
    kq, vq = (O.values(*O.quantise(f64(x), e), e) for x, e in ((k, cache.k_exp), (v, cache.v_exp)))
    for b in range(2):
        rows = slice(b * T, b * T + T)
        kk, vv = (np.concatenate([x[b], y[rows]]) for x, y in ((cache.k, kq), (cache.v, vq)))
        ref, avg, e = O.attention(f64(q)[rows], kk, vv, range(49, 49 + T), 0.125)
        assert (np.abs(f64(out)[rows] - ref) <= bound(ref, avg, e, vv)).all(), b
    again = slot[torch.tensor([0, 0, 9, 3, 9, 9, 1, 0, 3, 2])].contiguous()
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    dfl.dflash_kv4_gather(dims, again, view, ko, vo, ws)
    pick = [0, 0, 9, 3, 9, 9, 1, 0, 3, 2]
    np.testing.assert_array_equal(f64(ko), kq[pick])
    np.testing.assert_array_equal(f64(vo), vq[pick])


def test_gains_past_their_ends_count_as_the_ends():
    dfl = _dfl()
    rng = np.random.default_rng(81)
    far, near = i32([100, -2 ** 31]), i32([64, -64])
    got = []
    x = bf16(rng.normal(size=(20, 2, 64)) * np.ldexp(1.0, [64, -64])[:, None])
    q = bf16(rng.normal(size=(20, 4, 64)) * np.ldexp(1.0, [-64, -64, 64, 64])[:, None])
    for exp in (far, near):
        view = dfl.KV4View(dfl.alloc_kv4_cells(2, 2, 16, 64), i32([20]), 32, i32([[1, 0]]),
                           i32([0, 0]), i32([0]), 16, exp, exp)
        dims = dfl.make_kv4_dims(1, 20, 20, 4, 2, 64)
        ws = dfl.alloc_kv4_workspace(dims)
        slot = i32([16 + i if i < 16 else i - 16 for i in range(20)])
        dfl.dflash_kv4_append(dims, x, x, slot, view, ws)
        ko, vo, out = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(q)
        dfl.dflash_kv4_gather(dims, slot, view, ko, vo, ws)
        dfl.dflash_kv4_attention(dims, q, i32([0, 20]), view, 0.125, True, out, ws)
        assert status(ws) == 0
        got.append((view.cells, ko, vo, out))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    e = np.array([64, -64])
    ref = O.values(*O.quantise(f64(x), e), e)
    np.testing.assert_array_equal(f64(got[0][1]), ref)
    ref, avg, s = O.attention(f64(q), ref, ref, range(1, 21), 0.125)
    for h in range(4):                                   # (bound() head by head: sizes 2^128 apart)
        tol = bound(ref[:, h], avg[:, h], s, f64(x)[:, h // 2])
        assert (np.abs(f64(got[0][3])[:, h] - ref[:, h]) <= tol).all(), h


@pytest.mark.parametrize("d", [64, 128])
def test_norm_rope_keeps_bad_values_in_their_heads(d):
    """NaN and infinities of one head leave the head beside it in the warp, and other rows, alone;
    a row of zeros stays zero; subnormal and large values are normed like others."""
    dfl = _dfl()
    rng = np.random.default_rng(d)
    n, hq, hkv = 4, 6, 3
    q0, k0 = rng.normal(size=(n, hq, d)), rng.normal(size=(n, hkv, d))
    q0[2, 1], k0[1, 2] = 0, 0
    q0[1, 2] *= 2.0 ** 40
    w = bf16(1 + 0.2 * rng.normal(size=d))
    pos = [5, 0, 70000, 1]
    dims = dfl.make_kv4_dims(1, n, n, hq, hkv, d)
    runs = []
    for bad in (False, True):
        q, k = bf16(q0), bf16(k0)
        if bad:
            q[0, 3, 7], q[3, 0, d - 1], k[2, 0, 0] = float("nan"), float("inf"), float("-inf")
        qo, ko = torch.zeros_like(q), torch.zeros_like(k)
        dfl.dflash_qk_norm_rope(dims, q, k, w, w, i32(pos), 1e6, 1e-6, qo, ko)
        runs.append((qo, ko))
    (qa, ka), (qb, kb) = runs
    for a, b, at in ((qa, qb, [(0, 3), (3, 0)]), (ka, kb, [(2, 0)])):
        for i in at:
            assert torch.isnan(b[i]).any()
            b[i] = a[i]
        assert torch.equal(a, b)
    assert (qa[2, 1] == 0).all() and (ka[1, 2] == 0).all()
    ref = O.norm_rope(f64(bf16(q0)), f64(w), pos, 1e6, 1e-6)
    pair = np.abs(ref) + np.abs(np.roll(ref, d // 2, axis=-1))
    tol = 2.0 ** -8 * np.abs(ref) + pair * (2.0 ** -16 + np.abs(pos)[:, None, None] * 2.0 ** -52)
    assert (np.abs(f64(qa) - ref) <= tol).all()
