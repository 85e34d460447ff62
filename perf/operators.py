"""What is measured of the serving calls over a KV cache held in 4 bits.

Operators: the page reservation with its position and slot maps
(``dflash_kv_reserve``), the per-head norms of queries and keys with the
position rotation (``dflash_qk_norm_rope``), the append of K/V rows in 4 bits
and their read-back (``dflash_kv4_append``, ``dflash_kv4_gather``), and the
attention of ragged query rows over that cache (``dflash_kv4_attention``).

``run`` holds each operator's plain form; with ``own`` set it makes the calls
of this package.

The cache is cut into cells: 16 rows of one KV head, 18 D bytes,
    K codes  [D/32][16 rows][16 bytes]   byte j of a piece: dims 2j (low nibble), 2j + 1
    V codes  [D/2][16 rows]              byte (p, r): dims 2p (low nibble), 2p + 1 of row r
    K scales [16 rows][D/16]             e4m3, one for 16 dims
    V scales [D/16][16 rows]
and an element is 2^exp[head] * scale * code, code in e2m1 (+-{0, .5, 1, 1.5, 2, 3, 4, 6}).
"""
import math

import torch

own = False

PAGE = 16
THETA, EPS = 1.0e6, 1.0e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _reserve(name, batch, new, ctx, pad=0):
    return {"name": name, "op": "reserve", "batch": batch, "new_lo": new[0], "new_hi": new[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "pad": pad}


def _norm(name, tokens, hq, hkv, d, far=0, pad=0):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d,
            "far": far, "pad": pad}


def _append(name, batch, new, ctx, hkv, d):
    return {"name": name, "op": "append", "batch": batch, "new_lo": new[0], "new_hi": new[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "hkv": hkv, "d": d}


def _attn(name, batch, new, ctx, hq, hkv, d, causal):
    return {"name": name, "op": "attention", "batch": batch, "new_lo": new[0], "new_hi": new[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "hq": hq, "hkv": hkv, "d": d, "causal": causal}


def listed():
    return [
        # a batch of blocks about to be verified: 16 new rows for each of 32 sequences
        _reserve("reserve blocks b32", 32, (16, 16), (512, 16384)),
        # prompts of uneven lengths entering next to sequences that only take one token,
        # in a batch padded to a fixed number of rows
        _reserve("reserve mixed b64", 64, (1, 2047), (0, 8192), pad=37),
        # one block of one sequence through one layer
        _norm("norm rope block b1", 16, 32, 8, 128),
        # a long prompt chunk through one layer of the widest configuration, far positions
        _norm("norm rope prompt", 8191, 64, 8, 128, far=100000, pad=1),
        # the blocks of 32 sequences appended in the middle of pages and read back
        _append("append blocks b32", 32, (16, 16), (512, 16384), 8, 128),
        # prompts appended to empty and short caches and read back
        _append("append prompts b8", 8, (301, 4096), (0, 40), 8, 128),
        # one token of one short sequence, the tiny configuration
        _attn("attention tiny token", 1, (1, 1), (128, 128), 4, 2, 64, True),
        # one block over a long context (the drafter's view: no causal mask)
        _attn("attention block 8k b1", 1, (16, 16), (8192, 8192), 32, 8, 128, False),
        # single tokens of a ragged batch
        _attn("attention tokens b32", 32, (1, 1), (512, 16384), 32, 8, 128, True),
        # verification blocks of a ragged batch
        _attn("attention blocks b32", 32, (16, 16), (512, 16384), 32, 8, 128, True),
        # long contexts with eight query heads to a KV head
        _attn("attention blocks 32k b4", 4, (16, 16), (32768, 32768), 64, 8, 128, True),
        # prompt chunks of uneven lengths, some with a context behind them
        _attn("attention chunks b4", 4, (257, 1024), (0, 6000), 32, 8, 128, True),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["reserve", "norm_rope", "append", "attention", "attention", "attention"])
    heads = rng.choice([(32, 8, 128), (64, 8, 128), (4, 2, 64), (16, 8, 128), (8, 8, 64)])
    if op == "reserve":
        new = sorted(_logint(rng, 1, 2048) for _ in range(2))
        ctx = sorted(_logint(rng, 1, 16384) - 1 for _ in range(2))
        c = _reserve("", _logint(rng, 1, 64), new, ctx, rng.choice([0, 0, 13, 64]))
    elif op == "norm_rope":
        c = _norm("", _logint(rng, 1, 8192), *heads, far=_logint(rng, 1, 200000) - 1,
                  pad=rng.choice([0, 3]))
    elif op == "append":
        batch = _logint(rng, 1, 32)
        top = max(16, 16384 // batch)
        new = sorted(_logint(rng, 1, top) for _ in range(2))
        ctx = sorted(_logint(rng, 1, 16384) - 1 for _ in range(2))
        c = _append("", batch, new, ctx, *heads[1:])
    else:
        kind = rng.choice(["token", "block", "block", "any", "chunk"])
        batch = _logint(rng, 1, 32 if kind != "chunk" else 3)
        ctx = sorted(_logint(rng, 1, 16384 if batch > 4 and kind != "chunk" else
                             32768 if kind != "chunk" else 6000) - 1 for _ in range(2))
        new = {"token": [1, 1], "block": [16, 16],
               "any": sorted(rng.randint(1, 24) for _ in range(2)),
               "chunk": sorted(_logint(rng, 25, 1024) for _ in range(2))}[kind]
        if heads[0] == 64 and batch > 8:
            ctx = [x // 4 for x in ctx]
        c = _attn("", batch, new, ctx, *heads, causal=kind == "chunk" or rng.random() < 0.6)
    del c["name"]
    return c


def _spread(lo, hi, n, salt):
    """n lengths from lo to hi, both ends among them, in no order; the case alone fixes them."""
    if n == 1:
        return [hi]
    xs = [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    return [xs[(i * 7919 + salt) % n] if math.gcd(7919, n) == 1 else xs[i] for i in range(n)]


def _lens(case):
    """(context rows, new rows) of each sequence."""
    b = case["batch"]
    return (_spread(case["ctx_lo"], case["ctx_hi"], b, 3),
            _spread(case["new_lo"], case["new_hi"], b, 5))


def work(case):
    if case["op"] == "reserve":
        ctx, new = _lens(case)
        n = sum(new) + case["pad"]
        pages = sum((c + k - 1) // PAGE - c // PAGE + 1 for c, k in zip(ctx, new))
        return {"bytes": 8.0 * n + 4.0 * 4 * len(ctx) + 4.0 * 3 * pages, "flops": 0}
    if case["op"] == "norm_rope":
        row = (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": case["tokens"] * (4.0 * row + 4), "flops": 8.0 * case["tokens"] * row}
    if case["op"] == "append":
        n = sum(_lens(case)[1])
        el = 2 * n * case["hkv"] * case["d"]
        # rows in, cells out; cells in, rows out
        return {"bytes": 2 * (2.0 * el + el * 9 / 16) + 8.0 * n, "flops": 6.0 * el}
    ctx, new = _lens(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    cache = sum(c + k for c, k in zip(ctx, new)) * hkv * d * 2 * 9 / 16
    seen = sum(k * c + (k * (k + 1) // 2 if case["causal"] else k * k) for c, k in zip(ctx, new))
    return {"bytes": cache + 4.0 * sum(new) * hq * d, "flops": 4.0 * seen * hq * d}


# ---------------------------------------------------------------------------
# the 4-bit form, as tensors
# ---------------------------------------------------------------------------
def _codes(x, exp):
    """x [..., h, D] (fp32) and exp [h]: (nibbles [..., h, D], scales [..., h, D/16]).

    Every product and comparison here is exact in 32 bits for bf16 x."""
    x = torch.ldexp(x, -exp[:, None]).unflatten(-1, (-1, 16))
    a = x.abs()
    s = (a.amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()
    # nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; halfway cases go to the even code
    c = ((a > 0.25 * f).to(torch.uint8) + (a >= 0.75 * f) + (a > 1.25 * f) + (a >= 1.75 * f)
         + (a > 2.5 * f) + (a >= 3.5 * f) + (a > 5.0 * f))
    c = torch.where(f > 0, c, torch.zeros_like(c)) + 8 * (x < 0).to(torch.uint8)
    return c.flatten(-2), s.squeeze(-1)


def _grid(device):
    return torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6., -0., -.5, -1., -1.5, -2., -3., -4., -6.],
                        device=device)


def _values(nibbles, scales, exp):
    """The fp32 values that nibbles [..., h, D] with scales [..., h, D/16] stand for."""
    v = _grid(nibbles.device)[nibbles.int()].unflatten(-1, (-1, 16)) * scales.float()[..., None]
    return torch.ldexp(v.flatten(-2), exp[:, None])


def _cells(kn, ks, vn, vs):
    """Cells [n, h, 18 D] from nibbles [n, 16, h, D] and scales [n, 16, h, D/16]."""
    n, _, h, d = kn.shape

    def pairs(x):                                    # [n, 16, h, D/2] bytes
        return x[..., 0::2] | (x[..., 1::2] << 4)

    k = pairs(kn).view(n, 16, h, d // 32, 16).permute(0, 2, 3, 1, 4).reshape(n, h, -1)
    v = pairs(vn).permute(0, 2, 3, 1).reshape(n, h, -1)
    ks = ks.view(torch.uint8).permute(0, 2, 1, 3).reshape(n, h, -1)
    vs = vs.view(torch.uint8).permute(0, 2, 3, 1).reshape(n, h, -1)
    return torch.cat([k, v, ks, vs], dim=-1)


def _uncells(cells, d):
    """K and V nibbles [..., h, 16, D] and scales [..., h, 16, D/16] of cells [..., h, 18 D]."""
    k, v, ks, vs = cells.split([8 * d, 8 * d, d, d], dim=-1)
    k = k.unflatten(-1, (d // 32, 16, 16)).transpose(-3, -2).flatten(-2)
    v = v.unflatten(-1, (d // 2, 16)).transpose(-2, -1)
    ks = ks.unflatten(-1, (16, d // 16))
    vs = vs.unflatten(-1, (d // 16, 16)).transpose(-2, -1).contiguous()

    def nib(x):
        return torch.stack([x & 15, x >> 4], dim=-1).flatten(-2)

    return nib(k), ks.view(torch.float8_e4m3fn), nib(v), vs.view(torch.float8_e4m3fn)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _paged(g, ctx, new, spare):
    """Shuffled pages: (table of the context's pages [B, P], free list, free count)."""
    per = [-(-c // PAGE) for c in ctx]
    width = max(-(-(c + k) // PAGE) for c, k in zip(ctx, new))
    grow = sum(-(-(c + k) // PAGE) - p for c, k, p in zip(ctx, new, per))
    n_pages = sum(per) + grow + spare
    order = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32)
    p = torch.arange(width, device="cuda")[None, :]
    held = _i32(per)[:, None]
    rank = (held.cumsum(0) - held) + p
    table = torch.where(p < held, order[rank.clamp(max=n_pages - 1).long()], -1).int()
    free = torch.cat([order[sum(per):], order[:sum(per)]]).contiguous()
    return table.contiguous(), free, n_pages - sum(per), n_pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    s = {"case": case}
    if case["op"] == "norm_rope":
        n, hq, hkv, d = case["tokens"] + case["pad"], case["hq"], case["hkv"], case["d"]
        s["qkv"] = normal(n, (hq + 2 * hkv) * d)            # the fused projection's rows
        s["q"] = s["qkv"][:, :hq * d].unflatten(1, (hq, d))
        s["k"] = s["qkv"][:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        s["q_w"] = 1 + 0.1 * normal(d)
        s["k_w"] = 1 + 0.1 * normal(d)
        start = torch.randint(0, case["far"] + 1, (1,), generator=g, device="cuda")
        pos = (start + torch.arange(n, device="cuda")).int()
        s["pos"] = torch.where(torch.arange(n, device="cuda") < case["tokens"], pos, -1)
        s["q_out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros(n, hkv, d, dtype=torch.bfloat16, device="cuda")
        if own:
            import block_diffusion_speculative_02_gb300 as dfl
            s["dims"] = dfl.make_kv4_dims(1, n, n, hq, hkv, d)
        return s

    ctx, new = _lens(case)
    b, n = len(ctx), sum(new) + case.get("pad", 0)
    s["n_new"] = _i32(new)
    s["start"] = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
    if case["op"] == "reserve":
        table, free, count, n_pages = _paged(g, ctx, new, 64)
        # the free count and the page table in one buffer, so that one copy sets both back
        s["pool0"] = torch.cat([_i32([count, 0, 0, 0]), table.flatten()])
        s["pool"] = s["pool0"].clone()
        s["free_count"], s["table"] = s["pool"][:1], s["pool"][4:].view(table.shape)
        s["free"], s["seq_len"] = free, _i32(ctx)
        for name, size in (("pos", n), ("slot", n), ("new_len", b)):
            s[name] = torch.zeros(size, dtype=torch.int32, device="cuda")
        if own:
            import block_diffusion_speculative_02_gb300 as dfl
            s["dims"] = dfl.make_kv4_dims(b, n, max(new), 1, 1, 128)
            s["ws"] = dfl.alloc_kv4_workspace(s["dims"])
            s["view"] = dfl.KVView(None, None, s["seq_len"], table.shape[1] * PAGE, s["table"],
                                   free, s["free_count"], PAGE)
        return s

    hkv, d = case["hkv"], case["d"]
    total = [c + k for c, k in zip(ctx, new)]
    table, free, count, n_pages = _paged(g, total, [0] * b, 8)
    s["table"] = table
    s["k_exp"] = torch.randint(-2, 2, (hkv,), generator=g, device="cuda", dtype=torch.int32)
    s["v_exp"] = torch.randint(-6, -2, (hkv,), generator=g, device="cuda", dtype=torch.int32)
    seq_len = _i32(total)
    if case["op"] == "append":
        s["k"], s["v"] = normal(n, hkv, d), normal(n, hkv, d)
        s["k"] = torch.ldexp(s["k"], s["k_exp"][:, None])
        s["v"] = torch.ldexp(s["v"], s["v_exp"][:, None])
        s["cells"] = torch.zeros(n_pages, hkv, 1, 18 * d, dtype=torch.uint8, device="cuda")
        seq = torch.repeat_interleave(torch.arange(b, device="cuda"), s["n_new"])
        first = s["n_new"].cumsum(0) - s["n_new"]
        pos = torch.arange(n, device="cuda") - first[seq] + _i32(ctx)[seq]
        s["slot"] = (table[seq, pos // PAGE] * PAGE + pos % PAGE).int()
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        hq = hkv
    else:
        hq = case["hq"]
        s["start"][1:] = s["n_new"].cumsum(0)
        s["seq_len"] = seq_len
        zero = torch.zeros(hkv, dtype=torch.int32, device="cuda")
        s["cells"] = torch.empty(n_pages, hkv, 1, 18 * d, dtype=torch.uint8, device="cuda")
        for at in range(0, n_pages, 16384):
            m = min(16384, n_pages - at)
            s["cells"][at:at + m, :, 0] = _cells(*_codes(normal(m, 16, hkv, d).float(), zero),
                                                 *_codes(normal(m, 16, hkv, d).float(), zero))
        s["q"] = torch.ldexp(normal(n, hq, d), -s["k_exp"].repeat_interleave(hq // hkv)[:, None])
        s["out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
        s["scale"] = 1 / math.sqrt(d)
    if own:
        import block_diffusion_speculative_02_gb300 as dfl
        s["dims"] = dfl.make_kv4_dims(b, n, max(new), hq, hkv, d)
        s["ws"] = dfl.alloc_kv4_workspace(s["dims"])
        s["view"] = dfl.KV4View(s["cells"], seq_len, table.shape[1] * PAGE, table, free,
                                _i32([count]), PAGE, s["k_exp"], s["v_exp"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import block_diffusion_speculative_02_gb300 as dfl
        if op == "reserve":
            s["pool"].copy_(s["pool0"])
            dfl.dflash_kv_reserve(s["dims"], s["view"], s["n_new"], s["start"], s["pos"],
                                  s["slot"], s["new_len"], s["ws"])
            return [s[x] for x in ("table", "free_count", "start", "pos", "slot", "new_len")]
        if op == "norm_rope":
            dfl.dflash_qk_norm_rope(s["dims"], s["q"], s["k"], s["q_w"], s["k_w"], s["pos"],
                                    THETA, EPS, s["q_out"], s["k_out"])
            return [s["q_out"], s["k_out"]]
        if op == "append":
            dfl.dflash_kv4_append(s["dims"], s["k"], s["v"], s["slot"], s["view"], s["ws"])
            dfl.dflash_kv4_gather(s["dims"], s["slot"], s["view"], s["k_out"], s["v_out"], s["ws"])
            return [s["k_out"], s["v_out"]]
        dfl.dflash_kv4_attention(s["dims"], s["q"], s["start"], s["view"], s["scale"],
                                 s["case"]["causal"], s["out"], s["ws"])
        return [s["out"]]
    return {"reserve": _plain_reserve, "norm_rope": _plain_norm_rope, "append": _plain_append,
            "attention": _plain_attention}[op](s)


def _plain_reserve(s):
    s["pool"].copy_(s["pool0"])
    table, length, new = s["table"], s["seq_len"], s["n_new"]
    s["start"][1:] = new.cumsum(0)
    p = torch.arange(table.shape[1], device="cuda")[None, :]
    last = (length + new - 1)[:, None] // PAGE
    missing = (p >= (length // PAGE)[:, None]) & (p <= last) & (table < 0) & (new > 0)[:, None]
    rank = missing.flatten().cumsum(0).view(table.shape)        # 1, 2, ... in order
    take = s["free"][(s["free_count"] - rank).clamp(min=0).long()]
    table.copy_(torch.where(missing, take, table))
    s["free_count"].sub_(missing.sum())
    i = torch.arange(s["pos"].numel(), device="cuda")
    seq = torch.searchsorted(s["start"][1:], i, right=True)
    live = seq < new.numel()
    seq = seq.clamp(max=new.numel() - 1)
    pos = length[seq] + i - s["start"][seq]
    page = table[seq, (pos // PAGE).clamp(min=0, max=table.shape[1] - 1)]
    s["pos"].copy_(torch.where(live, pos, -1))
    s["slot"].copy_(torch.where(live, page * PAGE + pos % PAGE, -1))
    s["new_len"].copy_(length + new)
    return [s[x] for x in ("table", "free_count", "start", "pos", "slot", "new_len")]


def _plain_norm_rope(s):
    d = s["case"]["d"]
    pos = s["pos"]
    freq = THETA ** (torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / -d)
    angle = pos[:, None].double() * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, w, out):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        a, b = x[..., :d // 2], x[..., d // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1).to(torch.bfloat16)
        out.copy_(torch.where((pos >= 0)[:, None, None], y, out))   # rows behind the batch stay
        return out

    return [one(s["q"], s["q_w"], s["q_out"]), one(s["k"], s["k_w"], s["k_out"])]


def _plain_append(s):
    d = s["case"]["d"]
    kn, ks = _codes(s["k"].float(), s["k_exp"])
    vn, vs = _codes(s["v"].float(), s["v_exp"])
    slot = s["slot"].long()
    page, r = slot // PAGE, slot % PAGE
    k, v, k_s, v_s = s["cells"].squeeze(2).split([8 * d, 8 * d, d, d], dim=-1)
    pairs = kn[..., 0::2] | (kn[..., 1::2] << 4)
    k.unflatten(-1, (d // 32, 16, 16))[page, :, :, r] = pairs.unflatten(-1, (d // 32, 16))
    v.unflatten(-1, (d // 2, 16))[page, :, :, r] = vn[..., 0::2] | (vn[..., 1::2] << 4)
    k_s.unflatten(-1, (16, d // 16))[page, :, r] = ks.view(torch.uint8)
    v_s.unflatten(-1, (d // 16, 16))[page, :, :, r] = vs.view(torch.uint8)
    # back from the cells
    kn, ks, vn, vs = _uncells(s["cells"].squeeze(2)[page], d)
    i = torch.arange(len(slot), device="cuda")
    return [_values(kn[i, :, r], ks[i, :, r], s["k_exp"]).to(torch.bfloat16),
            _values(vn[i, :, r], vs[i, :, r], s["v_exp"]).to(torch.bfloat16)]


def _plain_attention(s):
    c = s["case"]
    hkv, d, t = c["hkv"], c["d"], c["new_hi"]
    group = c["hq"] // hkv
    b = s["n_new"].numel()
    length, new = s["seq_len"], s["n_new"]
    cells = s["cells"].squeeze(2)[s["table"].clamp(min=0).long()]       # [B, P, h, 18 D]
    kn, ks, vn, vs = _uncells(cells, d)

    def rows(n, sc, exp):                                               # [B, h, P * 16, D]
        return _values(n.transpose(-3, -2), sc.transpose(-3, -2), exp).permute(
            0, 3, 1, 2, 4).flatten(2, 3)

    k, v = rows(kn, ks, s["k_exp"]), rows(vn, vs, s["v_exp"])
    i = torch.arange(t, device="cuda")
    row = s["start"][:-1, None] + i                                     # [B, T]
    live = i < new[:, None]
    q = s["q"].float()[row.clamp(max=s["q"].shape[0] - 1).long()]       # [B, T, Hq, D]
    q = q.unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]                 # [B, h, G * T, keys]
    seen = (length - new)[:, None] + i + 1 if c["causal"] else length[:, None] + 0 * i
    seen = torch.minimum(seen, length[:, None]).repeat(1, group)[:, None, :, None]
    mask = torch.arange(k.shape[2], device="cuda") < seen
    x = torch.where(mask, x, -torch.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    v = torch.where((torch.arange(k.shape[2], device="cuda") < length[:, None])[:, None, :, None],
                    v, 0.0)
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    o = o.unflatten(2, (group, t)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, T, Hq, D]
    s["out"][row[live].long()] = o[live].to(torch.bfloat16)
    return [s["out"]]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e2m1_64(n):
    """Values of 4-bit codes from their fields: sign, two bits of exponent, one of mantissa."""
    e, m = ((n >> 1) & 3).double(), (n & 1).double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    return torch.where(n >= 8, -mag, mag)


def _e4m3_64(x):
    e, m = (x >> 3).double(), (x & 7).double()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)


def _fake4_64(x, exp):
    """x [..., h, D] in 64 bits, rounded to 4 bits and back."""
    x = x.double() * torch.exp2(-exp.double())[:, None]
    g = x.reshape(*x.shape[:-1], -1, 16)
    m = (g.abs().amax(-1) / 6).clamp(max=448)
    e = torch.floor(torch.log2(m.clamp(min=2.0 ** -6))).clamp(min=-6)
    q = torch.exp2(e - 3)
    scale = (torch.round(m / q) * q)[..., None]                        # ties to even
    y = (g.abs() / torch.where(scale > 0, scale, 1.0)).clamp(max=6)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    y = torch.round(y / step) * step
    y = torch.where(scale > 0, y * scale, 0.0) * torch.sign(g)
    return y.reshape(x.shape) * torch.exp2(exp.double())[:, None]


def _rows_64(s, b, n, part):
    """K (part 0) or V (part 1) of the first n rows of sequence b: [h, n, D] in 64 bits."""
    d, pages = s["case"]["d"], -(-n // PAGE)
    c = s["cells"][s["table"][b, :pages].long(), :, 0].long()          # [P, h, 18 D]
    h = c.shape[1]
    if part == 0:
        code = c[..., :8 * d].reshape(pages, h, d // 32, 16, 16).permute(1, 0, 3, 2, 4)
        scale = c[..., 16 * d:17 * d].reshape(pages, h, 16, d // 16).permute(1, 0, 2, 3)
        exp = s["k_exp"]
    else:
        code = c[..., 8 * d:16 * d].reshape(pages, h, d // 2, 16).permute(1, 0, 3, 2)
        scale = c[..., 17 * d:].reshape(pages, h, d // 16, 16).permute(1, 0, 3, 2)
        exp = s["v_exp"]
    code = code.reshape(h, pages * 16, d // 2)
    x = torch.empty(h, pages * 16, d, dtype=torch.float64, device="cuda")
    x[..., 0::2], x[..., 1::2] = _e2m1_64(code % 16), _e2m1_64(code // 16)
    x *= _e4m3_64(scale.reshape(h, pages * 16, d // 16)).repeat_interleave(16, dim=-1)
    return (x * torch.exp2(exp.double())[:, None, None])[:, :n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "reserve":
        return None                                     # whole numbers
    if case["op"] == "append":
        return [_fake4_64(s["k"], s["k_exp"]), _fake4_64(s["v"], s["v_exp"])]
    if case["op"] == "norm_rope":
        half = case["d"] // 2
        inv = torch.tensor([THETA ** (-i / half) for i in range(half)], dtype=torch.float64,
                           device="cuda")
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * inv)[:, None]
        out = []
        for x, w in ((s["q"], s["q_w"]), (s["k"], s["k_w"])):
            x = x.double()
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + EPS) * w.double()
            z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
            y = torch.cat([z.real, z.imag], dim=-1)
            y[s["pos"] < 0] = 0
            out.append(y)
        return out
    ctx, new = _lens(case)
    group = case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (c, t) in enumerate(zip(ctx, new)):
        n = c + t
        k, v = _rows_64(s, b, n, 0), _rows_64(s, b, n, 1)
        for lo in range(0, t, 256):
            hi = min(t, lo + 256)
            q = s["q"][at + lo:at + hi].double().transpose(0, 1)       # [Hq, T, D]
            x = (q @ k.repeat_interleave(group, dim=0).transpose(1, 2)) / math.sqrt(case["d"])
            if case["causal"]:
                key = torch.arange(n, device="cuda")
                last = c + torch.arange(lo, hi, device="cuda")
                x = x.masked_fill(key[None, :] > last[:, None], -math.inf)
            p = torch.softmax(x, dim=-1)
            out[at + lo:at + hi] = (p @ v.repeat_interleave(group, dim=0)).transpose(0, 1)
        at += t
    return [out]
