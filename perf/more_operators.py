"""What is measured of the linear layers in 8-bit floating point (e4m3, a scale for each block of 128).

Operators: the residual's addition with the RMS norm and the rounding of rows to
8 bits (``dflash_fp8_norm_rows``), the gated activation with the same rounding
(``dflash_fp8_silu_mul``), the rounding of weights (``dflash_fp8_weight``), the
product of rows and weights (``dflash_fp8_linear``), and such products grouped by
expert with ragged numbers of rows (``dflash_fp8_grouped``).

``run`` holds each operator's plain form; with ``own`` set it makes the calls
of this package.

Rows x [M, K] have a scale for each 128 columns, kept as [K/128, M]; weights
w [N, K] one for each block of 128 x 128, [N/128, K/128].  The last blocks may
be short.  An element is scale * code.
"""
import math
import random

import torch

own = False

EPS = 1.0e-6
TINY = 2.0 ** -117          # the least largest magnitude that a scale is made of


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, rows, cols, residual, norm):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "residual": residual,
            "norm": norm}


def _silu(name, rows, cols):
    return {"name": name, "op": "silu", "rows": rows, "cols": cols}


def _weight(name, groups, n, k):
    return {"name": name, "op": "weight", "groups": groups, "n": n, "k": k}


def _linear(name, rows, n, k):
    return {"name": name, "op": "linear", "rows": rows, "n": n, "k": k}


def _grouped(name, experts, tokens, top, n, k, gather, skew=0.5, pad=0):
    return {"name": name, "op": "grouped", "experts": experts, "tokens": tokens, "top": top,
            "n": n, "k": k, "gather": gather, "skew": skew, "pad": pad}


def listed():
    return [
        # one verified block of one sequence entering a layer
        _norm("norm block b1", 16, 4096, True, True),
        # a prompt chunk of the widest configuration
        _norm("norm prompt", 8191, 5120, True, True),
        # the MLP's activation for one block, and for a prompt
        _silu("silu block b1", 16, 12288),
        _silu("silu prompt", 8191, 12288),
        # weights laid out at load time: one matrix, odd number of rows, and a layer's experts
        _weight("weight", 1, 2567, 2560),
        _weight("weight experts", 64, 1536, 2048),
        # the attention's output projection for one block of one sequence
        _linear("linear block b1", 16, 4096, 4096),
        # gate and up projections of 32 verified blocks
        _linear("linear blocks b32", 512, 24576, 4096),
        # gate and up projections of a prompt chunk
        _linear("linear prompt", 8191, 24576, 4096),
        # one block of 16 tokens through experts of which each token takes eight
        _grouped("grouped block b1", 128, 16, 8, 1536, 2048, True),
        # 32 blocks: some 32 rows to an expert, some with none
        _grouped("grouped blocks b32", 128, 512, 8, 1536, 2048, True, pad=5),
        # the second product of a prompt, rows in the experts' order already
        _grouped("grouped prompt", 64, 4096, 8, 2048, 1408, False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cols(rng, lo, hi):
    """A number of columns: a multiple of 16, mostly of 128."""
    c = _logint(rng, lo, hi)
    return max(128, c // 128 * 128) if rng.random() < 0.6 else max(16, c // 16 * 16)


def draw(rng):
    op = rng.choice(["norm", "silu", "weight", "linear", "linear", "linear", "grouped", "grouped"])
    if op == "norm":
        c = _norm("", _logint(rng, 1, 8192), _cols(rng, 256, 5120), rng.random() < 0.6,
                  rng.random() < 0.7)
    elif op == "silu":
        c = _silu("", _logint(rng, 1, 8192), _cols(rng, 256, 12288))
    elif op == "weight":
        c = _weight("", _logint(rng, 1, 16), _logint(rng, 64, 8192), _cols(rng, 256, 1408))
    elif op == "linear":
        rows = _logint(rng, 1, 64) if rng.random() < 0.4 else _logint(rng, 1, 8191)
        c = _linear("", rows, _logint(rng, 128, 24576), _cols(rng, 256, 4096))
    else:
        top = rng.choice([1, 2, 4, 8])
        c = _grouped("", _logint(rng, 2, 128), _logint(rng, 1, 2048), top, _logint(rng, 128, 2048),
                     _cols(rng, 256, 2048), rng.random() < 0.6, rng.choice([0.0, 0.5, 1.5]),
                     rng.choice([0, 0, 7]))
    del c["name"]
    return c


def _counts(case):
    """Rows of each expert: uneven, some without any; the case alone fixes them."""
    e, n = case["experts"], case["tokens"] * case["top"]
    rng = random.Random("%d %d %s" % (e, n, case["skew"]))
    share = [rng.random() ** 2 / (i + 1) ** case["skew"] for i in range(e)]
    rng.shuffle(share)
    counts = [0] * e
    for x in rng.choices(range(e), share, k=n):
        counts[x] += 1
    return counts


def _up(x, n):
    return -(-x // n)


def work(case):
    if case["op"] == "norm":
        m, k = case["rows"], case["cols"]
        return {"bytes": m * k * (7.0 if case["residual"] else 3.0) + 4.0 * m * _up(k, 128),
                "flops": 6.0 * m * k}
    if case["op"] == "silu":
        m, k = case["rows"], case["cols"]
        return {"bytes": 5.0 * m * k + 4.0 * m * _up(k, 128), "flops": 8.0 * m * k}
    if case["op"] == "weight":
        g, n, k = case["groups"], case["n"], case["k"]
        return {"bytes": 3.0 * g * n * k + 4.0 * g * _up(n, 128) * _up(k, 128),
                "flops": 3.0 * g * n * k}
    n, k = case["n"], case["k"]
    weight = n * k + 4.0 * _up(n, 128) * _up(k, 128)
    row = k + 4.0 * _up(k, 128)
    if case["op"] == "linear":
        m = case["rows"]
        return {"bytes": weight + m * row + 2.0 * m * n, "flops": 2.0 * m * n * k}
    m = case["tokens"] * case["top"]
    hit = sum(c > 0 for c in _counts(case))
    return {"bytes": hit * weight + (case["tokens"] if case["gather"] else m) * row + 2.0 * m * n,
            "flops": 2.0 * m * n * k}


# ---------------------------------------------------------------------------
# the 8-bit form
# ---------------------------------------------------------------------------
def _blocks(x, dim):
    """Dimension ``dim`` cut into blocks of 128, the last one filled up with zeros."""
    n = x.shape[dim]
    pad = [0, 0] * (x.dim() - 1 - dim) + [0, -n % 128]
    return torch.nn.functional.pad(x, pad).unflatten(dim, (-1, 128))


def _round_rows(h):
    """h [M, K] fp32: e4m3 codes and the scales [K/128, M]."""
    a = _blocks(h.abs(), 1).amax(-1).clamp(min=TINY)                    # [M, K/128]
    q = h * (448.0 / a).repeat_interleave(128, dim=1)[:, :h.shape[1]]
    return q.to(torch.float8_e4m3fn), (a / 448.0).t().contiguous()


def _round_weight(w):
    """w [G, N, K]: e4m3 codes and the scales [G, N/128, K/128]."""
    w = w.float()
    a = _blocks(_blocks(w.abs(), 1), 3).amax((2, 4)).clamp(min=TINY)    # [G, N/128, K/128]
    r = (448.0 / a).repeat_interleave(128, dim=1)[:, :w.shape[1]]
    q = w * r.repeat_interleave(128, dim=2)[:, :, :w.shape[2]]
    return q.to(torch.float8_e4m3fn), a / 448.0


def _rows_value(q, scale):
    return q.float() * scale.t().repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _weight_value(q, scale):
    s = scale.repeat_interleave(128, dim=-2)[..., :q.shape[-2], :]
    return q.float() * s.repeat_interleave(128, dim=-1)[..., :q.shape[-1]]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    bf = torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def hidden(m, k):
        """Rows of a layer's input: some columns far larger than the others."""
        big = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        return (normal(m, k) * big).to(bf)

    def codes(m, k):
        return (torch.empty(m, k, dtype=torch.float8_e4m3fn, device="cuda"),
                torch.empty(_up(k, 128), m, device="cuda"))

    s = {"case": case}
    if case["op"] == "norm":
        m, k = case["rows"], case["cols"]
        s["x"] = hidden(m, k)
        s["residual"] = hidden(m, k) if case["residual"] else None
        s["norm_w"] = (1 + 0.1 * normal(k)).to(bf) if case["norm"] else None
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["q"], s["scale"] = codes(m, k)
        return s
    if case["op"] == "silu":
        m, k = case["rows"], case["cols"]
        s["x"] = (2 * normal(m, 2 * k)).to(bf)              # gate, then up
        s["q"], s["scale"] = codes(m, k)
        return s
    n, k = case["n"], case["k"]
    groups = case.get("groups", case.get("experts", 1))
    w = (0.02 * normal(groups, n, k)).to(bf)
    if case["op"] == "weight":
        s["w"] = w
        s["q"] = torch.empty(groups, n, k, dtype=torch.float8_e4m3fn, device="cuda")
        s["scale"] = torch.empty(groups, _up(n, 128), _up(k, 128), device="cuda")
        return s
    s["w"], s["w_scale"] = _round_weight(w)
    del w
    if case["op"] == "linear":
        m = rows = case["rows"]
        s["w"], s["w_scale"] = s["w"][0], s["w_scale"][0]
    else:
        m = case["tokens"] * case["top"]
        rows = case["tokens"] if case["gather"] else m
        counts = _counts(case)
        s["most"] = max(counts)
        start = torch.tensor([0] + counts, dtype=torch.int32, device="cuda")
        s["start"] = start.cumsum(0).int()
        m += case["pad"]
        s["rows"] = None
        if case["gather"]:
            s["rows"] = torch.randint(0, rows, (m,), generator=g, device="cuda",
                                      dtype=torch.int32)
        else:
            rows = m
    s["x"], s["x_scale"] = _round_rows(hidden(rows, k).float())
    s["out"] = torch.zeros(m, n, dtype=bf, device="cuda")
    if own:
        import block_diffusion_speculative_02_gb300 as dfl
        s["ws"] = dfl.alloc_fp8_workspace()
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import block_diffusion_speculative_02_gb300 as dfl
        if op == "norm":
            dfl.dflash_fp8_norm_rows(s["x"], s["residual"], s["norm_w"], EPS, s["sum"], s["q"],
                                     s["scale"])
            return [s["sum"], s["q"], s["scale"]]
        if op == "silu":
            dfl.dflash_fp8_silu_mul(s["x"], s["q"], s["scale"])
            return [s["q"], s["scale"]]
        if op == "weight":
            dfl.dflash_fp8_weight(s["w"], s["q"], s["scale"])
            return [s["q"], s["scale"]]
        if op == "linear":
            dfl.dflash_fp8_linear(s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"], s["ws"])
            return [s["out"]]
        dfl.dflash_fp8_grouped(s["x"], s["x_scale"], s["w"], s["w_scale"], s["start"], s["rows"],
                               s["out"], s["ws"])
        return [s["out"]]
    return {"norm": _plain_norm, "silu": _plain_silu, "weight": _plain_weight,
            "linear": _plain_linear, "grouped": _plain_grouped}[op](s)


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
        s["sum"].copy_(h)
    if s["norm_w"] is not None:
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["norm_w"].float()
    return [s["sum"], *_round_rows(h)]


def _plain_silu(s):
    gate, up = s["x"].float().chunk(2, dim=1)
    return list(_round_rows(gate / (1 + torch.exp(-gate)) * up))


def _plain_weight(s):
    return list(_round_weight(s["w"]))


def _plain_linear(s):
    y = _rows_value(s["x"], s["x_scale"]) @ _weight_value(s["w"], s["w_scale"]).t()
    s["out"].copy_(y)
    return [s["out"]]


def _plain_grouped(s):
    first, last = s["start"][:-1, None], s["start"][1:, None]
    i = first + torch.arange(s["most"], device="cuda")                  # [E, most]
    live = i < last
    i = torch.where(live, i, 0).long()
    src = i if s["rows"] is None else s["rows"][i].long()
    x = _rows_value(s["x"], s["x_scale"])[src]                          # [E, most, K]
    y = torch.bmm(x, _weight_value(s["w"], s["w_scale"]).transpose(1, 2))
    s["out"][i[live]] = y[live].to(torch.bfloat16)                      # rows behind them stay
    return [s["out"]]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _ratio_64(h):
    """h [M, K] over its scales, not rounded, and the scales [K/128, M]."""
    q, scale = torch.empty_like(h), []
    for lo in range(0, h.shape[1], 128):
        part = h[:, lo:lo + 128]
        scale.append(part.abs().max(dim=1).values.clamp(min=TINY) / 448)
        q[:, lo:lo + 128] = part / scale[-1][:, None]
    return q, torch.stack(scale)


def _decode_64(q):
    """Values of e4m3 codes from their fields."""
    b = q.view(torch.uint8).long()
    e, m = ((b >> 3) & 15).double(), (b & 7).double()
    v = torch.where(e > 0, (8 + m) * torch.exp2(e - 10), m * 2.0 ** -9)
    return torch.where(b >= 128, -v, v)


def _product_64(x, x_scale, w, w_scale):
    """[M, N] in 64 bits, block by block along K."""
    n, k = w.shape
    out = torch.zeros(x.shape[0], n, dtype=torch.float64, device="cuda")
    by_n = torch.arange(n, device="cuda") // 128
    for b, lo in enumerate(range(0, k, 1024)):
        hi = min(k, lo + 1024)
        col = torch.arange(lo, hi, device="cuda") // 128
        a = _decode_64(x[:, lo:hi]) * x_scale.double()[col].t()
        out += a @ (_decode_64(w[:, lo:hi]) * w_scale.double()[by_n][:, col]).t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        total = None
        if s["residual"] is not None:
            h = total = h + s["residual"].double()
        if s["norm_w"] is not None:
            h = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["cols"] + EPS)
            h = h * s["norm_w"].double()
        return [total, *_ratio_64(h)]
    if case["op"] == "silu":
        x, k = s["x"].double(), case["cols"]
        return list(_ratio_64(x[:, :k] * torch.sigmoid(x[:, :k]) * x[:, k:]))
    if case["op"] == "weight":
        q = torch.empty(s["w"].shape, dtype=torch.float64, device="cuda")
        scale = torch.empty(s["scale"].shape, dtype=torch.float64, device="cuda")
        for g in range(case["groups"]):
            for j, lo in enumerate(range(0, case["n"], 128)):
                part = s["w"][g, lo:lo + 128].double()
                most = part.abs().max(dim=0, keepdim=True).values
                _, c = _ratio_64(most)
                scale[g, j] = c[:, 0]
                q[g, lo:lo + 128] = part / c[:, 0].repeat_interleave(128)[:case["k"]]
        return [q, scale]
    if case["op"] == "linear":
        return [_product_64(s["x"], s["x_scale"], s["w"], s["w_scale"])]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for e, c in enumerate(_counts(case)):
        if c:
            src = torch.arange(at, at + c, device="cuda")
            src = src if s["rows"] is None else s["rows"][at:at + c].long()
            out[at:at + c] = _product_64(s["x"].view(torch.uint8)[src], s["x_scale"][:, src],
                                         s["w"][e], s["w_scale"][e])
        at += c
    return [out]
