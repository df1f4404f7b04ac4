"""Cases and plain forms of the operators in 8-bit floating point.

A layer's products with e4m3 operands and a scale for each block of 128:
``norm`` is the RMSNorm with the residual's addition and an 8-bit output,
``quant`` brings rows (through an index, as the experts' order needs it) and
``weights`` whole matrices into the format, ``gemm`` is the product with the
epilogues of a layer, ``grouped`` the same by expert over ragged groups of rows.

``own = False`` computes each in elementary torch operations; ``own = True``
calls the library.

The format: rows hold one fp32 scale for each 128 columns, laid out [column
block, row]; weights one for each 128 x 128 block, [row block, column block].  A
value is its code times its block's scale; s = max(max |x| / 448, 2^-126).
"""
import math

import torch

own = False

B = 128                     # columns (and, for weights, rows) of a block
E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -126


def _blocks(n):
    return -(-n // B)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of one request: latency alone
        dict(name="norm 1x4096", op="norm", rows=1, hidden=4096, resid=True),
        # the second norm of the 70B-shaped step, 4096 tokens
        dict(name="norm 4096x8192", op="norm", rows=4096, hidden=8192, resid=True),
        # 2047 tokens to two experts each, in the experts' order
        dict(name="quant 4094 of 2047x4096", op="quant", rows=4094, src=2047, cols=4096),
        # the attention output of a small decode batch, no index
        dict(name="quant 64x8192", op="quant", rows=64, src=0, cols=8192),
        # the 8B-shaped gate and up matrices, when a model is loaded
        dict(name="weights 2x14336x4096", op="weights", mats=2, rows=14336, cols=4096),
        # the small test layer's down projection, whose last block of columns has 48
        dict(name="weights 256x688", op="weights", mats=1, rows=256, cols=688),
        # one token through the 8B-shaped down projection: the weights' bytes
        dict(name="gemm 1x4096x14336 resid", op="gemm", m=1, n=4096, k=14336, epi="resid"),
        # 333 tokens (an odd prompt) through the 8B-shaped QKV projection
        dict(name="gemm 333x6144x4096", op="gemm", m=333, n=6144, k=4096, epi="store"),
        # the mixed 8B-shaped step's gate and up, 8 bits out for the down projection
        dict(name="gemm 2048x14336x4096 swiglu8", op="gemm", m=2048, n=14336, k=4096, epi="swiglu8"),
        # the 70B-shaped step's down projection, 4096 tokens: the largest
        dict(name="gemm 4096x8192x28672 resid", op="gemm", m=4096, n=8192, k=28672, epi="resid"),
        # a decode step of 32 requests through 8 experts, two each
        dict(name="grouped 64 of 8, swiglu8", op="grouped", m=64, groups=8, n=14336, k=4096, epi="swiglu8", skew=0.5, tail=0),
        # a mixed step of 2048 tokens through the experts' down projections: uneven groups, padding rows behind them
        dict(name="grouped 4096 of 8, store", op="grouped", m=4096, groups=8, n=4096, k=14336, epi="store", skew=1.0, tail=37),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "weights", "gemm", "gemm", "grouped"])
    cols = 16 * _spread(rng, 16, 512)
    if op == "norm":
        return dict(op=op, rows=_spread(rng, 1, 4096), hidden=cols, resid=rng.random() < 0.7)
    if op == "quant":
        rows = _spread(rng, 1, 8192)
        return dict(op=op, rows=rows, src=rng.choice([0, _spread(rng, 1, 4096)]), cols=cols)
    if op == "weights":
        mats = rng.choice([1, 2, 8])
        return dict(op=op, mats=mats, rows=8 * _spread(rng, 16, min(1792, 2 * 14336 * 4096 // (8 * mats * cols))), cols=cols)
    epi = rng.choice(["store", "resid", "swiglu", "swiglu8"] if op == "gemm" else ["store", "swiglu", "swiglu8"])
    k, m = 16 * _spread(rng, 16, 1792), _spread(rng, 1, 4096)
    groups = 1 if op == "gemm" else rng.choice([1, 4, 8, 16, 61])
    # a weight's bytes and the product's operations stay below the largest listed case's
    most = min(28672, 235_000_000 // (groups * k), 4096 * 8192 * 28672 // (2 * m * k))
    step = 16 if epi == "swiglu8" else 8
    n = step * _spread(rng, min(16, max(1, most // (2 * step))), max(1, most // (2 * step)))
    if op == "gemm":
        return dict(op=op, m=m, n=n, k=k, epi=epi)
    return dict(op=op, m=m, groups=groups, n=n, k=k, epi=epi, skew=rng.choice([0.0, 0.5, 1.0, 2.0]), tail=rng.choice([0, 0, _spread(rng, 1, 100)]))


def _two(case):
    return 2 if case["epi"].startswith("swiglu") else 1


def work(case):
    op = case["op"]
    if op == "norm":
        r, n = case["rows"], case["hidden"]
        return dict(bytes=float(r * n * (3 + (4 if case["resid"] else 0)) + 2 * n + 4 * r * _blocks(n)), flops=float(8 * r * n))
    if op == "quant":
        r, n = case["rows"], case["cols"]
        read = min(r, case["src"]) if case["src"] else r
        return dict(bytes=float(2 * read * n + r * n + 4 * r * _blocks(n) + (4 * r if case["src"] else 0)), flops=float(3 * r * n))
    if op == "weights":
        t, r, n = case["mats"], case["rows"], case["cols"]
        return dict(bytes=float(3 * t * r * n + 4 * t * _blocks(r) * _blocks(n)), flops=float(3 * t * r * n))
    m, n, k, two = case["m"], case["n"], case["k"], _two(case)
    g = case.get("groups", 1)
    rows = m - case.get("tail", 0) if m > case.get("tail", 0) else m
    used = min(g, rows)  # experts that can have a row at most
    out = rows * n * (1 if case["epi"] == "swiglu8" else 2) + (4 * rows * _blocks(n) if case["epi"] == "swiglu8" else 0)
    return dict(bytes=float(rows * k + 4 * rows * _blocks(k) + used * two * (n * k + 4 * _blocks(n) * _blocks(k)) + out + (2 * rows * n if case["epi"] == "resid" else 0)),
                flops=float(2 * two * rows * n * k))


# ------------------------------------------------------------------ inputs

def _gen(seed, i=0):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 16 + i)


def _codes(shape, std, gen):
    """Codes of normal values, as a block's scale spreads them: its largest magnitude is near 448."""
    x = torch.randn(shape, device="cuda", dtype=torch.bfloat16, generator=gen)
    return x.mul_(std).clamp_(-448, 448).to(E4M3)


def _scales(shape, mean, gen):
    return (torch.rand(shape, device="cuda", generator=gen) * 0.4 + 0.8) * mean


def _offsets(case, seed):
    """The experts' first rows (host): uneven groups, some of them empty, `tail` rows behind the last."""
    g = torch.Generator().manual_seed(int(seed) * 16 + 9)
    m, e = case["m"], case["groups"]
    rows = m - case["tail"] if m > case["tail"] else m
    p = torch.softmax(case["skew"] * torch.randn(e, generator=g), 0)
    count = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=e)
    return torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)])


def prepare(case, seed):
    op, s = case["op"], dict(case=case)
    if op == "norm":
        r, n = case["rows"], case["hidden"]
        s["x"] = torch.randn(r, n, device="cuda", generator=_gen(seed)).bfloat16()
        s["r"] = (torch.randn(r, n, device="cuda", generator=_gen(seed, 1)) * 0.5).bfloat16() if case["resid"] else None
        s["g"] = (1 + 0.1 * torch.randn(n, device="cuda", generator=_gen(seed, 2))).bfloat16()
        s["h"] = torch.empty_like(s["x"]) if case["resid"] else None
        s["q"], s["qs"] = torch.empty(r, n, device="cuda", dtype=E4M3), torch.empty(_blocks(n), r, device="cuda")
        return s
    if op == "quant":
        r, n = case["rows"], case["cols"]
        s["x"] = torch.randn(case["src"] or r, n, device="cuda", generator=_gen(seed)).bfloat16()
        s["index"] = torch.randint(0, case["src"], (r,), device="cuda", dtype=torch.int32, generator=_gen(seed, 1)) if case["src"] else None
        s["q"], s["qs"] = torch.empty(r, n, device="cuda", dtype=E4M3), torch.empty(_blocks(n), r, device="cuda")
        return s
    if op == "weights":
        t, r, n = case["mats"], case["rows"], case["cols"]
        s["w"] = torch.randn(t, r, n, device="cuda", dtype=torch.bfloat16, generator=_gen(seed)).mul_(0.02)
        s["q"], s["qs"] = torch.empty(t, r, n, device="cuda", dtype=E4M3), torch.empty(t, _blocks(r), _blocks(n), device="cuda")
        return s
    m, n, k, two = case["m"], case["n"], case["k"], _two(case)
    g = case.get("groups", 1)
    s["a"], s["as"] = _codes((m, k), 172, _gen(seed)), _scales((_blocks(k), m), 1 / 172, _gen(seed, 1))
    s["b"], s["bs"] = _codes((g, two, n, k), 109, _gen(seed, 2)), _scales((g, two, _blocks(n), _blocks(k)), 0.02 / 109, _gen(seed, 3))
    s["r"] = torch.randn(m, n, device="cuda", generator=_gen(seed, 4)).bfloat16() if case["epi"] == "resid" else None
    eight = case["epi"] == "swiglu8"
    s["c"] = torch.zeros(m, n, device="cuda", dtype=torch.bfloat16).to(E4M3 if eight else torch.bfloat16)
    s["cs"] = torch.zeros(_blocks(n), m, device="cuda") if eight else None
    if op == "grouped":
        off = _offsets(case, seed)
        s["off"], s["count"] = off.int().cuda(), (off[1:] - off[:-1]).tolist()
    else:
        s["b"], s["bs"] = s["b"][0], s["bs"][0]
    if two == 1:
        s["b"], s["bs"] = s["b"].squeeze(-3), s["bs"].squeeze(-3)
    else:
        s["b"] = s["b"].flatten(-3, -2)  # gate rows, then up rows
    return s


# ------------------------------------------------------------------ plain forms

def _pad(x, n, dim):
    """x with zeros up to n along dim."""
    more = list(x.shape)
    more[dim] = n - x.shape[dim]
    return torch.cat([x, x.new_zeros(more)], dim)


def _to_rows(y):
    """fp32 [rows, n] -> codes, scales [block, row]."""
    r, n = y.shape
    z = _pad(y, _blocks(n) * B, 1).view(r, -1, B)
    s = (z.abs().amax(2) / 448).clamp(min=TINY)
    q = (z / s[:, :, None]).clamp(-448, 448).view(r, -1)[:, :n]
    return q.to(E4M3), s.t().contiguous()


def _from_rows(q, s):
    """codes [rows, n], scales [block, row] -> fp32."""
    return q.float() * s.t().repeat_interleave(B, 1)[:, :q.shape[1]]


def _from_weights(q, s):
    """codes [..., n, k], scales [..., n block, k block] -> fp32."""
    return q.float() * s.repeat_interleave(B, -2)[..., :q.shape[-2], :].repeat_interleave(B, -1)[..., :q.shape[-1]]


def _weights_of(s):
    """The weights of a product in fp32, [groups?, two n, k]."""
    case, b, bs = s["case"], s["b"], s["bs"]
    if _two(case) == 1:
        return _from_weights(b, bs)
    n, k = case["n"], case["k"]
    return _from_weights(b.unflatten(-2, (2, n)), bs).flatten(-3, -2)


def _finish(s, acc):
    """A product's fp32 sums [rows, n or 2 n] through the epilogue."""
    epi, n = s["case"]["epi"], s["case"]["n"]
    if epi == "store":
        return [acc.bfloat16()]
    if epi == "resid":
        return [(s["r"].float() + acc).bfloat16()]
    gate, up = acc[:, :n], acc[:, n:]
    y = gate / (1 + torch.exp(-gate)) * up
    return [y.bfloat16()] if epi == "swiglu" else list(_to_rows(y))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = s["x"].float() + (s["r"].float() if case["resid"] else 0)
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5) * s["g"].float()
        return list(_to_rows(y)) + ([h.bfloat16()] if case["resid"] else [])
    if op == "quant":
        x = s["x"] if s["index"] is None else s["x"][s["index"].long()]
        return list(_to_rows(x.float()))
    if op == "weights":
        t, r, n = s["w"].shape
        z = _pad(_pad(s["w"].float(), _blocks(r) * B, 1), _blocks(n) * B, 2).view(t, _blocks(r), B, _blocks(n), B)
        sc = (z.abs().amax((2, 4)) / 448).clamp(min=TINY)
        q = (z / sc[:, :, None, :, None]).clamp(-448, 448).view(t, _blocks(r) * B, -1)[:, :r, :n]
        return [q.to(E4M3), sc]
    a = _from_rows(s["a"], s["as"])
    w = _weights_of(s)
    if op == "gemm":
        return _finish(s, a @ w.t())
    # by expert, one product each; the rows behind the last group multiply none
    parts = a.split(s["count"] + [case["m"] - sum(s["count"])])
    acc = torch.cat([x @ y.t() for x, y in zip(parts, w)] + [a.new_zeros(parts[-1].shape[0], w.shape[1])])
    used = s["off"][-1]
    out = _finish(s, acc)
    keep = torch.arange(case["m"], device="cuda") < used
    # rows behind the last group stay as they are
    if len(out) == 1:
        return [torch.where(keep[:, None], out[0], s["c"])]
    return [torch.where(keep[:, None], out[0].float(), s["c"].float()).to(E4M3), torch.where(keep, out[1], s["cs"])]


def run(s):
    if not own:
        return _plain(s)
    from nano_intra_device_gb300 import _lib
    case = s["case"]
    op = case["op"]
    if op == "norm":
        _lib.rmsnorm_fp8(s["x"], s["g"], s["q"], s["qs"], 1e-5, r=s["r"], h=s["h"])
        return [s["q"], s["qs"]] + ([s["h"]] if case["resid"] else [])
    if op == "quant":
        _lib.quant_fp8(s["x"], s["q"], s["qs"], index=s["index"])
        return [s["q"], s["qs"]]
    if op == "weights":
        _lib.quant_fp8_weights(s["w"], s["q"], s["qs"])
        return [s["q"], s["qs"]]
    epi = dict(store=_lib.NF_EPI_STORE, resid=_lib.NF_EPI_RESID, swiglu=_lib.NF_EPI_SWIGLU, swiglu8=_lib.NF_EPI_SWIGLU_FP8)[case["epi"]]
    if op == "gemm":
        _lib.gemm_fp8(s["a"], s["as"], s["b"], s["bs"], s["c"], c_s=s["cs"], r=s["r"], epilogue=epi)
    else:
        _lib.gemm_fp8_grouped(s["a"], s["as"], s["b"], s["bs"], s["off"], s["c"], c_s=s["cs"], epilogue=epi)
    return [s["c"]] if s["cs"] is None else [s["c"], s["cs"]]


# ------------------------------------------------------------------ 64 bits

def _exact_blocks(y):
    """Values over their block's scale (before the rounding to 8 bits), and the scales [block, row]."""
    n = y.shape[1]
    top = torch.stack([y[:, i:i + B].abs().max(1).values for i in range(0, n, B)])
    s = torch.maximum(top / 448, torch.full_like(top, TINY))
    which = torch.arange(n, device=y.device) // B
    return [y / s.t()[:, which], s]


def _exact_product(s, rows, b, bs):
    """One matrix's product of some rows in 64 bits; b [n, k], bs [n block, k block]."""
    k, n = b.shape[1], b.shape[0]
    kb, nb = torch.arange(k, device="cuda") // B, torch.arange(n, device="cuda") // B
    a = s["a"][rows].double() * s["as"].double()[:, rows].t()[:, kb]
    return torch.einsum("mk,nk->mn", a, b.double() * bs.double()[nb][:, kb])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double()
        if case["resid"]:
            h = h + s["r"].double()
        y = h * (h.square().sum(1) / h.shape[1] + 1e-5).rsqrt()[:, None] * s["g"].double()
        return _exact_blocks(y) + ([h] if case["resid"] else [])
    if op == "quant":
        x = s["x"].double()
        return _exact_blocks(x if s["index"] is None else x.index_select(0, s["index"].long()))
    if op == "weights":
        w = s["w"].double()
        q, sc = torch.empty_like(w), s["qs"].double()
        for i in range(0, w.shape[1], B):
            for j in range(0, w.shape[2], B):
                part = w[:, i:i + B, j:j + B]
                sc[:, i // B, j // B] = (part.abs().flatten(1).max(1).values / 448).clamp(min=TINY)
                q[:, i:i + B, j:j + B] = part / sc[:, i // B, j // B, None, None]
        return [q, sc]
    m, n, epi = case["m"], case["n"], case["epi"]
    off = s["off"].tolist() if op == "grouped" else [0, m]
    out = torch.zeros(m, n, device="cuda", dtype=torch.float64)
    for e in range(len(off) - 1):
        rows = torch.arange(off[e], off[e + 1], device="cuda")
        if not len(rows):
            continue
        b, bs = (s["b"][e], s["bs"][e]) if op == "grouped" else (s["b"], s["bs"])
        if _two(case) == 1:
            out[rows] = _exact_product(s, rows, b, bs)
        else:
            gate, up = _exact_product(s, rows, b[:n], bs[0]), _exact_product(s, rows, b[n:], bs[1])
            out[rows] = gate * torch.sigmoid(gate) * up
    if epi == "resid":
        out += s["r"].double()
    if epi != "swiglu8":
        return [out]
    q, sc = _exact_blocks(out)
    sc[:, off[-1]:] = 0
    return [q, sc]
