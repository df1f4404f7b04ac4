"""Cases and plain forms of the 4-bit KV cache's operators.

Four operators work on one paged cache: ``tables`` builds block tables and slot
maps on the GPU from request lengths, ``append`` norms and rotates queries and
keys and appends K and V, ``read`` takes rows of the 4-bit cache back out as
bf16, ``attend`` is attention over the 4-bit cache.

``own = False`` computes each in elementary torch operations; ``own = True``
calls the library.

The 4-bit format: a block is 16 channels of one (position, KV head); its scale
s is e4m3, its codes n are e2m1, and it stands for n * s * 2**E.  A pool is
uint8 [num_pages, n_kv, 2 (K, V), 9 d]: 16 rows of d / 2 code bytes (channel 2i
in the low nibble of byte i), then 16 rows of d / 16 scale bytes.
"""
import math

import numpy as np
import torch

own = False

P = 16                      # positions of a page
LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of a small server: 64 requests grow by one token
        dict(name="tables decode 64", op="tables", n_seq=64, median=600, prompts=0, plen=0, ended=0, lens=1),
        # a mixed iteration: most requests grow by one, some end, two prompts start
        dict(name="tables mixed 1801", op="tables", n_seq=1801, median=600, prompts=2, plen=255, ended=37, lens=2),
        # a burst of prompts: slot maps of about half a million tokens
        dict(name="tables prompts 4096", op="tables", n_seq=4096, median=300, prompts=1024, plen=1000, ended=500, lens=3),
        # one decode step's keys and values, 64 requests of the 8B shape
        dict(name="append fp4 64", op="append", tokens=64, chunk=0, n_q=32, n_kv=8, d=128, theta=5e5, pos=8192, cache="fp4", norm=True),
        # the largest prefill iteration of the 70B shape, an odd token count
        dict(name="append fp4 8191", op="append", tokens=8191, chunk=8000, n_q=64, n_kv=8, d=128, theta=1e4, pos=131072, cache="fp4", norm=True),
        # a mixed iteration that keeps a 16-bit cache
        dict(name="append bf16 2048", op="append", tokens=2048, chunk=256, n_q=32, n_kv=8, d=128, theta=5e5, pos=8192, cache="bf16", norm=True),
        # the rows of one step of a small model
        dict(name="read 333", op="read", tokens=333, n_kv=2, d=64),
        # a long prompt's cache handed to the 16-bit path
        dict(name="read 30000", op="read", tokens=30000, n_kv=8, d=128),
        # a decode step at the smallest batch: one row over a long context
        dict(name="attend 1 row long", op="attend", n_dec=1, median=65543, sigma=0.0, clip=65543, empty=0, chunks=0, qlen=0, prefix=0,
             n_q=32, n_kv=8, d=128, lens=1),
        # the stack's decode batch: 64 requests, lognormal contexts, and a padded batch's empty rows
        dict(name="attend 64 rows", op="attend", n_dec=66, median=600, sigma=1.0, clip=8192, empty=2, chunks=0, qlen=0, prefix=0,
             n_q=32, n_kv=8, d=128, lens=1),
        # a large decode batch at the 70B shape's group of 8
        dict(name="attend 1000 rows", op="attend", n_dec=1000, median=600, sigma=1.0, clip=2048, empty=0, chunks=0, qlen=0, prefix=0,
             n_q=64, n_kv=8, d=128, lens=2),
        # a serving iteration: decode rows beside a prompt chunk over a long prefix
        dict(name="attend mixed chunk", op="attend", n_dec=63, median=600, sigma=1.0, clip=4096, empty=0, chunks=1, qlen=1985, prefix=4099,
             n_q=32, n_kv=8, d=128, lens=3),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "read", "attend", "attend", "attend"])
    lens = rng.randrange(1, 1 << 20)
    if op == "tables":
        n = _spread(rng, 1, 4096)
        prompts = rng.randrange(0, 1 + n // 4)
        return dict(op=op, n_seq=n, median=_spread(rng, 8, 1000), prompts=prompts, plen=_spread(rng, 1, 1000) if prompts else 0,
                    ended=rng.randrange(0, 1 + n // 8), lens=lens)
    d, n_kv, grp = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    if op == "append":
        t = _spread(rng, 1, 8191)
        return dict(op=op, tokens=t, chunk=rng.randrange(0, t + 1), n_q=n_kv * grp, n_kv=n_kv, d=d, theta=rng.choice([1e4, 5e5, 1e6]),
                    pos=_spread(rng, 16, 131072), cache=rng.choice(["fp4", "fp4", "bf16"]), norm=rng.random() < 0.8)
    if op == "read":
        return dict(op=op, tokens=_spread(rng, 1, 30000), n_kv=n_kv, d=d)
    # positions that the plain form holds at once: at most what the largest listed case does
    clip = _spread(rng, 1, 65543)
    rows = max(1, min(1000, 2048000 * 1024 // (clip * n_kv * d)))
    n_dec = _spread(rng, 1, rows)
    chunks = rng.choice([0, 0, 1, 2]) if clip <= 8192 else 0
    if chunks and rng.random() < 0.2:
        n_dec = 0
    qlen = _spread(rng, 1, 1985 // chunks) if chunks else 0
    prefix = rng.choice([0, _spread(rng, 1, 4099)]) if chunks else 0
    return dict(op=op, n_dec=n_dec, median=_spread(rng, 1, max(1, clip)), sigma=rng.choice([0.0, 0.5, 1.0]), clip=clip,
                empty=rng.choice([0, 0, 1]) if n_dec > 1 else 0, chunks=chunks, qlen=qlen, prefix=prefix, n_q=n_kv * grp, n_kv=n_kv, d=d, lens=lens)


def _lengths(case):
    """The request lengths of a case (host): the program has them as whole numbers."""
    r = np.random.RandomState(case["lens"] % (1 << 31))
    if case["op"] == "tables":
        n, k, e = case["n_seq"], case["prompts"], case["ended"]
        held = np.clip(np.rint(case["median"] * np.exp(r.standard_normal(n))), 1, 8191).astype(np.int64)
        new = held + 1
        order = r.permutation(n)
        held[order[:k]] = 0
        new[order[:k]] = r.randint(max(1, case["plen"] // 2), case["plen"] + 1, k) if k else 0
        new[order[k:k + e]] = 0
        return held, new
    n, c = case["n_dec"], case["chunks"]
    ctx = np.clip(np.rint(case["median"] * np.exp(case["sigma"] * r.standard_normal(n))), 1, case["clip"]).astype(np.int64)
    if case["empty"]:
        ctx[r.permutation(n)[:case["empty"]]] = 0
    q = r.randint(max(1, case["qlen"] - case["qlen"] // 4), case["qlen"] + 1, c) if c else np.zeros(0, np.int64)
    if c:
        q[0] = case["qlen"]
    pre = np.full(c, case["prefix"]) + (r.randint(0, 16, c) if c and case["prefix"] else 0)
    return np.concatenate([ctx, pre + q]).astype(np.int64), np.concatenate([np.ones(n), q]).astype(np.int64)


def work(case):
    op = case["op"]
    if op == "tables":
        held, new = _lengths(case)
        moved = np.abs(-(-new // P) + (-held // P)).sum()
        return dict(bytes=float(8 * len(held) + 8 * moved + 4 * len(held) + 12 * np.clip(new - held, 0, None).sum()), flops=0)
    d, n_kv = case["d"], case["n_kv"]
    row4 = n_kv * 2 * (d // 2 + d // 16)  # bytes of one position in the 4-bit cache
    if op == "read":
        return dict(bytes=float(case["tokens"] * (row4 + 4 * n_kv * d + 4)), flops=float(case["tokens"] * n_kv * d * 2))
    if op == "append":
        t, n_q = case["tokens"], case["n_q"]
        kept = row4 + row4 + 4 * n_kv * d if case["cache"] == "fp4" else 4 * n_kv * d  # written (and, in 4 bits, read back)
        return dict(bytes=float(t * (2 * (n_q + 2 * n_kv) * d + 2 * n_q * d + kept + 8)), flops=float(t * (n_q + n_kv) * d * 8))
    lens, q = _lengths(case)
    pairs = sum(int(b) * max(0, int(a) - int(b)) + int(min(a, b)) * (int(min(a, b)) + 1) // 2 for a, b in zip(lens, q))
    n_tok = int(q.sum())
    return dict(bytes=float(lens.sum() * row4 + 4 * n_tok * case["n_q"] * d + 4 * (-(-lens // P)).sum() + 4 * len(lens)), flops=float(4 * d * case["n_q"] * pairs))


# ------------------------------------------------------------------ inputs

def _gen(seed, k=0):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 16 + k)


def _pool(n, n_kv, d, seed):
    """A filled 4-bit pool: uniform codes, scales as blocks of 16 unit normals have them (largest magnitude 1.2 to 3.5)."""
    pool = torch.randint(0, 256, (n, n_kv, 2, 9 * d), dtype=torch.uint8, device="cuda", generator=_gen(seed, 1))
    s = torch.rand(n, n_kv, 2, d, device="cuda", generator=_gen(seed, 2)) * 0.4 + 0.2
    pool[..., 8 * d:] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    return pool


def _paged(lens, seed, extra=0):
    """A block table for these lengths over shuffled pages."""
    need = -(-lens // P)
    width, total = max(1, int(need.max(initial=0))), int(need.sum())
    perm = torch.randperm(total + extra, generator=_gen(seed, 3), device="cuda").int()
    at = np.concatenate([[0], np.cumsum(need)[:-1]])
    j = torch.arange(width, device="cuda")
    need_t, at_t = torch.from_numpy(need).cuda(), torch.from_numpy(at).cuda()
    idx = at_t[:, None] + j
    bt = torch.where(j < need_t[:, None], perm[idx.clamp(max=max(0, total + extra - 1))] if total + extra else torch.zeros_like(idx).int(), -1)
    return bt.int().contiguous(), total, perm


def prepare(case, seed):
    torch.backends.cuda.matmul.allow_tf32 = False
    return globals()["_prepare_" + case["op"]](dict(case), seed)


def _prepare_tables(case, seed):
    held, new = _lengths(case)
    n = len(held)
    max_pages = 8192 // P
    bt, used, perm = _paged(held, seed, extra=int((-(-new // P)).sum()) + 5)
    table = torch.full((n, max_pages), -1, dtype=torch.int32, device="cuda")
    table[:, :bt.shape[1]] = bt
    num_pages = perm.numel()
    free = num_pages - used
    head = num_pages - free // 2 - 1  # the free part of the ring passes its end
    ring = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    ring[(torch.arange(free, device="cuda") + head) % num_pages] = perm[used:]
    cap = int(np.clip(new - held, 0, None).sum()) + 7  # rows behind the last token stay as they were
    out = dict(tok_begin=n + 1, tok_seq=cap, tok_pos=cap, tok_slot=cap, state_out=4)
    s = {k: torch.full((v,), -5, dtype=torch.int32, device="cuda") for k, v in out.items()}
    s |= dict(case=case, held=torch.from_numpy(held).int().cuda(), lens=torch.from_numpy(new).int().cuda(), table=table, ring=ring,
              state=torch.tensor([head, free], dtype=torch.int32, device="cuda"))
    if own:
        from nano_intra_device_gb300 import _lib
        s["args"] = _lib.BlockTables(s["held"], s["lens"], table, ring, s["state"], s["state_out"], s["tok_begin"], s["tok_seq"],
                                     s["tok_pos"], s["tok_slot"])
    return s


def _own_shape(case):
    from nano_intra_device_gb300 import _lib, workload
    return _lib.make_shape(workload.Shape(hidden=case["n_q"] * case["d"], n_q=case["n_q"], n_kv=case["n_kv"], head_dim=case["d"], ffn=16,
                                          rms_eps=1e-5, rope_theta=case.get("theta", 1e4)))


def _own_cache(case, shape, num_pages, k, v=None, exps=(0, 0)):
    from nano_intra_device_gb300 import _lib
    return _lib.KvCache(shape, num_pages, _lib.NF_KV_BF16 if v is not None else _lib.NF_KV_FP4, k, v, *exps)


def _prepare_append(case, seed):
    t, c, n_q, n_kv, d = (case[k] for k in ("tokens", "chunk", "n_q", "n_kv", "d"))
    g = _gen(seed)
    qkv = torch.randn(t, (n_q + 2 * n_kv) * d, device="cuda", generator=g)
    # keys have a few strong channels, values a spread of magnitudes
    qkv[:, :(n_q + n_kv) * d] *= torch.exp(0.5 * torch.randn((n_q + n_kv) * d, device="cuda", generator=g))
    qkv[:, (n_q + n_kv) * d:] *= torch.exp(0.5 * torch.randn(t, 1, device="cuda", generator=g))
    gains = (1 + 0.2 * torch.randn(2, d, device="cuda", generator=g)).bfloat16()
    # a chunk fills pages one after the other, decode rows have a page each
    num_pages = -(-c // P) + (t - c) + 1
    page = torch.randperm(num_pages, device="cuda", generator=g)
    i = torch.arange(t, device="cuda")
    start = torch.randint(0, max(1, case["pos"] - c), (t,), device="cuda", generator=g)
    pos = torch.where(i < c, start[0] // P * P + i, start)
    slot = page[torch.where(i < c, i // P, -(-c // P) + i - c)] * P + pos % P
    if t > 8:
        slot[t // 2] = -1  # a token that has no page
    s = dict(case=case, qkv=qkv.bfloat16(), q_gain=gains[0] if case["norm"] else None, k_gain=gains[1] if case["norm"] else None,
             pos=pos.int(), slot=slot.int(), q=torch.zeros(t, n_q, d, dtype=torch.bfloat16, device="cuda"), exps=(0, 1))
    size = (num_pages, n_kv, P, d)
    if case["cache"] == "bf16":
        s["k_pool"], s["v_pool"] = (torch.randn(size, device="cuda", generator=g).bfloat16() for _ in range(2))
    else:
        s["pool"] = _pool(num_pages, n_kv, d, seed)
        s["k"], s["v"] = (torch.zeros(t, n_kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:
        s["shape"] = _own_shape(case)
        s["cache"] = _own_cache(case, s["shape"], num_pages, s["k_pool"], s["v_pool"]) if case["cache"] == "bf16" else \
            _own_cache(case, s["shape"], num_pages, s["pool"], None, s["exps"])
    return s


def _prepare_read(case, seed):
    t, n_kv, d = case["tokens"], case["n_kv"], case["d"]
    num_pages = -(-t // P) + 3
    slot = torch.randperm(num_pages, device="cuda", generator=_gen(seed))[torch.arange(t, device="cuda") // P] * P + torch.arange(t, device="cuda") % P
    if t > 8:
        slot[t // 3] = -1
    s = dict(case=case, pool=_pool(num_pages, n_kv, d, seed), slot=slot.int(), exps=(1, -1))
    s["k"], s["v"] = (torch.zeros(t, n_kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:
        s["shape"] = _own_shape(dict(case, n_q=n_kv))
        s["cache"] = _own_cache(case, s["shape"], num_pages, s["pool"], None, s["exps"])
    return s


def _prepare_attend(case, seed):
    lens, q = _lengths(case)
    n_q, n_kv, d, n_dec = (case[k] for k in ("n_q", "n_kv", "d", "n_dec"))
    bt, pages, _ = _paged(lens, seed, extra=2)
    n_tok = int(q.sum())
    begin = np.concatenate([[0], np.cumsum(q)])
    s = dict(case=case, bt=bt, lens=torch.from_numpy(lens).int().cuda(), pool=_pool(pages + 2, n_kv, d, seed), exps=(0, -1),
             q=(1.5 * torch.randn(n_tok, n_q, d, device="cuda", generator=_gen(seed))).bfloat16(),
             o=torch.zeros(n_tok, n_q, d, dtype=torch.bfloat16, device="cuda"),
             begin=torch.from_numpy(begin).int().cuda() if case["chunks"] else None,
             width=(int(-(-lens[:n_dec].max(initial=0) // P)), int(-(-lens[n_dec:].max(initial=0) // P))))
    if case["chunks"]:  # where the chunks' rows stand in [chunk, longest chunk] rows, and the other way round
        qm, first = int(q[n_dec:].max()), n_dec
        i = torch.arange(qm, device="cuda")
        ql, qb = torch.from_numpy(q[first:]).cuda(), torch.from_numpy(begin[first:-1]).cuda()
        s["pad"] = (qb[:, None] + i.clamp(max=qm)).clamp(max=n_tok - 1)
        s["row_pos"] = torch.from_numpy(lens[first:]).cuda()[:, None] - ql[:, None] + i
        s["unpad"] = torch.nonzero((i < ql[:, None]).reshape(-1)).reshape(-1)
    if own:
        from nano_intra_device_gb300 import _lib
        s["shape"] = _own_shape(case)
        s["cache"] = _own_cache(case, s["shape"], pages + 2, s["pool"], None, s["exps"])
        s["handle"] = _lib.Kv4(s["shape"], pages + 2, bt.shape[1])
    return s


# ------------------------------------------------------------------ plain forms

def run(state):
    return globals()["_run_" + state["case"]["op"]](state)


def _run_tables(s):
    if own:
        from nano_intra_device_gb300 import _lib
        _lib.block_tables(s["args"])
        return {k: s[k] for k in ("table", "ring", "state_out", "tok_begin", "tok_seq", "tok_pos", "tok_slot")}
    held, new, table, ring = s["held"].long(), s["lens"].long(), s["table"], s["ring"]
    (n, width), num_pages = table.shape, ring.numel()
    ph, pl, q = (held + P - 1) // P, (new + P - 1) // P, (new - held).clamp(min=0)
    take, back = (pl - ph).clamp(min=0), (ph - pl).clamp(min=0)
    take_to, back_to, tok_to = take.cumsum(0), back.cumsum(0), q.cumsum(0)
    head, count = s["state"][0].long(), s["state"][1].long()
    short = take_to[-1] > count
    j = torch.arange(width, device=table.device)
    grown = (j >= ph[:, None]) & (j < pl[:, None])
    got = ring[(head + (take_to - take)[:, None] + j - ph[:, None]) % num_pages]
    table = torch.where(grown, torch.where(short, torch.full_like(got, -1), got), table)
    freed = (j >= pl[:, None]) & (j < ph[:, None]) & ~short
    at = torch.where(freed, (head + count + (back_to - back)[:, None] + j - pl[:, None]) % num_pages, num_pages)
    ring = torch.cat([ring, ring[:1]]).scatter(0, at.reshape(-1), s["table"].reshape(-1))[:num_pages]
    n_tok = tok_to[-1]
    state = torch.stack([torch.where(short, head, (head + take_to[-1]) % num_pages), torch.where(short, count, count - take_to[-1] + back_to[-1]),
                         n_tok, (take_to[-1] - count).clamp(min=0)]).int()
    t = torch.arange(s["tok_seq"].numel(), device=table.device)
    seq = torch.searchsorted(tok_to, t, right=True).clamp(max=n - 1)
    pos = held[seq] + t - (tok_to - q)[seq]
    page = table[seq, (pos // P).clamp(0, width - 1)].long()
    slot = torch.where(page >= 0, page * P + pos % P, -1)
    live = t < n_tok
    keep = lambda x, old: torch.where(live, x.int(), old)  # noqa: E731
    return dict(table=table, ring=ring, state_out=state, tok_begin=torch.cat([tok_to[:1] * 0, tok_to]).int(), tok_seq=keep(seq, s["tok_seq"]),
                tok_pos=keep(pos, s["tok_pos"]), tok_slot=keep(slot, s["tok_slot"]))


def _round_to(x, low, bits, most):
    """Magnitudes x to the nearest number of `bits` fraction bits, lowest exponent `low`, ties to even, at most `most`."""
    e = torch.frexp(x)[1] - 1
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=low) - bits)
    return (torch.round(x / step) * step).clamp(max=most)


def _through_4_bits(x, exp):
    """The values that the 4-bit cache holds for x [..., d]."""
    b = (x * 2.0 ** -exp).unflatten(-1, (-1, 16))
    a = b.abs()
    s = _round_to(a.amax(-1, keepdim=True) / 6, -6, 3, 448.0)
    n = torch.where(s > 0, _round_to(a / s, 0, 1, 6.0), torch.zeros_like(a))
    return (torch.copysign(n, b) * s).flatten(-2) * 2.0 ** exp


def _norm_rope(u, gain, pos, theta, eps):
    d = u.shape[-1]
    if gain is not None:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + eps) * gain.to(u.dtype)
    inv = torch.tensor(theta, dtype=torch.float64, device=u.device) ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=u.device) / d)
    angle = pos.double()[:, None] * inv  # far positions: the angle needs 64 bits
    c, s = angle.cos().to(u.dtype)[:, None], angle.sin().to(u.dtype)[:, None]
    a, b = u[..., :d // 2], u[..., d // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _run_append(s):
    case = s["case"]
    if own:
        from nano_intra_device_gb300 import _lib
        _lib.qk_norm_rope(s["shape"], s["qkv"], s["q_gain"], s["k_gain"], s["pos"], s["slot"], s["q"], s["cache"])
        if case["cache"] == "bf16":
            return dict(q=s["q"], k_pool=s["k_pool"], v_pool=s["v_pool"])
        _lib.kv4_read(s["shape"], s["cache"], s["slot"], s["k"], s["v"])
        return dict(q=s["q"], k=s["k"], v=s["v"])
    n_q, n_kv, d = case["n_q"], case["n_kv"], case["d"]
    x = s["qkv"].view(-1, n_q + 2 * n_kv, d)
    q = _norm_rope(x[:, :n_q].float(), s["q_gain"], s["pos"], case["theta"], 1e-5).bfloat16()
    slot, v = s["slot"].long(), x[:, n_q + n_kv:]
    if case["cache"] == "bf16":
        k = _norm_rope(x[:, n_q:n_q + n_kv].float(), s["k_gain"], s["pos"], case["theta"], 1e-5).bfloat16()
        at = torch.where(slot >= 0, slot, s["k_pool"].shape[0] * P)  # a token without a page goes to a row that is cut off
        put = lambda pool, r: torch.cat([pool.transpose(1, 2).flatten(0, 1), r[:1]]).index_copy(0, at, r)[:-1].unflatten(0, (-1, P)).transpose(1, 2).contiguous()  # noqa: E731
        return dict(q=q, k_pool=put(s["k_pool"], k), v_pool=put(s["v_pool"], v))
    # in 64 bits: a code goes by which side of a border its value lies
    k = _norm_rope(x[:, n_q:n_q + n_kv].double(), s["k_gain"], s["pos"], case["theta"], 1e-5)
    here = (slot >= 0)[:, None, None]
    return dict(q=q, k=torch.where(here, _through_4_bits(k, s["exps"][0]), 0.0).bfloat16(),
                v=torch.where(here, _through_4_bits(v.float(), s["exps"][1]), 0.0).bfloat16())


def _values(part, d, exp):
    """fp32 values of K or V: part [..., 9 d] bytes of (page, KV head) blocks -> [..., P, d]."""
    codes = part[..., :8 * d].unflatten(-1, (P, d // 2))
    scale = part[..., 8 * d:].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (P, d // 16))
    lut = torch.tensor(LUT, device=part.device)
    n = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    return n * (scale * 2.0 ** exp).repeat_interleave(16, -1)


def _run_read(s):
    if own:
        from nano_intra_device_gb300 import _lib
        _lib.kv4_read(s["shape"], s["cache"], s["slot"], s["k"], s["v"])
        return dict(k=s["k"], v=s["v"])
    d, slot = s["case"]["d"], s["slot"].long()
    at, here = slot.clamp(min=0), (slot >= 0)[:, None, None]
    row = lambda i: torch.where(here, _values(s["pool"][:, :, i], d, s["exps"][i]).transpose(1, 2).flatten(0, 1)[at], 0.0).bfloat16()  # noqa: E731
    return dict(k=row(0), v=row(1))


def _attend_padded(s, q, bt, seen):
    """q [n, h, g, rows, d] over the pages bt [n, pages], row r of sequence n sees the first seen[n, r] positions."""
    d = q.shape[-1]
    held = s["pool"][bt.clamp(min=0).long()]  # [n, pages, h, 2, 9 d]
    k = _values(held[..., 0, :], d, s["exps"][0]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(q.float().flatten(2, 3), k.transpose(-1, -2)).unflatten(2, q.shape[2:4]) / math.sqrt(d)
    del k
    see = (torch.arange(x.shape[-1], device=x.device) < seen[..., None])[:, None, None]
    x = x.masked_fill(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    del x
    v = _values(held[..., 1, :], d, s["exps"][1]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p.flatten(2, 3), v).unflatten(2, q.shape[2:4]) / torch.where(total > 0, total, 1.0)


def _run_attend(s):
    if own:
        from nano_intra_device_gb300 import _lib
        _lib.attention_kv4(s["handle"], s["q"], s["cache"], s["bt"], s["lens"], s["o"], s["begin"])
        return s["o"]
    c, parts = s["case"], []
    n, h = c["n_dec"], c["n_kv"]
    if n and not s["width"][0]:
        parts.append(torch.zeros_like(s["q"][:n]))
    elif n:
        o = _attend_padded(s, s["q"][:n].unflatten(1, (h, -1)).unsqueeze(3), s["bt"][:n, :s["width"][0]], s["lens"][:n, None])
        parts.append(o.flatten(1, 3).bfloat16())
    if c["chunks"]:
        q = s["q"][s["pad"]].unflatten(2, (h, -1)).permute(0, 2, 3, 1, 4)  # [chunk, h, g, rows, d]
        o = _attend_padded(s, q, s["bt"][n:, :s["width"][1]], s["row_pos"] + 1)
        parts.append(o.permute(0, 3, 1, 2, 4).flatten(0, 1).flatten(1, 2)[s["unpad"]].bfloat16())
    return torch.cat(parts)


# ------------------------------------------------------------------ the definition in 64 bits

E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])
E2M1 = np.array(LUT[:8])


def _nearest(x, grid):
    """Magnitudes x to the nearest entry of grid (ascending; its even entries end in a 0 bit), ties to the even entry."""
    grid = torch.from_numpy(grid).to(x.device)
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - x, x - grid[lo]
    return grid[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]


def _held(x, exp):
    y = x.reshape(*x.shape[:-1], -1, 16) / 2.0 ** exp
    s = _nearest(y.abs().max(-1, keepdim=True).values / 6, E4M3)
    n = _nearest(torch.where(s > 0, y.abs() / s, 0.0), E2M1)
    return (torch.sign(y) * n * s * 2.0 ** exp).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)


def _exact_tables(s):
    """Request by request on the host."""
    held, new, table, ring = (s[k].cpu().numpy().astype(np.int64) for k in ("held", "lens", "table", "ring"))
    head, count = (int(v) for v in s["state"])
    need = [max(0, -(-int(b) // P) - -(-int(a) // P)) for a, b in zip(held, new)]
    short, taken, freed, tok = sum(need) > count, 0, 0, 0
    out_table, out_ring, begin = table.copy(), ring.copy(), [0]
    rows = [s[k].cpu().numpy().astype(np.int64) for k in ("tok_seq", "tok_pos", "tok_slot")]
    for i, (a, b) in enumerate(zip(held.tolist(), new.tolist())):
        for j in range(-(-a // P), -(-b // P)):
            out_table[i, j] = -1 if short else ring[(head + taken) % len(ring)]
            taken += 1
        for j in range(-(-b // P), -(-a // P)):
            if not short:
                out_ring[(head + count + freed) % len(ring)] = table[i, j]
                freed += 1
        pos = np.arange(a, max(a, b))
        page = out_table[i, pos // P]
        for r, v in zip(rows, (np.full(len(pos), i), pos, np.where(page >= 0, page * P + pos % P, -1))):
            r[tok:tok + len(pos)] = v
        tok += len(pos)
        begin.append(tok)
    state = [head, count, tok, sum(need) - count] if short else [(head + taken) % len(ring), count - taken + freed, tok, 0]
    return {k: torch.from_numpy(np.asarray(v)).int() for k, v in dict(table=out_table, ring=out_ring, state_out=state, tok_begin=begin,
                                                                    tok_seq=rows[0], tok_pos=rows[1], tok_slot=rows[2]).items()}


def _exact_append(s):
    c = s["case"]
    n_q, n_kv, d, t = c["n_q"], c["n_kv"], c["d"], c["tokens"]
    heads = s["qkv"].double().reshape(t, -1, d)
    i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones(t, d // 2, dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * torch.exp(-2 * i / d * math.log(c["theta"])))

    def rotated(u, gain):
        if gain is not None:
            u = u / (u.pow(2).sum(-1, keepdim=True) / d + 1e-5).sqrt() * gain.double()
        z = torch.complex(u[..., :d // 2].contiguous(), u[..., d // 2:].contiguous()) * turn[:, None]
        return torch.cat([z.real, z.imag], -1)

    q, k, v = rotated(heads[:, :n_q], s["q_gain"]), rotated(heads[:, n_q:n_q + n_kv], s["k_gain"]), heads[:, n_q + n_kv:]
    slot = s["slot"].long()
    live = slot >= 0
    if c["cache"] == "fp4":
        return dict(q=q, k=_held(k, s["exps"][0]) * live[:, None, None], v=_held(v, s["exps"][1]) * live[:, None, None])
    pools = {}
    for name, r in (("k_pool", k), ("v_pool", v)):
        pools[name] = s[name].double()
        pools[name][slot[live] // P, :, slot[live] % P] = r[live]
    return dict(q=q, **pools)


def _blocks(s, pages, part):
    """Values [len(pages) * P, n_kv, d] of K (part 0) or V (1) in 64 bits, nibble by nibble."""
    d = s["case"]["d"]
    raw = s["pool"][pages, :, part]
    b = raw[..., :8 * d].reshape(*raw.shape[:2], P, d // 2).long()
    val = torch.empty(*raw.shape[:2], P, d, dtype=torch.float64, device="cuda")
    grid = torch.from_numpy(E2M1).cuda()
    val[..., 0::2] = grid[b % 8] * (1 - 2 * (b // 8 % 2))
    val[..., 1::2] = grid[b // 16 % 8] * (1 - 2 * (b // 128))
    e = raw[..., 8 * d:].reshape(*raw.shape[:2], P, d // 16, 1).long()
    val = (val.reshape(*raw.shape[:2], P, d // 16, 16) * torch.from_numpy(E4M3).cuda()[e]).reshape(val.shape)
    return (val * 2.0 ** s["exps"][part]).permute(0, 2, 1, 3).reshape(-1, raw.shape[1], d)


def _exact_read(s):
    slot = s["slot"].long()
    every = torch.arange(s["pool"].shape[0], device="cuda")
    live = (slot >= 0).double()[:, None, None]
    return {name: _blocks(s, every, i)[slot.clamp(min=0)] * live for i, name in enumerate("kv")}


def _exact_attend(s):
    c = s["case"]
    lens, q_lens = _lengths(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (length, m) in enumerate(zip(lens.tolist(), q_lens.tolist())):
        if length:
            pages = s["bt"][i, :-(-length // P)].long()
            k, v = (_blocks(s, pages, part)[:length].permute(1, 0, 2) for part in (0, 1))  # [h, positions, d]
            q = s["q"][at:at + m].double().reshape(m, c["n_kv"], -1, c["d"]).permute(1, 2, 0, 3)
            x = torch.einsum("hgmd,hnd->hgmn", q, k) * c["d"] ** -0.5
            x = x + torch.triu(torch.full((m, length), -math.inf, dtype=torch.float64, device="cuda"), diagonal=length - m + 1)
            out[at:at + m] = torch.einsum("hgmn,hnd->mhgd", torch.softmax(x, -1), v).reshape(m, -1, c["d"])
        at += m
    return out
