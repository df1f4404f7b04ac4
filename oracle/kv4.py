"""The 4-bit KV cache and its operators in float64 on the CPU.

A block is 16 channels of one (position, KV head) of K or V.  With the exponent
E of K or V: a = max |x_i|, s = e4m3(a / (6 * 2^E)), n_i = e2m1(x_i / (s * 2^E)),
nearest with ties to the even code, saturating; n_i = 0 where s = 0, and a zero
code has no sign; a NaN makes s NaN; the block stands for n_i * s * 2^E.  A pool is uint8
[num_pages, n_kv, 2, 9 d]: 16 rows of d / 2 code bytes (channel 2i in the low
half of byte i), then 16 rows of d / 16 scale bytes.

Everything here goes element by element through tables of the formats' values;
nothing is shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from oracle.layer import rope

P = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])  # codes 0 .. 126; 127 is NaN


def nearest(x, grid):
    """Codes of the grid values nearest to the magnitudes x; ties to the even code; saturating."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    up, down = grid[hi] - x, x - grid[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x, exp):
    """x [..., d] -> (codes uint8 [..., d] in 0 .. 15, scale bytes uint8 [..., d / 16])."""
    y = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 16) * 2.0 ** -exp
    bad = np.isnan(y).any(-1)
    a = np.abs(np.where(np.isnan(y), 0.0, y))
    top = np.minimum(a.max(-1) / 6, 1e9)
    s = nearest(top, E4M3)
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.where(E4M3[s][..., None] > 0, np.minimum(a / E4M3[s][..., None], 1e9), 0.0)
    n = nearest(u, E2M1)
    n |= ((n > 0) & np.signbit(y)) << 3  # a zero has no sign
    n = np.where(bad[..., None] | (s == 0)[..., None], 0, n)
    return n.reshape(x.shape).astype(np.uint8), np.where(bad, 127, s).astype(np.uint8)


def values(codes, scales, exp):
    """The float64 values that codes [..., d] and scale bytes [..., d / 16] stand for."""
    e = np.concatenate([E4M3, [np.nan]])
    s = np.where(scales & 128, -1.0, 1.0) * e[scales & 127]
    n = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    return n * np.repeat(s, 16, -1) * 2.0 ** exp


def put(pool, slot, part, codes, scales):
    """Store the codes [n_kv, d] and scales [n_kv, d / 16] of one token in a pool (numpy, in place)."""
    d = codes.shape[-1]
    page, row = slot // P, slot % P
    pool[page, :, part, row * d // 2:(row + 1) * d // 2] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    pool[page, :, part, 8 * d + row * d // 16:8 * d + (row + 1) * d // 16] = scales


def take(pool, slots, part, exp):
    """Values [n, n_kv, d] of the slots; zeros for a slot outside the pool."""
    d = pool.shape[-1] // 9
    out = np.zeros((len(slots), pool.shape[1], d))
    for i, slot in enumerate(slots):
        if 0 <= slot < pool.shape[0] * P:
            page, row = slot // P, slot % P
            b = pool[page, :, part, row * d // 2:(row + 1) * d // 2]
            codes = np.stack([b & 15, b >> 4], -1).reshape(len(b), d)
            out[i] = values(codes, pool[page, :, part, 8 * d + row * d // 16:8 * d + (row + 1) * d // 16], exp)
    return out


def norm_rope(u, gain, pos, theta, eps):
    """u [N, heads, d] float64, gain [d] or None: RMSNorm of each head, then the rotation."""
    if gain is not None:
        u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * gain
    return rope(u, np.asarray(pos), theta)


def block_tables(held, lens, table, ring, state, caps):
    """nf_block_tables, request by request: returns a dict of the outputs.  table, ring,
    and caps = (tok_seq, tok_pos, tok_slot) as before the call are not modified."""
    most = table.shape[1] * P
    held, lens = np.clip(held, 0, most).tolist(), np.clip(lens, 0, most).tolist()
    head, count = int(state[0]), int(state[1])
    pages = lambda n: -(-n // P)  # noqa: E731
    need = sum(max(0, pages(b) - pages(a)) for a, b in zip(held, lens))
    short = need > count
    out, r = table.copy(), ring.copy()
    rows = [c.copy() for c in caps]
    begin, taken, given, tok = [], 0, 0, 0
    for s, (a, b) in enumerate(zip(held, lens)):
        begin.append(tok)
        for j in range(pages(a), pages(b)):
            out[s, j] = -1 if short else ring[(head + taken) % len(ring)]
            taken += 1
        for j in range(pages(b), pages(a)):
            if not short and count + given < len(ring):
                r[(head + count + given) % len(ring)] = table[s, j]
            given += 1
        for pos in range(a, b):
            page = out[s, pos // P]
            if tok < len(rows[0]):
                rows[0][tok], rows[1][tok] = s, pos
                rows[2][tok] = page * P + pos % P if 0 <= page < len(ring) else -1
            tok += 1
    begin.append(tok)
    state = [head, count, tok, need - count] if short else \
        [(head + taken) % len(ring), min(count - taken + given, len(ring)), tok, 0]
    return dict(block_table=out, ring=r, state_out=np.array(state), tok_begin=np.array(begin),
                tok_seq=rows[0], tok_pos=rows[1], tok_slot=rows[2])


def attention(q, pool, exps, block_table, lens, q_lens):
    """o [T, n_q, d] float64, and for every output the weighted mean of |v| (for error bounds):
    the rows of request s sit at its last q_lens[s] positions and see what lies at or before them."""
    d = pool.shape[-1] // 9
    n_kv = pool.shape[1]
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    at = 0
    for s, (n, m) in enumerate(zip(lens, q_lens)):
        n, m = int(n), int(m)
        if n > 0:
            slots = np.concatenate([block_table[s, j] * P + np.arange(P) for j in range(-(-n // P))])[:n]
            k, v = (take(pool, slots, i, exps[i]) for i in (0, 1))
            for i in range(m):
                see = n - m + i + 1
                if see <= 0:
                    continue
                x = np.einsum("hgd,nhd->hgn", q[at + i].reshape(n_kv, -1, d), k[:see]) / np.sqrt(d)
                w = np.exp(x - x.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                o[at + i] = np.einsum("hgn,nhd->hgd", w, v[:see]).reshape(-1, d)
                mag[at + i] = np.einsum("hgn,nhd->hgd", w, np.abs(v[:see])).reshape(-1, d)
        at += m
    return o, mag
