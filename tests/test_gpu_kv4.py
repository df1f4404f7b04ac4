"""The 4-bit KV cache's operators on the GPU against the float64 oracle.

Integers and what 4 bits hold are compared exactly.  Bounds of bf16 outputs:

* q (and k in a 16-bit cache) is rounded once: half a step, 2^-8 of the value;
  the fp32 norm, rotation and their products err by at most 2^-19 of the pair's
  magnitude before it, at most 2^-18 of the head's largest value.
* attention: the stored output half a step; the weights enter the product in
  fp16 (2^-11 each, so 2^-11 of the weighted mean of |v|); a score's fp32 sum of
  d products errs by at most d 2^-24 of sum |q k| (each product is exact), its
  exponential by that much relative, and 2^ex by 2^-22: together
  (2^-11 + 2 (d 2^-24 max_j sum |q k_j| / sqrt(d)) + 2^-20) of the weighted mean
  of |v|, the factor 2 for numerator and denominator.  A weight is held in fp16
  as 2^7 of its share of the largest one seen, so it also errs by half of
  fp16's smallest step, 2^-25, over 2^7: n 2^-32 max |v| over n positions (a
  row whose heavy positions all hold zeros shows nothing but those).
"""
import numpy as np
import pytest
import torch

from nano_intra_device_gb300 import _lib, workload as wl
from oracle import kv4 as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"


def shape_of(n_q, n_kv, d, theta=1e4, eps=1e-5):
    return wl.Shape(hidden=n_q * d, n_q=n_q, n_kv=n_kv, head_dim=d, ffn=16, rms_eps=eps, rope_theta=theta)


def dev32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def host(t):
    return t.detach().cpu().numpy()


# ------------------------------------------------------------------ block tables

def make_tables(r, n, width, num, held, head, tok_cap):
    """A consistent state: shuffled pages, the free ones in the ring from `head`."""
    perm, used = r.permutation(num), 0
    table = r.integers(-3, num + 3, (n, width))  # entries past the end may hold anything
    for s in range(n):
        k = -(-int(held[s]) // 16)
        table[s, :k] = perm[used:used + k]
        used += k
    ring = np.full(num, -7)
    ring[(head + np.arange(num - used)) % num] = perm[used:]
    return table, ring, num - used, [np.full(tok_cap, -5 - i) for i in range(3)]


def run_tables(held, lens, table, ring, state, rows, twice=True):
    n = len(held)
    t = dict(held=dev32(held), seq_lens=dev32(lens), block_table=dev32(table), ring=dev32(ring), state_in=dev32(state),
             state_out=dev32([-9] * 4), tok_begin=dev32([-9] * (n + 1)), tok_seq=dev32(rows[0]), tok_pos=dev32(rows[1]), tok_slot=dev32(rows[2]))
    args = _lib.BlockTables(**t)
    for _ in range(2 if twice else 1):  # repeating a call changes nothing
        _lib.block_tables(args)
    want = orc.block_tables(held, lens, table, ring, state, rows)
    for k, w in want.items():
        assert np.array_equal(host(t[k]), w), k
    return t, want


@pytest.mark.parametrize("n,width,kind", [(1, 1, "grow"), (1, 9, "mixed"), (3, 4, "mixed"), (31, 8, "end"), (64, 64, "decode"), (511, 5, "mixed"),
                                          (512, 5, "mixed"), (513, 5, "mixed"), (700, 300, "prompts"), (1025, 3, "mixed"), (5000, 4, "decode"),
                                          (17, 600, "prompts")])
@pytest.mark.parametrize("seed", [0, 1])
def test_block_tables(n, width, kind, seed):
    r = np.random.default_rng(1000 * seed + n)
    most = width * 16
    held = r.integers(0, most + 1, n)
    lens = {"grow": np.minimum(held + 17, most), "mixed": r.integers(0, most + 1, n), "end": np.where(r.random(n) < 0.5, 0, held),
            "decode": np.minimum(held + 1, most), "prompts": np.where(r.random(n) < 0.3, held, r.integers(0, most + 1, n))}[kind]
    if kind == "prompts":
        held[::3] = 0
    num = int((-(-np.maximum(held, lens) // 16)).sum()) + 3
    tok = int(np.clip(lens - held, 0, None).sum())
    head = int(r.integers(0, num))
    table, ring, free, rows = make_tables(r, n, width, num, held, head, tok + 5)
    _, want = run_tables(held, lens, table, ring, (head, free), rows)
    assert want["state_out"][3] == 0 and want["state_out"][2] == tok


def test_block_tables_of_a_large_batch():
    """Tens of thousands of requests and tokens, some prompts of thousands."""
    r = np.random.default_rng(21)
    n, width = 20000, 300
    held = r.integers(0, 200, n)
    lens = np.where(r.random(n) < 0.9, held + 1, r.integers(0, 200, n))
    lens[r.integers(0, n, 40)] = 4800
    num = int((-(-np.maximum(held, lens) // 16)).sum()) + 3
    table, ring, free, rows = make_tables(r, n, width, num, held, num - 5, int(np.clip(lens - held, 0, None).sum()))
    run_tables(held, lens, table, ring, (num - 5, free), rows)


def test_block_tables_short_ring_changes_nothing():
    r = np.random.default_rng(5)
    held, lens = np.array([5, 16, 40, 30]), np.array([6, 33, 0, 200])
    table, ring, free, rows = make_tables(r, 4, 13, 14, held, 9, 300)
    t, want = run_tables(held, lens, table, ring, (9, free), rows)
    assert want["state_out"].tolist() == [9, free, 1 + 17 + 170, 2 + 11 - free] and np.array_equal(host(t["ring"]), ring)
    # positions 5 and 30, 31 lie in pages held before (1 and 2 pages); every other one has none
    assert np.flatnonzero(host(t["tok_slot"])[:188] >= 0).tolist() == [0, 18, 19]


def test_block_tables_bad_inputs_stay_inside():
    r = np.random.default_rng(6)
    n, width, num = 40, 5, 300
    held = r.integers(0, 81, n)
    table, ring, free, rows = make_tables(r, n, width, num, held, 250, 50)  # fewer token rows than tokens
    held[3], held[4] = -5, 10 ** 6  # clamped; request 4's pages past the end are whatever the table holds
    lens = np.where(r.random(n) < 0.5, 2 ** 31 - 1, -(2 ** 31))
    run_tables(held, lens, table, ring, (250, free), rows)
    table[:] = r.integers(-2 ** 31, 2 ** 31 - 1, table.shape)  # ids outside the pool give slot -1
    ring[:] = r.integers(-2 ** 31, 2 ** 31 - 1, ring.shape)
    run_tables(np.full(n, 3), np.full(n, 40), table, ring, (299, 300), rows)
    run_tables(np.full(n, 33), np.full(n, 3), table, ring, (0, 250), rows)  # more given back than the ring has room for


def test_block_tables_steps_in_one_graph():
    """Growth step by step in a captured graph, the state ping-ponging between two buffers."""
    n, width, num = 33, 4, 140
    held = np.arange(n) % 20
    r = np.random.default_rng(7)
    table, ring, free, rows = make_tables(r, n, width, num, held, 0, n)
    bt, rg = dev32(table), dev32(ring)
    lens = [dev32(held + i) for i in range(3)]
    st = [dev32([0, free]), dev32([0, 0, 0, 0]), dev32([0] * 4)]
    tok = [dev32(x) for x in rows]
    begin = dev32([0] * (n + 1))
    a = _lib.BlockTables(lens[0], lens[1], bt, rg, st[0], st[1], begin, *tok)
    b = _lib.BlockTables(lens[1], lens[2], bt, rg, st[1][:2], st[2], begin, *tok)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _lib.block_tables(a)
        _lib.block_tables(b)
    g.replay()
    w1 = orc.block_tables(held, held + 1, table, ring, (0, free), rows)
    w2 = orc.block_tables(held + 1, held + 2, w1["block_table"], w1["ring"], w1["state_out"][:2], [w1[k] for k in ("tok_seq", "tok_pos", "tok_slot")])
    for t, k in ((bt, "block_table"), (rg, "ring"), (st[2], "state_out"), (tok[2], "tok_slot"), (begin, "tok_begin")):
        assert np.array_equal(host(t), w2[k]), k


# ------------------------------------------------------------------ norm, rotation, append

def append_case(r, n_tok, n_q, n_kv, d, num_pages, pos_max, scale=1.0, pad=0):
    width = (n_q + 2 * n_kv) * d
    x = torch.from_numpy(r.standard_normal((n_tok, width + pad)) * scale).to(torch.bfloat16)
    pos = r.integers(0, pos_max, n_tok)
    slot = r.permutation(num_pages * 16)[:n_tok]
    return x, pos, slot


def check_append(shape, x, gains, pos, slot, fmt, num_pages, exps=(0, 0), seed=9):
    """Run the call, compare q, every byte of the cache and what lies beside it with the oracle."""
    n_q, n_kv, d = shape.n_q, shape.n_kv, shape.head_dim
    n = x.shape[0]
    width = (n_q + 2 * n_kv) * d
    xd = x.to(DEV)
    gd = [None if g is None else g.to(DEV) for g in gains]
    q = torch.full((n + 1, n_q, d), 7.0, dtype=torch.bfloat16, device=DEV)
    u = x[:, :width].double().numpy().reshape(n, -1, d)
    g64 = [None if g is None else g.double().numpy() for g in gains]
    eps = float(np.float32(shape.rms_eps))
    theta = float(np.float32(shape.rope_theta))
    with np.errstate(all="ignore"):
        wq = orc.norm_rope(u[:, :n_q], g64[0], pos, theta, eps)
        wk = orc.norm_rope(u[:, n_q:n_q + n_kv], g64[1], pos, theta, eps)
    wv = u[:, n_q + n_kv:]
    inside = [i for i in range(n) if 0 <= slot[i] < num_pages * 16]
    g = torch.Generator().manual_seed(seed)
    if fmt == _lib.NF_KV_FP4:
        pool = torch.randint(0, 256, (num_pages, n_kv, 2, 9 * d), dtype=torch.uint8, generator=g)
        want = pool.numpy().copy()
        for i in inside:
            for part, w in ((0, wk), (1, wv)):
                orc.put(want, int(slot[i]), part, *orc.quantise(w[i], exps[part]))
        pd = pool.to(DEV)
        cache = _lib.KvCache(shape, num_pages, fmt, pd, None, *exps)
    else:
        kp, vp = (torch.randn(num_pages, n_kv, 16, d, generator=g).to(torch.bfloat16) for _ in range(2))
        kd, vd = kp.to(DEV), vp.to(DEV)
        cache = _lib.KvCache(shape, num_pages, fmt, kd, vd)
    _lib.qk_norm_rope(shape, xd, gd[0], gd[1], dev32(pos), dev32(slot), q[:n], cache)

    def near(got, ref, name):
        bad = ~np.isfinite(ref)
        assert np.array_equal(np.isnan(got), np.isnan(ref)), name
        big = np.abs(np.where(bad, 0, ref)).max(-1, keepdims=True)
        bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * big + 1e-37
        off = np.abs(got[~bad] - ref[~bad])
        assert (off <= bound[~bad]).all(), (name, off.max())

    got_q = q.double().cpu().numpy()
    near(got_q[:n], wq, "q")
    assert (got_q[n] == 7.0).all()
    if fmt == _lib.NF_KV_FP4:
        got = host(pd)
        if not np.array_equal(got, want):
            at = np.argwhere(got != want)
            raise AssertionError(f"{len(at)} bytes differ, first at {at[0]}: {got[tuple(at[0])]:#x}, want {want[tuple(at[0])]:#x}")
        return pd, cache
    for t, src, w, name in ((kd, kp, wk, "k"), (vd, vp, wv, "v")):
        got = t.double().cpu().numpy()
        ref = src.double().numpy().copy()
        for i in inside:
            near(got[slot[i] // 16, :, slot[i] % 16], w[i], name)
            ref[slot[i] // 16, :, slot[i] % 16] = got[slot[i] // 16, :, slot[i] % 16]
        assert np.array_equal(got, ref, equal_nan=True), name


def gains_of(r, d, kind="both"):
    g = [torch.from_numpy(1 + 0.3 * r.standard_normal(d)).to(torch.bfloat16) for _ in range(2)]
    return [g[0] if kind in ("both", "q") else None, g[1] if kind in ("both", "k") else None]


@pytest.mark.parametrize("fmt", [_lib.NF_KV_FP4, _lib.NF_KV_BF16])
@pytest.mark.parametrize("n_q,n_kv,d", [(1, 1, 64), (2, 2, 128), (4, 2, 64), (8, 1, 128), (32, 8, 128), (12, 3, 64), (5, 5, 128), (56, 7, 64)])
@pytest.mark.parametrize("n_tok", [1, 3, 17, 150])
def test_append(fmt, n_q, n_kv, d, n_tok):
    r = np.random.default_rng(n_tok * 7 + n_q + d)
    x, pos, slot = append_case(r, n_tok, n_q, n_kv, d, 13, 5000)
    if n_tok > 3:
        slot[1], slot[2], pos[0] = -1, 13 * 16, 0
    check_append(shape_of(n_q, n_kv, d), x, gains_of(r, d), pos, slot, fmt, 13, (0, 1))


@pytest.mark.parametrize("n_tok", [700, 2500])
def test_append_many_tokens(n_tok):
    """Enough tokens for every number of tokens a CTA takes."""
    r = np.random.default_rng(n_tok)
    x, pos, slot = append_case(r, n_tok, 2, 1, 64, n_tok // 16 + 1, 5000)
    check_append(shape_of(2, 1, 64), x, gains_of(r, 64), pos, slot, _lib.NF_KV_FP4, n_tok // 16 + 1)


@pytest.mark.parametrize("fmt", [_lib.NF_KV_FP4, _lib.NF_KV_BF16])
@pytest.mark.parametrize("n_q,n_kv,d", [(2, 1, 64), (8, 4, 128), (16, 8, 64)])
@pytest.mark.parametrize("per_sm,more", [(6, -1), (6, 0), (6, 5), (12, -1), (12, 0), (12, 3), (24, -1), (24, 0), (24, 5)])
def test_append_on_both_sides_of_every_number_of_tokens_a_cta_takes(per_sm, more, n_q, n_kv, d, fmt):
    """One token a CTA below 6 an SM, then 2, from 12 on 4, from 24 on 8, there in two launches where whole
    warps of heads are queries or keys (the last two shapes), with odd tails."""
    n_tok = per_sm * torch.cuda.get_device_properties(0).multi_processor_count + more
    r = np.random.default_rng(n_tok + d)
    x, pos, slot = append_case(r, n_tok, n_q, n_kv, d, n_tok // 16 + 2, 5000)
    slot[3::101] = -1
    check_append(shape_of(n_q, n_kv, d), x, gains_of(r, d), pos, slot, fmt, n_tok // 16 + 2, (1, -1))


@pytest.mark.parametrize("fmt", [_lib.NF_KV_FP4, _lib.NF_KV_BF16])
@pytest.mark.parametrize("n_tok,n_q,n_kv,d", [(3700, 8, 8, 64), (5001, 8, 2, 128), (4000, 16, 4, 64)])
def test_append_of_thousands(fmt, n_tok, n_q, n_kv, d):
    r = np.random.default_rng(n_tok)
    x, pos, slot = append_case(r, n_tok, n_q, n_kv, d, n_tok // 16 + 2, 5000)
    slot[5::97] = -1
    check_append(shape_of(n_q, n_kv, d), x, gains_of(r, d), pos, slot, fmt, n_tok // 16 + 2, (-1, 2))


@pytest.mark.parametrize("n_tok", [40, 4500])
def test_append_in_a_graph_and_on_another_stream(n_tok):
    r = np.random.default_rng(n_tok)
    n_q, n_kv, d, num = 8, 4, 128, n_tok // 16 + 2
    shape = shape_of(n_q, n_kv, d)
    x, pos, slot = append_case(r, n_tok, n_q, n_kv, d, num, 5000)
    g = [t.to(DEV) for t in gains_of(r, d)]
    xd, pd, sd = x.to(DEV), dev32(pos), dev32(slot)
    side = torch.cuda.Stream()
    outs = []
    for way in ("plain", "graph", "stream"):
        pool = torch.zeros(num, n_kv, 2, 9 * d, dtype=torch.uint8, device=DEV)
        q, k, v = (torch.zeros(n_tok, h, d, dtype=torch.bfloat16, device=DEV) for h in (n_q, n_kv, n_kv))
        cache = _lib.KvCache(shape, num, _lib.NF_KV_FP4, pool)

        def run(stream=None):
            _lib.qk_norm_rope(shape, xd, g[0], g[1], pd, sd, q, cache, stream=stream)
            _lib.kv4_read(shape, cache, sd, k, v, stream=stream)  # behind the append, whatever it launches
        torch.cuda.synchronize()
        if way == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
            for _ in range(3):
                pool.zero_()
                q.zero_()
                graph.replay()
        else:
            run(side if way == "stream" else None)
        torch.cuda.synchronize()
        outs.append([pool, q, k, v])
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    assert outs[0][2].any() and outs[0][3].any()


@pytest.mark.parametrize("kind", ["none", "q", "k"])
@pytest.mark.parametrize("fmt", [_lib.NF_KV_FP4, _lib.NF_KV_BF16])
def test_append_gains_are_optional_and_rows_may_be_strided(kind, fmt):
    r = np.random.default_rng(3)
    x, pos, slot = append_case(r, 37, 4, 2, 128, 5, 100, pad=40)
    check_append(shape_of(4, 2, 128), x, gains_of(r, 128, kind), pos, slot, fmt, 5)


def test_append_far_and_negative_positions():
    r = np.random.default_rng(4)
    x, pos, slot = append_case(r, 40, 2, 2, 64, 5, 100)
    pos[:20] = [2 ** 17, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 31 - 1, -1, -2 ** 31, -77, 10 ** 9, 2 ** 30 + 3, 131071] * 2
    for theta in (1e4, 5e5, 0.5):
        check_append(shape_of(2, 2, 64, theta), x, gains_of(r, 64), pos, slot, _lib.NF_KV_FP4, 5)
        check_append(shape_of(2, 2, 64, theta), x, gains_of(r, 64), pos, slot, _lib.NF_KV_BF16, 5)


@pytest.mark.parametrize("exps", [(0, 0), (3, -2), (-20, 20), (64, -64)])
@pytest.mark.parametrize("scale", [1e-6, 1.0, 3e4])
def test_append_exponents_and_magnitudes(exps, scale):
    r = np.random.default_rng(5)
    x, pos, slot = append_case(r, 30, 2, 2, 64, 4, 9, scale)
    check_append(shape_of(2, 2, 64), x, gains_of(r, 64, "q"), pos, slot, _lib.NF_KV_FP4, 4, exps)


def test_append_ties_and_borders():
    """Values that lie exactly on the borders between codes and between scales: unrotated K (position 0,
    no gain) is exact in fp32, V always is."""
    r = np.random.default_rng(6)
    d, n = 64, 200
    u = r.choice([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 0, 0.251, 4.98], (n, 6, d)) * r.choice([-1, 1], (n, 6, d))
    s = r.choice([1.0, 0.5, 1.125, 1.375, 0.0625, 2.0 ** -9, 3 * 2.0 ** -9, 448.0, 500.0], (n, 6, d // 16))
    x = torch.from_numpy((u * np.repeat(s, 16, -1)).reshape(n, -1)).to(torch.bfloat16)
    # blocks whose largest magnitude is six times the middle of two scales
    mid = (orc.E4M3[1:] + orc.E4M3[:-1]) / 2 * 6
    x.view(n, 6, d)[:126, 2, 5] = torch.from_numpy(mid).to(torch.bfloat16)
    x.view(n, 6, d)[:126, 4, 7] = torch.from_numpy(mid).to(torch.bfloat16)
    check_append(shape_of(2, 2, d), x, [None, None], np.zeros(n, int), r.permutation(16 * 13)[:n], _lib.NF_KV_FP4, 13)


def test_append_nan_inf_and_zero_rows():
    r = np.random.default_rng(7)
    x, pos, slot = append_case(r, 20, 2, 2, 64, 3, 50)
    h = x.view(20, 6, 64)
    h[0] = 0.0
    h[1, :, 3] = float("nan")
    h[2, 4:, 9] = float("inf")    # V saturates
    h[3, 4:, 40] = -float("inf")
    h[4, 4, :] = -0.0
    h[6, 2, 11] = float("inf")    # a key's pair, and with it two blocks, to infinity or NaN
    h[7, 3, 40] = -float("inf")
    pos[7] = 0
    h[5, 5, :16] = float("nan")
    for fmt in (_lib.NF_KV_FP4, _lib.NF_KV_BF16):
        for kind in ("both", "none"):
            check_append(shape_of(2, 2, 64), x, gains_of(r, 64, kind), pos, slot, fmt, 3)


def test_append_codes_are_those_of_64_bits():
    """Two million rotated keys: some lie within the fp32 error of a border."""
    r = np.random.default_rng(8)
    x, pos, slot = append_case(r, 2000, 8, 8, 128, 130, 10 ** 5)
    check_append(shape_of(8, 8, 128, 5e5), x, gains_of(r, 128), pos, slot, _lib.NF_KV_FP4, 130)


# ------------------------------------------------------------------ rows by slot

@pytest.mark.parametrize("n_kv,d", [(1, 64), (3, 128), (8, 64), (8, 128)])
@pytest.mark.parametrize("n", [1, 5, 1000])
@pytest.mark.parametrize("exps", [(0, 0), (-7, 30)])
def test_read(n_kv, d, n, exps):
    r = np.random.default_rng(n + d)
    pool = r.integers(0, 256, (9, n_kv, 2, 9 * d)).astype(np.uint8)
    slots = r.integers(0, 9 * 16, n)  # the same slot may come twice
    slots[n // 2] = [-1, 9 * 16, 2 ** 31 - 1, -2 ** 31][n % 4]
    k, v = (torch.full((n + 1, n_kv, d), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = _lib.KvCache(shape_of(n_kv, n_kv, d), 9, _lib.NF_KV_FP4, torch.from_numpy(pool).to(DEV), None, *exps)
    _lib.kv4_read(shape_of(n_kv, n_kv, d), cache, dev32(slots), k[:n], v[:n])
    for t, part in ((k, 0), (v, 1)):
        got = t.double().cpu().numpy()
        assert np.array_equal(got[:n], orc.take(pool, slots, part, exps[part]), equal_nan=True)
        assert (got[n] == 3.0).all()


# ------------------------------------------------------------------ attention

def filled_pool(r, num_pages, n_kv, d, nan_slots=()):
    """Blocks as unit normals give them; the slots listed hold NaN scales and random codes."""
    pool = r.integers(0, 256, (num_pages, n_kv, 2, 9 * d)).astype(np.uint8)
    s = torch.from_numpy(r.uniform(0.2, 0.6, (num_pages, n_kv, 2, d))).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    pool[..., 8 * d:] = s
    for slot in nan_slots:
        row = slot % 16
        pool[slot // 16, :, :, 8 * d + row * d // 16:8 * d + (row + 1) * d // 16] = r.choice([0x7F, 0xFF])
    return pool


def attention_case(r, n_q, n_kv, d, lens, q_lens, q_scale=1.0, spare=2, width=None):
    """Shuffled pages; every slot that no position of a request owns holds NaN."""
    lens, q_lens = np.asarray(lens), np.asarray(q_lens)
    need = -(-lens // 16)
    num = int(need.sum()) + spare
    perm = r.permutation(num)
    width = max(1, int(need.max())) if width is None else width
    bt, used, owned = np.full((len(lens), width), -1), 0, set()
    for s, n in enumerate(lens):
        bt[s, :need[s]] = perm[used:used + need[s]]
        used += need[s]
        owned |= {int(bt[s, p // 16]) * 16 + p % 16 for p in range(n)}
    pool = filled_pool(r, num, n_kv, d, [x for x in range(num * 16) if x not in owned])
    q = torch.from_numpy(r.standard_normal((int(q_lens.sum()), n_q, d)) * q_scale).to(torch.bfloat16)
    return pool, bt, q


def run_attention(shape, pool, bt, q, lens, q_lens, exps=(0, 0), begin=None, pad_rows=0, handle=None, poll=True):
    n = q.shape[0]
    h = handle or _lib.Kv4(shape, pool.shape[0], bt.shape[1])
    o = torch.full((n + pad_rows + 1, shape.n_q, shape.head_dim), 5.0, dtype=torch.bfloat16, device=DEV)
    qd = torch.zeros(n + pad_rows, shape.n_q, shape.head_dim, dtype=torch.bfloat16, device=DEV)
    qd[:n] = q.to(DEV)
    if begin is None and (np.any(np.asarray(q_lens) != 1) or pad_rows):
        begin = np.concatenate([[0], np.cumsum(q_lens)])
    cache = _lib.KvCache(shape, pool.shape[0], _lib.NF_KV_FP4, torch.from_numpy(pool).to(DEV), None, *exps)
    _lib.attention_kv4(h, qd, cache, dev32(bt), dev32(lens), o[:n + pad_rows], None if begin is None else dev32(begin))
    if poll:
        h.poll()
    assert (host(o.float())[n:] == 5.0).all()  # rows behind the last request stay
    return o[:n].double().cpu().numpy()


def check_attention(shape, pool, bt, q, lens, q_lens, exps=(0, 0), **kw):
    got = run_attention(shape, pool, bt, q, lens, q_lens, exps, **kw)
    q64 = q.double().numpy()
    want, mag = orc.attention(q64, pool, exps, bt, lens, q_lens)
    d = shape.head_dim
    # sum |q k| of a score is at most sum |q| * the largest |k|
    top, vtop = (np.nan_to_num(np.abs(orc.take(pool, range(pool.shape[0] * 16), i, exps[i]))).max() for i in (0, 1))
    mass = np.abs(q64).sum(-1, keepdims=True) * top / np.sqrt(d)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * d * 2.0 ** -24 * mass) * mag
    bound += max(lens) * 2.0 ** -32 * vtop
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) - bound).max()
    assert worst <= 0, (worst, np.abs(got - want).max())
    return got


HEADS = [(1, 1, 64), (2, 1, 128), (4, 1, 64), (8, 1, 128), (16, 2, 64), (32, 8, 128), (6, 3, 128), (24, 3, 64), (12, 3, 64), (5, 5, 128)]


@pytest.mark.parametrize("n_q,n_kv,d", HEADS)
@pytest.mark.parametrize("lens", [[1], [16], [17], [0], [2, 0, 15, 33, 16, 47, 1], [300, 129, 1, 64, 77]])
def test_attention_decode(n_q, n_kv, d, lens):
    r = np.random.default_rng(n_q * 100 + len(lens) + d)
    case = attention_case(r, n_q, n_kv, d, lens, [1] * len(lens))
    got = check_attention(shape_of(n_q, n_kv, d), *case, lens, [1] * len(lens))
    assert not got[np.asarray(lens) == 0].any()


@pytest.mark.parametrize("n_q,n_kv,d", [(4, 4, 64), (8, 1, 128), (4, 2, 128), (16, 4, 64)])
@pytest.mark.parametrize("length", [2047, 2049, 5003])
def test_attention_one_long_row(n_q, n_kv, d, length):
    r = np.random.default_rng(length)
    check_attention(shape_of(n_q, n_kv, d), *attention_case(r, n_q, n_kv, d, [length], [1]), [length], [1])


@pytest.mark.parametrize("n", [40, 333, 1500])
def test_attention_many_rows(n):
    r = np.random.default_rng(n)
    lens = np.clip(np.rint(20 * np.exp(r.standard_normal(n))), 0, 300).astype(int)
    lens[::7] = 0
    check_attention(shape_of(4, 2, 64), *attention_case(r, 4, 2, 64, lens, [1] * n), lens, [1] * n)


WIDE = 40000  # pages a request may have: chunks of a few rows on go to the tiles, with None to the kernel of few rows


@pytest.mark.parametrize("width", [None, WIDE])
@pytest.mark.parametrize("n_q,n_kv,d", [(1, 1, 64), (2, 1, 128), (8, 2, 128), (8, 1, 64), (8, 8, 128)])
@pytest.mark.parametrize("lens,q_lens", [([2], [2]), ([9], [9]), ([40, 7], [3, 7]), ([5, 130, 1, 0, 17], [1, 5, 1, 2, 17]),
                                         ([200, 64, 300], [127, 64, 129]), ([3, 500], [5, 33]), ([1000], [40])])
def test_attention_chunks(n_q, n_kv, d, lens, q_lens, width):
    """Chunks from two rows on, whole prompts and continued ones; more rows than positions (zeros first)."""
    r = np.random.default_rng(sum(lens) + n_q)
    got = check_attention(shape_of(n_q, n_kv, d), *attention_case(r, n_q, n_kv, d, lens, q_lens, width=width), lens, q_lens)
    at = 0
    for n, m in zip(lens, q_lens):
        assert not got[at:at + max(0, m - n)].any()
        at += m


@pytest.mark.parametrize("width", [9, WIDE])
def test_attention_padded_batch_and_empty_requests(width):
    r = np.random.default_rng(11)
    lens, q_lens = [50, 0, 33, 20], [3, 0, 1, 20]
    case = attention_case(r, 4, 2, 64, lens, q_lens, width=width)
    check_attention(shape_of(4, 2, 64), *case, lens, q_lens, pad_rows=13)


@pytest.mark.parametrize("width", [None, WIDE])
@pytest.mark.parametrize("exps", [(0, 0), (2, -3), (-5, 20)])
@pytest.mark.parametrize("q_scale", [1e-4, 1.0, 30.0, 1e18])
def test_attention_magnitudes(exps, q_scale, width):
    """Flat to one-hot weights; queries far outside fp16's range."""
    r = np.random.default_rng(12)
    lens, q_lens = [120, 1, 16, 100], [1, 1, 1, 50]
    scale = q_scale if q_scale < 1e10 else 1.0
    pool, bt, q = attention_case(r, 4, 2, 64, lens, q_lens, scale, width=width)
    if q_scale > 1e10:  # one row large, where its scores stay apart: one-hot
        q[0] = (q[0].float() * q_scale).to(torch.bfloat16)
        q[1] = (q[1].float() / q_scale).to(torch.bfloat16)
        shape = shape_of(4, 2, 64)
        got = run_attention(shape, pool, bt, q, lens, q_lens, exps)
        want, _ = orc.attention(q.double().numpy(), pool, exps, bt, lens, q_lens)
        # scores of row 0 differ by far more than fp32's error, or tie exactly
        assert np.abs(got[0] - want[0]).max() <= 2.0 ** -8 * np.abs(want[0]).max()
        assert np.abs(got[1] - want[1]).max() <= 2.0 ** -8 * np.abs(want[1]).max()
        return
    check_attention(shape_of(4, 2, 64), pool, bt, q, lens, q_lens, exps)


@pytest.mark.parametrize("width", [None, WIDE])
@pytest.mark.parametrize("exps", [(0, 0), (-5, 20)])
def test_attention_extreme_queries_inside_a_chunk(exps, width):
    """Rows of a chunk 10^18 times larger and smaller than their neighbours, in one call.

    A huge row's weights are one-hot where its two largest scores lie further apart than twice a score's error
    (d 2^-24 of its mass, as above) and 20 more: e^-20 is far below the output's half step.  A tiny row's scores
    are all zero to 2^-50, so its output is the mean.  The others keep the ordinary bound."""
    r = np.random.default_rng(25)
    d, lens, q_lens = 64, [120, 300, 100], [1, 150, 50]
    pool, bt, q = attention_case(r, 4, 2, d, lens, q_lens, width=width)
    big, small = [0, 3, 40, 100, 149, 170, 200], [1, 17, 90, 155, 199]
    q[big] = (q[big].float() * 1e18).to(torch.bfloat16)
    q[small] = (q[small].float() * 1e-18).to(torch.bfloat16)
    shape = shape_of(4, 2, d)
    got = run_attention(shape, pool, bt, q, lens, q_lens, exps)
    q64 = q.double().numpy()
    want, mag = orc.attention(q64, pool, exps, bt, lens, q_lens)
    assert np.isfinite(got).all()
    top, vtop = (np.nan_to_num(np.abs(orc.take(pool, range(pool.shape[0] * 16), i, exps[i]))).max() for i in (0, 1))
    mass = np.abs(q64).sum(-1, keepdims=True) * top / np.sqrt(d)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * d * 2.0 ** -24 * mass) * mag + max(lens) * 2.0 ** -32 * vtop
    plain = np.setdiff1d(np.arange(len(q)), big)
    assert (np.abs(got - want) <= bound)[plain].all()
    seq = np.repeat(np.arange(3), q_lens)
    begin = np.concatenate([[0], np.cumsum(q_lens)])
    apart = 0
    for i in big:
        s = seq[i]
        see = lens[s] - q_lens[s] + i - begin[s] + 1
        k = orc.take(pool, [int(bt[s, p // 16]) * 16 + p % 16 for p in range(see)], 0, exps[0])
        for h in range(4):
            x = np.sort(k[:, h // 2] @ q64[i, h] / np.sqrt(d))
            if x[-1] - x[-2] > 2 * d * 2.0 ** -24 * mass[i, h, 0] + 20:
                apart += 1
                assert (np.abs(got[i, h] - want[i, h]) <= 2.0 ** -8 * np.abs(want[i, h]) + see * 2.0 ** -32 * vtop).all()
            else:  # whatever the weights, a mean of the values that the row sees
                assert (np.abs(got[i, h]) <= vtop * (1 + 2.0 ** -8)).all()
    assert apart >= 20


def ladder_pool(d, n, steps, value=1.5):
    """A cache of one request and KV head: K holds 2688 in channel 0 and steps[p // 64] in channel 16, V is constant."""
    pages = -(-n // 16)
    pool = np.zeros((pages, 1, 2, 9 * d), np.uint8)
    for p in range(n):
        k = np.zeros((1, d))
        k[0, 0], k[0, 16] = 2688.0, steps[p // 64]
        orc.put(pool, p, 0, *orc.quantise(k, 0))
        orc.put(pool, p, 1, *orc.quantise(np.full((1, d), value), 0))
    return pool


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("chunk", [False, True])
def test_attention_scores_in_coarse_steps(chunk, d):
    """Scores of 2^20 to 2^30, where fp32's steps reach those by which a maximum may be passed before it is
    raised: whatever the weights come to, they are finite and add up to one.  V is constant, so the output is
    that constant, up to a weight's half step in fp16 (2^-11) and the output's in bf16 (2^-8)."""
    n, steps = 300, [0.0, 1.0, 1.5, 2.0, 3.0]
    pool = ladder_pool(d, n, steps)
    rows = []
    for e in range(20, 31):
        for f in (1.0, 1.19, 1.41, 1.68):
            for b in (22.0, 36.0, 40.0, 42.0, 44.0, 45.0, 46.0, 48.0, 56.0, 64.0, 72.0, 80.0, 88.0, 90.0, 112.0, 128.0):
                rows.append((2.0 ** e * f * np.sqrt(d) / 1.4427 / 2688, b * np.sqrt(d / 64)))
    n_q = 8 if chunk else 1
    q = np.zeros((len(rows), d))
    q[:, 0], q[:, 16] = np.array(rows).T
    q = torch.from_numpy(q.reshape(-1, n_q, d)).to(torch.bfloat16)
    shape = shape_of(n_q, 1, d)
    pages = pool.shape[0]
    if chunk:  # 200 chunks of 44 rows: every CTA has several blocks of a chunk to itself
        n_seq, q_lens = 200, [44] * 200
        q = q.repeat(100, 1, 1)
        bt = np.full((n_seq, WIDE), -1)
        bt[:, :pages] = np.arange(pages)
    else:
        n_seq, q_lens = len(rows), [1] * len(rows)
        bt = np.tile(np.arange(pages), (n_seq, 1))
    got = run_attention(shape, pool, bt, q, [n] * n_seq, q_lens)
    assert np.isfinite(got).all()
    assert np.abs(got - 1.5).max() <= 1.5 * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16)


@pytest.mark.parametrize("width,q_len", [(None, 1), (None, 20), (WIDE, 20)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_attention_an_infinite_query_is_nan(bad, width, q_len):
    """Scores of one infinity, of either sign, have no softmax: NaN, also where all of them are minus infinity.
    A row that sees no position is zero all the same."""
    d = 64
    pool = ladder_pool(d, 40, [1.0])
    bt = np.full((2, width or 3), -1)
    bt[:, :3] = np.arange(3)
    lens, q_lens = [40, 5], [q_len, q_len]
    r = np.random.default_rng(24)
    q = torch.from_numpy(r.standard_normal((2 * q_len, 8, d))).to(torch.bfloat16)
    q[:, 3, 0] = bad     # against 2688 everywhere
    q[:, 5, 40] = bad    # against 0 everywhere
    got = run_attention(shape_of(8, 1, d), pool, bt, q, lens, q_lens)
    blind = np.concatenate([np.zeros(q_len, bool), np.arange(q_len) < q_len - 5])
    assert not got[blind].any()
    for h in range(8):
        assert np.isnan(got[~blind, h]).all() if h in (3, 5) else np.isfinite(got[:, h]).all()


def test_attention_sink_and_faint_tail():
    """One position far above two thousand faint ones, whose sum still counts."""
    r = np.random.default_rng(13)
    d = 64
    pool, bt, q = attention_case(r, 1, 1, d, [2000], [1])
    zero = orc.quantise(np.zeros((1, d)), 0)
    for p in range(2000):
        orc.put(pool, int(bt[0, p // 16]) * 16 + p % 16, 0, *zero)
    e = np.zeros((1, d))
    e[0, 0] = 6.0
    orc.put(pool, int(bt[0, 100]) * 16 + 7, 0, *orc.quantise(e, 0))
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16)
    q[0, 0, 0] = 16.0  # the sink's score is 12, e^-12 = 6e-6 a position beside it
    check_attention(shape_of(1, 1, d), pool, bt, q, [2000], [1])


def test_attention_bad_pages_and_lengths_are_reported():
    r = np.random.default_rng(14)
    shape = shape_of(4, 2, 64)
    lens = [40, 20]
    pool, bt, q = attention_case(r, 4, 2, 64, lens, [1, 1])
    good = bt.copy()
    h = _lib.Kv4(shape, pool.shape[0], bt.shape[1])
    for page in (pool.shape[0], -1, 2 ** 31 - 1, -2 ** 31):
        bt = good.copy()
        bt[0, 1] = page
        run_attention(shape, pool, bt, q, lens, [1, 1], handle=h, poll=False)
        with pytest.raises(_lib.NanoflowError) as e:
            h.poll()
        assert e.value.code == _lib.NF_ERR_DEVICE and "page" in str(e.value)
        h.poll()
    for n in (49, -1, 2 ** 31 - 1):
        got = run_attention(shape, pool, good, q, [n, 20], [1, 1], handle=h, poll=False)
        with pytest.raises(_lib.NanoflowError):
            h.poll()
        assert not got[0].any() and got[1].any()
    check_attention(shape, pool, good, q, lens, [1, 1], handle=h)


@pytest.mark.parametrize("width", [None, WIDE])
def test_attention_bad_rows_stay_inside(width):
    r = np.random.default_rng(15)
    shape = shape_of(4, 2, 64)
    lens = [40, 20, 30]
    pool, bt, q = attention_case(r, 4, 2, 64, lens, [2, 3, 1], width=width)
    h = _lib.Kv4(shape, pool.shape[0], bt.shape[1])
    for begin in ([0, 2, 5, 900], [0, -4, 5, 6], [2 ** 31 - 1, 2, 5, 6], [3, 2, 1, 0], [-2 ** 31, 0, 2 ** 31 - 1, 6]):
        run_attention(shape, pool, bt, q, lens, [2, 3, 1], begin=begin, handle=h, poll=False)
        with pytest.raises(_lib.NanoflowError) as e:
            h.poll()
        assert e.value.code == _lib.NF_ERR_DEVICE
    check_attention(shape, pool, bt, q, lens, [2, 3, 1], handle=h)


def test_attention_refusals():
    shape = shape_of(4, 2, 64)
    h = _lib.Kv4(shape, 8, 4)
    pool = torch.zeros(8, 2, 2, 576, dtype=torch.uint8, device=DEV)
    cache = _lib.KvCache(shape, 8, _lib.NF_KV_FP4, pool)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    bt, sl = dev32(np.zeros((2, 4))), dev32([1, 1])
    with pytest.raises(_lib.NanoflowError):
        _lib.attention_kv4(h, q, cache, bt, sl, torch.empty_like(q))  # three rows, two requests, no tok_begin
    with pytest.raises(ValueError):
        _lib.attention_kv4(h, q[:2], cache, dev32(np.zeros((2, 5))), sl, torch.empty_like(q))
    other = _lib.KvCache(shape, 7, _lib.NF_KV_FP4, pool[:7])
    with pytest.raises(_lib.NanoflowError):
        _lib.attention_kv4(h, q[:2], other, bt, sl, torch.empty_like(q))
    with pytest.raises(_lib.NanoflowError):
        _lib.attention_kv4(h, q[:2], cache, bt, sl, torch.empty_like(q).view(-1)[1:])
    bf = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(_lib.NanoflowError):
        _lib.attention_kv4(h, q[:2], _lib.KvCache(shape, 8, _lib.NF_KV_BF16, bf, bf), bt, sl, torch.empty_like(q))


@pytest.mark.parametrize("width", [None, WIDE])
def test_attention_repeats_bit_for_bit_in_a_graph_and_on_another_stream(width):
    r = np.random.default_rng(16)
    shape = shape_of(8, 2, 128)
    lens, q_lens = [700, 3, 260, 150], [1, 1, 1, 140]
    pool, bt, q = attention_case(r, 8, 2, 128, lens, q_lens, width=width)
    h = _lib.Kv4(shape, pool.shape[0], bt.shape[1])
    cache = _lib.KvCache(shape, pool.shape[0], _lib.NF_KV_FP4, torch.from_numpy(pool).to(DEV))
    qd, btd, ld = q.to(DEV), dev32(bt), dev32(lens)
    begin = dev32(np.concatenate([[0], np.cumsum(q_lens)]))
    first = torch.empty_like(qd)
    _lib.attention_kv4(h, qd, cache, btd, ld, first, begin)
    outs = [torch.empty_like(qd) for _ in range(3)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for o in outs:
            _lib.attention_kv4(h, qd, cache, btd, ld, o, begin)
    for _ in range(3):
        g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    last = torch.empty_like(qd)
    _lib.attention_kv4(h, qd, cache, btd, ld, last, begin, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    h.poll()
    for o in outs + [last]:
        assert torch.equal(o, first)


def poison(r, pool, bt, n, lo, d):
    """NaN scales in a few K and V blocks at positions [lo, n) of request 0's first and last KV head."""
    n_kv = pool.shape[1]
    for part in (0, 1, 1):
        p, g = int(r.integers(lo, n)), int(r.choice([0, n_kv - 1]))
        at = 8 * d + p % 16 * (d // 16) + int(r.integers(0, d // 16))
        pool[bt[0, p // 16], g, part, at] = r.choice([0x7F, 0xFF])


@pytest.mark.parametrize("n_q,n_kv,d", [(1, 1, 64), (4, 2, 128), (8, 2, 64), (8, 1, 128)])
@pytest.mark.parametrize("lens,q_lens", [([40], [12]), ([9], [9]), ([300, 5], [200, 1]), ([1000, 33], [70, 17]), ([17, 200], [17, 8])])
@pytest.mark.parametrize("seed,width", [(0, None), (1, None), (2, WIDE), (3, WIDE)])
def test_attention_nan_reaches_the_rows_that_see_it(n_q, n_kv, d, lens, q_lens, seed, width):
    """A NaN of K or V at a position of the chunk: rows before it keep their values."""
    r = np.random.default_rng(100 * seed + lens[0])
    shape = shape_of(n_q, n_kv, d)
    pool, bt, q = attention_case(r, n_q, n_kv, d, lens, q_lens, width=width)
    poison(r, pool, bt, lens[0], lens[0] - q_lens[0], d)
    got = run_attention(shape, pool, bt, q, lens, q_lens)
    q64 = q.double().numpy()
    want, mag = orc.attention(q64, pool, (0, 0), bt, lens, q_lens)
    hit = np.isnan(want)
    assert hit.any() and np.isnan(got[hit]).all()
    clean = ~hit.any(-1)  # (row, head) pairs that see no NaN
    top, vtop = (np.nan_to_num(np.abs(orc.take(pool, range(pool.shape[0] * 16), i, 0))).max() for i in (0, 1))
    mass = np.abs(q64).sum(-1, keepdims=True) * top / np.sqrt(d)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * d * 2.0 ** -24 * mass) * mag + max(lens) * 2.0 ** -32 * vtop
    assert (np.abs(got - want)[clean] <= bound[clean]).all()


@pytest.mark.parametrize("q_len,width", [(1, None), (9, None), (60, None), (60, WIDE), (70, WIDE)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_a_bad_query_spoils_its_own_row(q_len, bad, width):
    r = np.random.default_rng(q_len)
    lens, q_lens = [200, 70], [q_len, q_len]
    pool, bt, q = attention_case(r, 4, 2, 64, lens, q_lens, width=width)
    shape = shape_of(4, 2, 64)
    good = run_attention(shape, pool, bt, q, lens, q_lens)
    q[0, 1, 5] = bad
    got = run_attention(shape, pool, bt, q, lens, q_lens)
    assert not np.isfinite(got[0, 1]).all()
    got[0, 1] = good[0, 1]
    assert np.array_equal(got, good)


@pytest.mark.parametrize("width", [None, WIDE])
@pytest.mark.parametrize("n_q,n_kv,d,lens,q_lens", [
    (8, 1, 128, [6000], [130]), (4, 4, 64, [5000, 3, 900, 64], [77, 3, 65, 64]), (8, 2, 128, [2500, 60, 16, 18, 200], [900, 17, 16, 18, 1]), (2, 1, 64, [333, 32, 5000], [33, 32, 31]),
    (2, 2, 128, [1500], [1500]), (16, 2, 64, [40, 0, 10, 700, 8], [40, 30, 40, 128, 9])])
def test_attention_long_chunks(n_q, n_kv, d, lens, q_lens, width):
    """Tiles cut between CTAs, chunks on both sides of what one kernel takes, tiles without a position."""
    r = np.random.default_rng(lens[0])
    check_attention(shape_of(n_q, n_kv, d), *attention_case(r, n_q, n_kv, d, lens, q_lens, width=width), lens, q_lens, pad_rows=3)


@pytest.mark.parametrize("width", [None, 1000])
@pytest.mark.parametrize("n_q,n_kv", [(2, 2), (8, 1)])
def test_attention_many_chunks(n_q, n_kv, width):
    """More requests than threads, every third of them with rows for the tiles."""
    r = np.random.default_rng(n_q)
    q_lens = np.where(np.arange(700) % 3 == 0, 64 * n_kv // n_q - 1 + np.arange(700) % 5, np.arange(700) % 4)
    lens = np.maximum(q_lens + r.integers(-2, 60, 700), 0)
    check_attention(shape_of(n_q, n_kv, 64), *attention_case(r, n_q, n_kv, 64, lens, q_lens, width=width), lens, q_lens)


def test_attention_two_handles_at_once():
    r = np.random.default_rng(18)
    shape = shape_of(8, 2, 128)
    jobs = []
    for lens, q_lens in (([3000, 40], [300, 1]), ([2000, 500, 7], [1, 200, 7])):
        pool, bt, q = attention_case(r, 8, 2, 128, lens, q_lens, width=WIDE)
        h = _lib.Kv4(shape, pool.shape[0], bt.shape[1])
        cache = _lib.KvCache(shape, pool.shape[0], _lib.NF_KV_FP4, torch.from_numpy(pool).to(DEV))
        args = (h, q.to(DEV), cache, dev32(bt), dev32(lens))
        begin = dev32(np.concatenate([[0], np.cumsum(q_lens)]))
        alone = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
        _lib.attention_kv4(*args, alone, begin)
        jobs.append((args, begin, alone, [torch.empty_like(alone) for _ in range(8)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(8):
        for args, begin, _, outs, stream in jobs:
            _lib.attention_kv4(*args, outs[i], begin, stream=stream)
    torch.cuda.synchronize()
    for args, _, alone, outs, _ in jobs:
        args[0].poll()
        assert all(torch.equal(o, alone) for o in outs)


def test_attention_too_many_pages_for_a_call_is_reported():
    """43 requests of 100,000 pages and 1024 KV heads: past 2^32 (page, head) pairs nothing is written."""
    shape = shape_of(1024, 1024, 64)
    pages, n = 100_000, 43
    h = _lib.Kv4(shape, 1, pages)
    cache = _lib.KvCache(shape, 1, _lib.NF_KV_FP4, torch.zeros(1, 1024, 2, 576, dtype=torch.uint8, device=DEV))
    o = torch.full((n, 1024, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    _lib.attention_kv4(h, torch.zeros_like(o), cache, dev32(np.zeros((n, pages))), dev32([16 * pages] * n), o)
    with pytest.raises(_lib.NanoflowError) as e:
        h.poll()
    assert e.value.code == _lib.NF_ERR_DEVICE and "too many" in str(e.value)
    assert (o == 5.0).all()


@pytest.mark.parametrize("cta", [0, 77])
@pytest.mark.parametrize("part,block", [(0, 0), (1, 0), (0, 1), (1, 1), (0, 4), (1, 5)])
def test_attention_a_lost_arrival_is_reported_and_the_handle_recovers(part, block, cta):
    """A wait of the kernel of longer chunks runs out at several stages: with nothing issued, with scores or
    weighted sums under way, with pieces of cut requests counted.  Then the handle is as new."""
    r = np.random.default_rng(22)
    shape = shape_of(8, 2, 128)
    lens, q_lens = [6000, 40, 500], [900, 1, 200]
    pool, bt, q = attention_case(r, 8, 2, 128, lens, q_lens, width=WIDE)
    h = _lib.Kv4(shape, pool.shape[0], bt.shape[1])
    cache = _lib.KvCache(shape, pool.shape[0], _lib.NF_KV_FP4, torch.from_numpy(pool).to(DEV))
    args = (h, q.to(DEV), cache, dev32(bt), dev32(lens))
    begin = dev32(np.concatenate([[0], np.cumsum(q_lens)]))
    good, got = (torch.empty(q.shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    _lib.attention_kv4(*args, good, begin)
    h.poll()
    h.set_timeout(20_000_000)
    h.selftest_drop(cta, part, block)
    for _ in range(2):
        _lib.attention_kv4(*args, got, begin)
        with pytest.raises(_lib.NanoflowError) as e:
            h.poll()
        assert e.value.code == _lib.NF_ERR_TIMEOUT
        h.poll()  # reported once
    h.selftest_drop(cta, part, 100_000)  # a block that no CTA has: nothing is left out
    for _ in range(3):
        got.zero_()
        _lib.attention_kv4(*args, got, begin)
        h.poll()
        assert torch.equal(got, good)
    h.selftest_drop(-1)
    _lib.attention_kv4(*args, got, begin)
    h.poll()
    assert torch.equal(got, good)
    for bad in ((lambda: h.set_timeout(0)), (lambda: h.set_timeout(10 ** 10 + 1)), (lambda: h.selftest_drop(10 ** 6)),
                (lambda: h.selftest_drop(0, 2)), (lambda: h.selftest_drop(0, 0, -1))):
        with pytest.raises(_lib.NanoflowError) as e:
            bad()
        assert e.value.code == _lib.NF_ERR_INVALID_ARG


@pytest.mark.parametrize("width", [None, WIDE])
def test_a_new_handle_on_a_stream_beside_a_busy_default_stream(width):
    """The handle's counters are zero when the handle is there, whatever the default stream still has to do."""
    r = np.random.default_rng(23)
    shape = shape_of(8, 2, 128)
    lens, q_lens = [5000, 3, 260], [130, 1, 1]
    pool, bt, q = attention_case(r, 8, 2, 128, lens, q_lens, width=width)
    cache = _lib.KvCache(shape, pool.shape[0], _lib.NF_KV_FP4, torch.from_numpy(pool).to(DEV))
    qd, btd, ld = q.to(DEV), dev32(bt), dev32(lens)
    begin = dev32(np.concatenate([[0], np.cumsum(q_lens)]))
    first = _lib.Kv4(shape, pool.shape[0], bt.shape[1])
    good, got = torch.empty_like(qd), torch.full_like(qd, 5.0)
    _lib.attention_kv4(first, qd, cache, btd, ld, good, begin)
    first.poll()
    a, side = torch.randn(8192, 8192, device=DEV), torch.cuda.Stream()
    used = torch.ones(64 << 20, dtype=torch.uint8, device=DEV)  # memory that is not zero, for the handle to get
    torch.cuda.synchronize()
    del used
    torch.cuda.empty_cache()
    for _ in range(30):
        a = a @ a
        a = a / a.abs().max()
    h = _lib.Kv4(shape, pool.shape[0], bt.shape[1])
    _lib.attention_kv4(h, qd, cache, btd, ld, got, begin, stream=side)
    side.synchronize()
    assert torch.equal(got, good)
    h.poll()


@pytest.mark.parametrize("limit", [1, 1000, 4000, 16_000])
def test_attention_limits_shorter_than_its_waits(limit):
    """Limits of the order of a wait, so that any role may be the one that gives up: a call computes or reports
    a timeout, and with the ordinary limit the handle is as new."""
    r = np.random.default_rng(29)
    shape = shape_of(8, 2, 128)
    lens, q_lens = [3000, 40, 500], [500, 1, 200]
    pool, bt, q = attention_case(r, 8, 2, 128, lens, q_lens, width=WIDE)
    h = _lib.Kv4(shape, pool.shape[0], bt.shape[1])
    cache = _lib.KvCache(shape, pool.shape[0], _lib.NF_KV_FP4, torch.from_numpy(pool).to(DEV))
    args = (h, q.to(DEV), cache, dev32(bt), dev32(lens))
    begin = dev32(np.concatenate([[0], np.cumsum(q_lens)]))
    good, got = (torch.empty(q.shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    _lib.attention_kv4(*args, good, begin)
    h.poll()
    for _ in range(5):
        got.zero_()
        h.set_timeout(limit)
        _lib.attention_kv4(*args, got, begin)
        try:
            h.poll()
            assert torch.equal(got, good)
        except _lib.NanoflowError as e:
            assert e.code == _lib.NF_ERR_TIMEOUT
        h.set_timeout(2_000_000_000)
        _lib.attention_kv4(*args, got, begin)
        h.poll()
        assert torch.equal(got, good)


def test_polls_without_waiting_report_a_status_once():
    """Polls beside a running call on another stream: the bit is reported by one of them and never again."""
    r = np.random.default_rng(28)
    shape = shape_of(4, 2, 64)
    lens = [40, 20]
    pool, bt, q = attention_case(r, 4, 2, 64, lens, [1, 1])
    bt[1, 0] = -5
    h = _lib.Kv4(shape, pool.shape[0], bt.shape[1])
    cache = _lib.KvCache(shape, pool.shape[0], _lib.NF_KV_FP4, torch.from_numpy(pool).to(DEV))
    args = (h, q.to(DEV), cache, dev32(bt), dev32(lens), torch.empty(2, 4, 64, dtype=torch.bfloat16, device=DEV))
    a, side = torch.randn(4096, 4096, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            a = a @ a
            a = a / a.abs().max()
        _lib.attention_kv4(*args)
    reports = 0
    for wait in [False] * 50 + [True] * 2:
        try:
            h.poll(wait)
        except _lib.NanoflowError as e:
            assert e.code == _lib.NF_ERR_DEVICE
            reports += 1
    assert reports == 1


def test_binding_refuses_tensors_of_another_device():
    """One tensor of a call on the CPU: refused on the host, before its address goes anywhere."""
    shape, b = shape_of(4, 2, 64), torch.bfloat16
    z = lambda *n, t=torch.int32: torch.zeros(n, dtype=t, device=DEV)  # noqa: E731
    cache = _lib.KvCache(shape, 8, _lib.NF_KV_FP4, z(8, 2, 2, 576, t=torch.uint8))
    with pytest.raises(ValueError, match="V pool"):
        _lib.KvCache(shape, 8, _lib.NF_KV_BF16, z(8, 2, 16, 64, t=b), z(8, 2, 16, 64, t=b).cpu())
    h = _lib.Kv4(shape, 8, 5)
    for call, good in ((lambda *a: _lib.block_tables(_lib.BlockTables(*a)), [z(3), z(3), z(3, 4), z(8), z(2), z(4), z(4), z(9), z(9), z(9)]),
                       (lambda *a: _lib.qk_norm_rope(shape, *a, cache), [z(3, 512, t=b), z(64, t=b), z(64, t=b), z(3), z(3) - 1, z(3, 256, t=b)]),
                       (lambda *a: _lib.kv4_read(shape, cache, *a), [z(3), z(3, 128, t=b), z(3, 128, t=b)]),
                       (lambda q, *a: _lib.attention_kv4(h, q, cache, *a), [z(3, 256, t=b), z(2, 5), z(2), z(3, 256, t=b), z(3)])):
        call(*good)
        for at in range(len(good)):
            with pytest.raises(ValueError, match="cpu|cuda"):
                call(*[t.cpu() if i == at else t for i, t in enumerate(good)])
    torch.cuda.synchronize()


# ------------------------------------------------------------------ sizes past 32 bits

def test_a_pool_past_32_bits():
    """A cache of more than 2^32 bytes: append, rows by slot and attention at its far end."""
    n_q, n_kv, d, num = 32, 8, 128, 240_000
    shape = shape_of(n_q, n_kv, d)
    r = np.random.default_rng(19)
    n = 100
    x, pos, _ = append_case(r, n, n_q, n_kv, d, num, 1000)
    slot = num * 16 - 1 - r.permutation(7 * 16)[:n]
    outs = []
    for pages, shift in ((num, 0), (7, (num - 7) * 16)):  # the same slots in a pool of the last pages alone
        pool = torch.full((pages, n_kv, 2, 9 * d), 0x7F, dtype=torch.uint8, device=DEV)
        cache = _lib.KvCache(shape, pages, _lib.NF_KV_FP4, pool)
        q = torch.empty(n, n_q, d, dtype=torch.bfloat16, device=DEV)
        _lib.qk_norm_rope(shape, x.to(DEV), None, None, dev32(pos), dev32(slot - shift), q, cache)
        k, v = (torch.empty(n, n_kv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        _lib.kv4_read(shape, cache, dev32(slot - shift), k, v)
        pool[-7:, :, :, 8 * d:][pool[-7:, :, :, 8 * d:] == 0x7F] = 0x30
        o = torch.empty(40, n_q, d, dtype=torch.bfloat16, device=DEV)
        h = _lib.Kv4(shape, pages, 3)
        bt = dev32([[num - 1, num - 4, num - 2], [num - 7, num - 3, num - 6]]) - shift // 16
        _lib.attention_kv4(h, q[:40], cache, bt, dev32([45, 48]), o, dev32([0, 5, 40]))
        h.poll()
        outs.append([pool[-7:].clone(), q, k, v, o])
        del pool, cache
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert np.array_equal(host(outs[0][2].float())[0].astype(float), orc.take(host(outs[1][0]), [int(slot[0]) - (num - 7) * 16], 0, 0)[0])


def test_rows_past_32_bits():
    """Rows whose offsets in qkv, q and the read-out pass 2^32 bytes give what they give in a small call."""
    shape = shape_of(32, 8, 128)
    n, tail = 400_000, 50
    g = torch.Generator(device=DEV).manual_seed(20)
    x = torch.zeros(n, 48 * 128, dtype=torch.bfloat16, device=DEV)
    x[-tail:] = torch.randn(tail, 48 * 128, generator=g, device=DEV).to(torch.bfloat16)
    slot = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    slot[-tail:] = torch.arange(tail, dtype=torch.int32, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    outs = []
    for m in (n, tail):
        pool = torch.zeros(4, 8, 2, 9 * 128, dtype=torch.uint8, device=DEV)
        q = torch.empty(m, 32, 128, dtype=torch.bfloat16, device=DEV)
        _lib.qk_norm_rope(shape, x[-m:], None, None, pos[-m:].contiguous(), slot[-m:].contiguous(), q, _lib.KvCache(shape, 4, _lib.NF_KV_FP4, pool))
        outs.append([pool, q[-tail:].clone()])
        del q
    del x
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    n = 2_200_000
    k, v = (torch.empty(n, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.arange(n, dtype=torch.int32, device=DEV) % 64
    cache = _lib.KvCache(shape, 4, _lib.NF_KV_FP4, outs[0][0])
    _lib.kv4_read(shape, cache, slots, k, v)
    ks, vs = (torch.empty(64, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    _lib.kv4_read(shape, cache, slots[:64].contiguous(), ks, vs)
    assert ks.any() and all(torch.equal(a[-64:], b.roll(-(n % 64), 0)) for a, b in ((k, ks), (v, vs)))


@pytest.mark.parametrize("rows,pages", [(1, 1 << 26), (9, 1 << 22)])
def test_attention_of_the_longest_requests(rows, pages):
    """2^30 positions, the most that a request may have, and a chunk over 2^26: every page is the same one, so
    the output is that of its 16 positions.  The fp32 sums of a warp (of a CTA of the tiles) take
    pages / (12 x 100) (blocks / 100) additions at least a hundred SMs share: each errs by 2^-24."""
    d, n_q = 64, 8
    shape = shape_of(n_q, 1, d)
    r = np.random.default_rng(26)
    pool = filled_pool(r, 1, 1, d)
    q = torch.from_numpy(r.standard_normal((rows, n_q, d))).to(torch.bfloat16)
    bt = torch.zeros(1, pages, dtype=torch.int32, device=DEV)
    h = _lib.Kv4(shape, 1, pages)
    cache = _lib.KvCache(shape, 1, _lib.NF_KV_FP4, torch.from_numpy(pool).to(DEV))
    o = torch.empty(rows, n_q, d, dtype=torch.bfloat16, device=DEV)
    _lib.attention_kv4(h, q.to(DEV), cache, bt, dev32([16 * pages]), o, dev32([0, rows]))
    h.poll()
    got = o.double().cpu().numpy()
    q64 = q.double().numpy()
    want, mag = (np.concatenate(x) for x in zip(*(orc.attention(q64[i:i + 1], pool, (0, 0), np.zeros((1, 1), int), [16], [1]) for i in range(rows))))
    top = np.abs(orc.take(pool, range(16), 0, 0)).max()
    mass = np.abs(q64).sum(-1, keepdims=True) * top / np.sqrt(d)
    adds = pages / 1200 if rows == 1 else pages / 8 / 100 * 16  # a block is 16 steps of 8 positions
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * adds * 2.0 ** -24 + 2 * d * 2.0 ** -24 * mass + rows / pages) * mag
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / mag).max()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("n_q,n_kv,d", [(8, 2, 128), (4, 4, 64)])
def test_a_served_batch(n_q, n_kv, d):
    """Prompts, then decode steps, a request that ends and a new one in its place: tables, append and
    attention of every step on the GPU, against the oracle that follows from the same inputs."""
    shape = shape_of(n_q, n_kv, d)
    r = np.random.default_rng(17)
    n, width, num = 4, 8, 20
    exps = (0, 1)
    table, ring = np.full((n, width), -1), np.arange(num)[::-1].copy()
    pool = np.full((num, n_kv, 2, 9 * d), 0x7F, np.uint8)  # NaN scales: an unwritten slot that is read shows
    state = np.array([0, num])
    t = dict(block_table=dev32(table), ring=dev32(ring), tok_begin=dev32([0] * (n + 1)))
    st = [dev32([0, num, 0, 0]), dev32([0] * 4)]
    pd = torch.from_numpy(pool).to(DEV)
    cache = _lib.KvCache(shape, num, _lib.NF_KV_FP4, pd, None, *exps)
    h = _lib.Kv4(shape, num, width)
    gains = gains_of(r, d)
    gd = [g.to(DEV) for g in gains]
    held = np.zeros(n, int)
    plan = [[37, 16, 1, 0], [38, 17, 2, 20], [39, 18, 3, 21], [40, 0, 4, 22], [41, 31, 5, 23], [48, 32, 6, 24]]
    for step, lens in enumerate(plan):
        lens = np.array(lens)
        tok = int(np.clip(lens - held, 0, None).sum())
        rows = [np.full(tok, -5)] * 3
        td = [dev32(x) for x in rows]
        _lib.block_tables(_lib.BlockTables(dev32(held), dev32(lens), t["block_table"], t["ring"], st[step % 2][:2], st[1 - step % 2],
                                           t["tok_begin"], *td))
        x = torch.from_numpy(r.standard_normal((tok, (n_q + 2 * n_kv) * d))).to(torch.bfloat16)
        q = torch.empty(tok, n_q, d, dtype=torch.bfloat16, device=DEV)
        o = torch.empty_like(q)
        _lib.qk_norm_rope(shape, x.to(DEV), gd[0], gd[1], td[1], td[2], q, cache)
        _lib.attention_kv4(h, q, cache, t["block_table"], dev32(lens), o, t["tok_begin"])
        h.poll()
        want = orc.block_tables(held, lens, table, ring, state[:2], rows)
        table, ring, state = want["block_table"], want["ring"], want["state_out"]
        u = x.double().numpy().reshape(tok, -1, d)
        for i, part, w in ((1, 0, orc.norm_rope(u[:, n_q:n_q + n_kv], gains[1].double().numpy(), want["tok_pos"], 1e4, float(np.float32(1e-5)))),
                           (0, 1, u[:, n_q + n_kv:])):
            for k in range(tok):
                orc.put(pool, int(want["tok_slot"][k]), part, *orc.quantise(w[k], exps[part]))
        assert np.array_equal(host(pd), pool)
        q64 = q.double().cpu().numpy()
        ref, mag = orc.attention(q64, pool, exps, table, lens, np.clip(lens - held, 0, None))
        bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -20 + 2 * d * 2.0 ** -24 * np.abs(q64).sum(-1, keepdims=True) * 10) * mag
        assert (np.abs(o.double().cpu().numpy() - ref) <= bound).all()
        held = lens


def test_the_attention_half_of_a_layer():
    """RMSNorm, QKV GEMM, tables, append, attention and the O GEMM with its residual over the 4-bit cache: a
    prompt step call by call, every stage against float64 from the stage before, then decode steps of the same
    padded batch in one captured graph, bit for bit what single calls give."""
    n_q, n_kv, d, hidden = 8, 2, 64, 256
    shape = shape_of(n_q, n_kv, d)
    r = np.random.default_rng(27)
    n, width, num, cap = 5, 6, 24, 64
    width_qkv = (n_q + 2 * n_kv) * d
    rnd = lambda *s, std=1.0: torch.from_numpy(std * r.standard_normal(s)).to(torch.bfloat16)  # noqa: E731
    norm, w_qkv, w_o = 1 + 0.1 * rnd(hidden), rnd(width_qkv, hidden, std=0.06), rnd(hidden, n_q * d, std=0.05)
    gains = gains_of(r, d)
    g = dict(norm=norm.to(DEV), w_qkv=w_qkv.to(DEV), w_o=w_o.to(DEV), q=gains[0].to(DEV), k=gains[1].to(DEV))
    xs = rnd(cap, hidden).to(DEV)
    lens0 = np.array([20, 1, 0, 16, 17])

    def state():
        z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
        pool = torch.full((num, n_kv, 2, 9 * d), 0x7F, dtype=torch.uint8, device=DEV)
        s = dict(held=z(n), lens=dev32(lens0), bt=z(n, width) - 1, ring=torch.arange(num, dtype=torch.int32, device=DEV), st=dev32([0, num]),
                 out=z(4), begin=z(n + 1), seq=z(cap), pos=z(cap), slot=z(cap) - 1, pool=pool, cache=_lib.KvCache(shape, num, _lib.NF_KV_FP4, pool),
                 handle=_lib.Kv4(shape, num, width))
        b = torch.bfloat16
        s |= dict(n1=z(cap, hidden, t=b), qkv=z(cap, width_qkv, t=b), q=z(cap, n_q, d, t=b), o=z(cap, n_q, d, t=b), y=z(cap, hidden, t=b))
        s["args"] = _lib.BlockTables(s["held"], s["lens"], s["bt"], s["ring"], s["st"], s["out"], s["begin"], s["seq"], s["pos"], s["slot"])
        return s

    def step(s):
        s["slot"].fill_(-1)  # rows behind the step's tokens store nothing
        _lib.block_tables(s["args"])
        _lib.rmsnorm(xs, g["norm"], s["n1"], 1e-5)
        _lib.gemm(s["n1"], g["w_qkv"], s["qkv"])
        _lib.qk_norm_rope(shape, s["qkv"], g["q"], g["k"], s["pos"], s["slot"], s["q"], s["cache"])
        _lib.attention_kv4(s["handle"], s["q"], s["cache"], s["bt"], s["lens"], s["o"], s["begin"])
        _lib.gemm(s["o"].view(cap, -1), g["w_o"], s["y"], R=xs, epilogue=_lib.NF_EPI_RESID)

    def grow(s):  # the next step: every request one token longer
        s["st"].copy_(s["out"][:2])
        s["held"].copy_(s["lens"])
        s["lens"].add_(1)

    a = state()
    step(a)
    a["handle"].poll()
    h = {k: v.double().cpu().numpy() for k, v in a.items() if isinstance(v, torch.Tensor) and v.dtype == torch.bfloat16}
    x64, tok = xs.double().cpu().numpy(), int(lens0.sum())
    assert host(a["out"]).tolist() == [6, num - 6, tok, 0]  # 2 + 1 + 0 + 1 + 2 pages

    def near(got, ref, mass, k):  # one rounding to bf16, k products summed in fp32
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -24 * mass).all()

    n1 = x64 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + float(np.float32(1e-5))) * norm.double().numpy()
    near(h["n1"], n1, np.abs(n1), hidden)
    w64, o64 = w_qkv.double().numpy(), w_o.double().numpy()
    near(h["qkv"], h["n1"] @ w64.T, np.abs(h["n1"]) @ np.abs(w64).T, hidden)
    u, pos, slot = h["qkv"].reshape(cap, -1, d), host(a["pos"]), host(a["slot"])
    want = np.full((num, n_kv, 2, 9 * d), 0x7F, np.uint8)
    keys = orc.norm_rope(u[:tok, n_q:n_q + n_kv], gains[1].double().numpy(), pos[:tok], 1e4, float(np.float32(1e-5)))
    for i in range(tok):
        orc.put(want, int(slot[i]), 0, *orc.quantise(keys[i], 0))
        orc.put(want, int(slot[i]), 1, *orc.quantise(u[i, n_q + n_kv:], 0))
    assert np.array_equal(host(a["pool"]), want)
    ref, mag = orc.attention(h["q"][:tok], want, (0, 0), host(a["bt"]), lens0, lens0)
    mass = np.abs(h["q"][:tok]).sum(-1, keepdims=True) * np.nan_to_num(np.abs(orc.take(want, slot[:tok], 0, 0))).max() / np.sqrt(d)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -20 + 2 * d * 2.0 ** -24 * mass) * mag + 64 * 2.0 ** -32 * 8
    assert (np.abs(h["o"][:tok] - ref) <= bound).all() and not h["o"][tok:].any()
    of = h["o"].reshape(cap, -1)
    near(h["y"], x64 + of @ o64.T, np.abs(x64) + np.abs(of) @ np.abs(o64).T, n_q * d + 1)

    b = state()
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grow(b)
        step(b)
    for _ in range(4):
        grow(a)
        step(a)
        graph.replay()
        for k in ("bt", "ring", "out", "begin", "slot", "pool", "q", "o", "y"):
            assert torch.equal(a[k], b[k]), k
    for s in (a, b):
        s["handle"].poll()
    assert host(a["out"])[2:].tolist() == [n, 0] and host(a["lens"]).tolist() == (lens0 + 4).tolist()
