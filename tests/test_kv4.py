"""The 4-bit cache without a GPU: the oracle against closed forms and brute force, and the
refusals of its entry points (nothing is launched)."""
import ctypes
import os
import types

import numpy as np
import pytest
import torch

from nano_intra_device_gb300 import _lib, workload as wl
from oracle import kv4 as orc

SHAPE = wl.Shape(hidden=256, n_q=4, n_kv=2, head_dim=64, ffn=16)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from nano_intra_device_gb300 import build
        build.build()
    return _lib.lib()


# ------------------------------------------------------------------ the oracle

def test_formats_hold_the_listed_values():
    # e2m1: sign, 2 exponent bits (bias 1), 1 fraction bit; e4m3: bias 7, largest 448, no infinity
    for c in range(8):
        e, m = c >> 1, c & 1
        assert orc.E2M1[c] == (m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, orc.E4M3)


def test_nearest_is_the_nearest_and_ties_go_to_even():
    for grid in (orc.E2M1, orc.E4M3):
        mids = (grid[1:] + grid[:-1]) / 2
        code = orc.nearest(mids, grid)
        assert np.all(code % 2 == 0) and np.all(np.abs(grid[code] - mids) <= (grid[1:] - grid[:-1]) / 2)
        x = np.random.default_rng(0).uniform(0, grid[-1] * 1.2, 2000)
        brute = np.abs(x[:, None] - grid).argmin(1)
        assert np.array_equal(orc.nearest(x, grid), brute)


def test_quantise_of_representable_blocks_is_exact():
    r = np.random.default_rng(1)
    for exp in (-3, 0, 5):
        codes = r.integers(0, 16, (7, 64)).astype(np.uint8)
        codes[:, ::16] = 7  # the largest code in every block fixes its scale
        scales = r.integers(8, 127, (7, 4)).astype(np.uint8)
        x = orc.values(codes, scales, exp)
        c2, s2 = orc.quantise(x, exp)
        assert np.array_equal(s2, scales)
        assert np.array_equal(orc.values(c2, s2, exp), x)


def test_quantise_special_blocks():
    x = np.zeros((4, 16))
    x[1, 3] = np.nan
    x[2, 5], x[2, 6] = np.inf, 1.0
    x[3] = 2.0 ** -13  # below half of the smallest scale: zero scale, zero codes
    codes, scales = orc.quantise(x, 0)
    assert scales[:, 0].tolist() == [0, 127, 126, 0]
    assert not codes[[0, 1, 3]].any() and codes[2, 5] == 7


def test_put_and_take_invert_each_other():
    r = np.random.default_rng(2)
    pool = r.integers(0, 255, (3, 2, 2, 9 * 64)).astype(np.uint8)
    before = pool.copy()
    codes, scales = r.integers(0, 16, (2, 64)).astype(np.uint8), r.integers(0, 127, (2, 4)).astype(np.uint8)
    orc.put(pool, 37, 1, codes, scales)
    assert np.array_equal(orc.take(pool, [37], 1, 2)[0], orc.values(codes, scales, 2))
    assert (pool != before).sum() <= 2 * (32 + 4)
    assert not orc.take(pool, [-1, 48], 0, 0).any()


def test_attention_of_equal_keys_is_the_mean():
    pool = np.zeros((4, 1, 2, 9 * 64), np.uint8)
    r = np.random.default_rng(3)
    for slot in range(40):
        c, s = orc.quantise(r.standard_normal((1, 64)), 0)
        orc.put(pool, slot, 1, c, s)
    bt = np.array([[0, 1, 2]], np.int32)
    q = r.standard_normal((3, 2, 64))
    o, _ = orc.attention(q, pool, (0, 0), bt, [40], [3])
    v = orc.take(pool, range(40), 1, 0)[:, 0]
    for i in range(3):
        assert np.allclose(o[i], v[:38 + i].mean(0)[None])
    o, _ = orc.attention(q, pool, (0, 0), bt, [1], [3])  # two rows before position 0
    assert not o[:2].any() and np.allclose(o[2], v[0])


def test_block_tables_conserve_pages():
    r = np.random.default_rng(4)
    n, width, num = 9, 6, 40
    held = r.integers(0, 50, n)
    perm = r.permutation(num)
    table, used = np.full((n, width), -1), 0
    for s in range(n):
        k = -(-held[s] // 16)
        table[s, :k] = perm[used:used + k]
        used += k
    ring, head = np.full(num, -7), 33
    ring[(head + np.arange(num - used)) % num] = perm[used:]
    for step in range(20):
        lens = r.integers(0, width * 16 + 1, n) if step % 3 else held + (held < width * 16)
        caps = [np.full(400, -5) for _ in range(3)]
        got = orc.block_tables(held, lens, table, ring, (head, num - used), caps)
        if got["state_out"][3]:
            assert np.array_equal(got["ring"], ring)
            continue
        table, ring, head = got["block_table"], got["ring"], got["state_out"][0]
        held, used = lens, num - got["state_out"][1]
        owned = [p for s in range(n) for p in table[s, :-(-held[s] // 16)]]
        free = ring[(head + np.arange(num - used)) % num]
        assert sorted([*owned, *free]) == list(range(num))


# ------------------------------------------------------------------ refusals

def _cache(**kw):
    c = _lib.nf_kv_cache(_lib.NF_KV_FP4, 8, 1 << 20, None, 0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _refused(code):
    assert code == _lib.NF_ERR_INVALID_ARG
    return _lib.lib().nf_last_error().decode()


def _shape(**kw):
    s = _lib.make_shape(SHAPE)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


BAD_SHAPES = [dict(head_dim=96), dict(head_dim=0), dict(n_q_heads=3), dict(n_q_heads=6), dict(n_kv_heads=0), dict(page_size=32)]
BAD_CACHES = [dict(format=2), dict(num_pages=0), dict(num_pages=1 << 27), dict(k=None), dict(k=(1 << 20) + 8), dict(v=1 << 20),
              dict(k_exp=65), dict(v_exp=-65), dict(format=_lib.NF_KV_BF16), dict(format=_lib.NF_KV_BF16, v=(1 << 20) + 2)]
P16 = 1 << 20  # an aligned address that nothing reads: every call here is refused on the host


def test_pool_bytes(L):
    n = ctypes.c_size_t()
    assert L.nf_kv4_pool_bytes(ctypes.byref(_shape()), 5, ctypes.byref(n)) == _lib.NF_OK
    assert n.value == 5 * 2 * 2 * (16 * 32 + 16 * 4)
    for bad in BAD_SHAPES:
        _refused(L.nf_kv4_pool_bytes(ctypes.byref(_shape(**bad)), 5, ctypes.byref(n)))
    _refused(L.nf_kv4_pool_bytes(ctypes.byref(_shape()), 0, ctypes.byref(n)))
    _refused(L.nf_kv4_pool_bytes(None, 5, ctypes.byref(n)))


def test_block_tables_refusals(L):
    good = [P16, P16, 3, P16, 4, P16, 8, P16, P16 + 64, P16, P16, P16, P16, 10, None]
    for at in (0, 1, 3, 5, 7, 8, 9, 10, 11, 12):
        assert "NULL" in _refused(L.nf_block_tables(*[None if i == at else v for i, v in enumerate(good)]))
    for at, v in ((2, 0), (2, -1), (4, 0), (4, 1 << 27), (6, 0), (6, 1 << 27), (13, -1), (8, P16), (8, P16 + 4), (8, P16 - 12)):
        _refused(L.nf_block_tables(*[v if i == at else x for i, x in enumerate(good)]))


def test_qk_norm_rope_refusals(L):
    def call(shape=None, cache=None, **kw):
        a = dict(qkv=P16, ld=512, q_gain=None, k_gain=None, pos=P16, slot=P16, n=3, q=P16) | kw
        return L.nf_qk_norm_rope(ctypes.byref(shape or _shape()), a["qkv"], a["ld"], a["q_gain"], a["k_gain"], a["pos"], a["slot"],
                                 a["n"], a["q"], ctypes.byref(cache or _cache()), None)
    for bad in BAD_SHAPES + [dict(rope_theta=0.0), dict(rope_theta=float("inf")), dict(rope_theta=float("nan")), dict(rms_eps=-1.0)]:
        _refused(call(shape=_shape(**bad)))
    for bad in BAD_CACHES:
        _refused(call(cache=_cache(**bad)))
    for bad in (dict(qkv=None), dict(pos=None), dict(slot=None), dict(q=None), dict(qkv=P16 + 2), dict(q=P16 + 8), dict(q_gain=P16 + 4),
                dict(k_gain=P16 + 4), dict(ld=504), dict(ld=516), dict(ld=0), dict(n=-1)):
        _refused(call(**bad))
    assert call(n=0) == _lib.NF_OK


def test_kv4_read_refusals(L):
    def call(shape=None, cache=None, slots=P16, n=3, k=P16, v=P16):
        return L.nf_kv4_read(ctypes.byref(shape or _shape()), ctypes.byref(cache or _cache()), slots, n, k, v, None)
    for bad in BAD_SHAPES:
        _refused(call(shape=_shape(**bad)))
    for bad in BAD_CACHES + [dict(format=_lib.NF_KV_BF16, v=P16)]:
        _refused(call(cache=_cache(**bad)))
    for bad in (dict(slots=None), dict(k=None), dict(v=None), dict(n=-1), dict(k=P16 + 2), dict(v=P16 + 8)):
        _refused(call(**bad))
    assert call(n=0) == _lib.NF_OK


def test_handle_refusals(L):
    h = ctypes.c_void_p()
    for bad in BAD_SHAPES:
        _refused(L.nf_kv4_create(ctypes.byref(_shape(**bad)), 8, 4, ctypes.byref(h)))
        assert not h
    for pages, width in ((0, 4), (8, 0), (1 << 27, 4), (8, 1 << 27)):
        _refused(L.nf_kv4_create(ctypes.byref(_shape()), pages, width, ctypes.byref(h)))
    _refused(L.nf_kv4_create(ctypes.byref(_shape()), 8, 4, None))
    _refused(L.nf_kv4_poll(None, 0))
    L.nf_kv4_destroy(None)
    c = _cache()
    _refused(L.nf_attention_kv4(None, P16, ctypes.byref(c), P16, P16, None, 2, 2, P16, None))


def test_binding_checks_tensors():
    i, u = torch.int32, torch.uint8
    pool = torch.zeros(8, 2, 2, 576, dtype=u)
    _lib.KvCache(SHAPE, 8, _lib.NF_KV_FP4, pool)
    for t in (pool[..., :-1], pool.to(i), pool.transpose(0, 1), pool[:7]):
        with pytest.raises(ValueError):
            _lib.KvCache(SHAPE, 8, _lib.NF_KV_FP4, t)
    with pytest.raises(ValueError):
        _lib.KvCache(SHAPE, 8, _lib.NF_KV_BF16, torch.zeros(8, 2, 16, 64), torch.zeros(8, 2, 16, 64))
    z = lambda *n: torch.zeros(n, dtype=i)  # noqa: E731
    good = [z(3), z(3), z(3, 4), z(8), z(2), z(4), z(4), z(9), z(9), z(9)]
    _lib.BlockTables(*good)
    for at, t in ((0, z(3).long()), (1, z(4)), (2, z(2, 4)), (2, z(3, 8)[:, ::2]), (4, z(3)), (5, z(2)), (6, z(3)), (8, z(8))):
        with pytest.raises(ValueError):
            _lib.BlockTables(*[t if k == at else x for k, x in enumerate(good)])


def test_binding_checks_a_calls_tensors():
    """Types, sizes and strides that the addresses alone do not show, and a cache of another shape."""
    i, b = torch.int32, torch.bfloat16
    cache = _lib.KvCache(SHAPE, 8, _lib.NF_KV_FP4, torch.zeros(8, 2, 2, 576, dtype=torch.uint8))
    other = _lib.KvCache(wl.Shape(hidden=256, n_q=4, n_kv=4, head_dim=64, ffn=16), 8, _lib.NF_KV_FP4, torch.zeros(8, 4, 2, 576, dtype=torch.uint8))
    n, row = 3, SHAPE.n_q * 64
    z = lambda *n, t=i: torch.zeros(n, dtype=t)  # noqa: E731
    good = dict(qkv=z(n, 512, t=b), q_gain=z(64, t=b), k_gain=None, tok_pos=z(n), tok_slot=z(n), q=z(n, row, t=b), cache=cache)
    for bad in (dict(qkv=z(n, 512)), dict(qkv=z(512, n, t=b).T), dict(qkv=z(n, 504, t=b)), dict(q_gain=z(64)), dict(k_gain=z(32, t=b)),
                dict(tok_pos=z(n + 1)), dict(tok_slot=z(n).long()), dict(q=z(n, row)), dict(q=z(n + 1, row, t=b)), dict(q=z(row, n, t=b).T),
                dict(cache=other)):
        with pytest.raises(ValueError):
            _lib.qk_norm_rope(SHAPE, **(good | bad))
    good = dict(cache=cache, slots=z(n), k=z(n, 128, t=b), v=z(n, 128, t=b))
    for bad in (dict(slots=z(n).long()), dict(slots=z(2 * n)[::2]), dict(k=z(n, 128)), dict(v=z(n, 64, t=b)), dict(cache=other)):
        with pytest.raises(ValueError):
            _lib.kv4_read(SHAPE, **(good | bad))
    handle = types.SimpleNamespace(h=None, max_pages=5, heads=(2, 64), row=row)
    good = dict(q=z(n, row, t=b), cache=cache, block_table=z(2, 5), seq_lens=z(2), o=z(n, row, t=b), tok_begin=z(3))
    for bad in (dict(q=z(n, row)), dict(q=z(n, row // 2, t=b)), dict(block_table=z(2, 4)), dict(block_table=z(3, 5)), dict(block_table=z(2, 10)[:, ::2]),
                dict(seq_lens=z(2).long()), dict(o=z(n - 1, row, t=b)), dict(o=z(n, row)), dict(o=z(row, n, t=b).T), dict(tok_begin=z(2)), dict(cache=other)):
        with pytest.raises(ValueError):
            _lib.attention_kv4(handle, **(good | bad))


def test_handle_settings_refusals(L):
    assert "NULL" in _refused(L.nf_kv4_set_timeout(None, 1000))
    assert "NULL" in _refused(L.nf_kv4_selftest_drop(None, -1, 0, 0))


def test_handle_refuses_requests_whose_positions_pass_32_bits(L):
    h = ctypes.c_void_p()
    for width in ((1 << 26) + 1, (1 << 27) - 1):
        assert "max_pages_per_seq" in _refused(L.nf_kv4_create(ctypes.byref(_shape()), 8, width, ctypes.byref(h)))
        assert not h


def test_binding_refuses_tensors_of_the_cpu():
    """Right types and sizes, but addresses that no kernel may get."""
    i, b = torch.int32, torch.bfloat16
    z = lambda *n, t=i: torch.zeros(n, dtype=t)  # noqa: E731
    cache = _lib.KvCache(SHAPE, 8, _lib.NF_KV_FP4, torch.zeros(8, 2, 2, 576, dtype=torch.uint8))
    n, row = 3, SHAPE.n_q * 64
    calls = (lambda: _lib.block_tables(_lib.BlockTables(z(3), z(3), z(3, 4), z(8), z(2), z(4), z(4), z(9), z(9), z(9))),
             lambda: _lib.qk_norm_rope(SHAPE, z(n, 512, t=b), z(64, t=b), None, z(n), z(n), z(n, row, t=b), cache),
             lambda: _lib.kv4_read(SHAPE, cache, z(n), z(n, 128, t=b), z(n, 128, t=b)),
             lambda: _lib.attention_kv4(types.SimpleNamespace(h=None, max_pages=5, heads=(2, 64), row=row), z(n, row, t=b), cache, z(2, 5), z(2),
                                        z(n, row, t=b), z(3)))
    for call in calls:
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(ValueError, match="V pool"):
        _lib.KvCache(SHAPE, 8, _lib.NF_KV_BF16, z(8, 2, 16, 64, t=b))
