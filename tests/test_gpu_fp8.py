"""The 8-bit operators on the GPU against float64.

Quantisation of given values is compared exactly (codes and scales).  Bounds elsewhere:

* norm: x + r rounds once (2^-24 of it); the squares' sum errs by at most 2^-24 for each of a thread's 64
  terms at most and some 20 more additions; root, quotients and products round once each: together below
  2^-17 of y, and so of s.  A code is off by half a step (2^-4 of the value, 2^-10 below the normal
  codes), beside the errors of y and s, 2^-16 of the value.
* products: a block's 128 products are exact and summed in fp32 by the tensor core (each addition may
  truncate: 2^-23 of the sum of magnitudes), then scaled and added up, one rounding each, over the blocks
  of K: (128 * 2^-23 + (blocks + 3) * 2^-24) of the sum of magnitudes, beside the stored value's half step
  2^-8.  SwiGLU: the products' errors through silu'(g) u and silu(g), |silu'| <= 1.1, |silu(g)| <= |g|,
  and its own arithmetic, 2^-19 of the value: exp within 2^-21 up to |g| = 8, a quotient and two products.  At larger -g
  the rounded product g log2 e moves the exponential by up to 2^-18 of a value that is below |g u| e^-8 there, which the
  term above, 128 * 2^-23 |g u| at least, is larger than.
"""
import numpy as np
import pytest
import torch

from nano_intra_device_gb300 import _lib
from oracle import fp8 as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3, F32, BF16, I32 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32
STORE, RESID, SWIGLU, SWIGLU8 = _lib.NF_EPI_STORE, _lib.NF_EPI_RESID, _lib.NF_EPI_SWIGLU, _lib.NF_EPI_SWIGLU_FP8


def empty(*n, t=BF16):
    return torch.empty(n, dtype=t, device=DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def same(a, b):
    """Equal values, NaN with NaN."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    assert a.shape == b.shape and ((a == b) | (np.isnan(a) & np.isnan(b))).all()


# ------------------------------------------------------------------ quantisation

def quant(x, index=None):
    rows = len(x) if index is None else len(index)
    q, s = empty(rows, x.shape[1], t=E4M3), empty(orc.blocks(x.shape[1]), rows, t=F32)
    _lib.quant_fp8(x, q, s, index=index)
    return q, s


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 112), (2, 128), (5, 144), (33, 272), (7, 688), (2, 4096), (3, 4112), (2, 8192), (1, 16384), (2, 16400), (1, 32768)])
def test_quant(rows, cols):
    x = (torch.randn(rows, cols, device=DEV, generator=torch.Generator(DEV).manual_seed(cols)) * 3).to(BF16)
    q, s = quant(x)
    want = orc.quantise_rows(x.float().cpu().numpy())
    same(f64(q), want[0]), same(f64(s), want[1])


@pytest.mark.parametrize("src,index", [(4, [3, 3, 0, 1, 2, 0]), (1, [0]), (3, [-1, 0, 3, 2, 2147483647, -2147483648, 1]), (5, [])])
def test_quant_through_an_index(src, index):
    """Rows twice, none, and indices outside: a row of zeros."""
    x = torch.randn(src, 400, device=DEV).to(BF16)
    q, s = quant(x, torch.tensor(index, dtype=I32, device=DEV))
    h = x.float().cpu().numpy()
    rows = np.stack([h[i] if 0 <= i < src else np.zeros(400, np.float32) for i in index]) if index else np.zeros((0, 400), np.float32)
    want = orc.quantise_rows(rows)
    same(f64(q), want[0]), same(f64(s), want[1])


def special():
    r = np.random.default_rng(5)
    x = r.standard_normal((9, 272)).astype(np.float32)
    x[0] = 0
    x[1, 5], x[1, 200] = np.nan, np.inf
    x[2, 270] = -np.inf
    x[3] *= 2.0 ** -130            # subnormal values, the least scale
    x[4] *= 1e38 / np.abs(x[4]).max() * 3
    x[5, :128] = np.linspace(-448, 448, 128)
    x[6, 0] = 2.0 ** 20            # everything else far below its scale
    x[7] = -0.0
    x[8, 1:128:2], x[8, 0] = 1.0625, 448  # ties
    return torch.from_numpy(x).to(BF16)


def test_quant_special_values():
    x = special()
    q, s = quant(x.to(DEV))
    want = orc.quantise_rows(x.float().numpy())
    same(f64(s), want[1])
    same(f64(q), want[0])


@pytest.mark.parametrize("rows,cols", [(6601, 272), (5003, 400), (5001, 512), (3509, 688), (2301, 1040), (613, 4240), (70001, 144)])
def test_quant_many_rows(rows, cols):
    """Enough blocks for several a thread: special values in every block's place, rows by an index with some outside."""
    x = (torch.randn(1009, cols, generator=torch.Generator().manual_seed(cols)) * 3).to(BF16)
    sp = special()
    for i in range(0, 1009 - 9, 27):
        at = (i // 27 * 128) % (cols - 16)
        n = min(272, cols - at)
        x[i:i + 9, at:at + n] = sp[:, :n]
    index = torch.randint(-20, 1029, (rows,), generator=torch.Generator().manual_seed(rows), dtype=I32)
    q, s = quant(x.to(DEV), index.to(DEV))
    want_q, want_s = orc.quantise_rows(x.float().numpy())
    inside = (index >= 0) & (index < 1009)
    pick = index.clamp(0, 1008).long().numpy()
    zero_q, zero_s = orc.quantise_rows(np.zeros((1, cols), np.float32))
    same(f64(q), np.where(inside.numpy()[:, None], want_q[pick], zero_q))
    same(f64(s), np.where(inside.numpy()[None], want_s[:, pick], zero_s))
    q2, s2 = quant(x[pick].to(DEV))
    same(f64(q2), want_q[pick]), same(f64(s2), want_s[:, pick])


def test_quotients_are_cudas():
    """All pairs of 8-bit significands as value and largest of a block: codes as of the fp32 quotient."""
    top = torch.arange(128, 256, device=DEV).float()
    x = torch.zeros(128, 256, device=DEV)
    x[:, 0], x[:, 128] = top, top
    x[:, 1:128], x[:, 129:] = torch.arange(129, 256, device=DEV).float() / 2, torch.arange(129, 256, device=DEV).float() / 16
    q, s = quant(x.to(BF16))
    scale = top / torch.full_like(top, 448)  # by a number, torch multiplies with its reciprocal
    assert torch.equal(s, scale[None].expand(2, -1))
    assert torch.equal(q.float(), (x / scale[:, None]).to(E4M3).float())


@pytest.mark.parametrize("shape", [(1, 1, 16), (2, 128, 128), (1, 129, 272), (3, 200, 144), (1, 256, 688), (5, 7, 1040)])
def test_weights(shape):
    w = (torch.randn(shape, device=DEV) * 0.02).to(BF16)
    q, s = empty(*shape, t=E4M3), empty(shape[0], orc.blocks(shape[1]), orc.blocks(shape[2]), t=F32)
    _lib.quant_fp8_weights(w, q, s)
    for i in range(shape[0]):
        want = orc.quantise_weights(w[i].float().cpu().numpy())
        same(f64(q[i]), want[0]), same(f64(s[i]), want[1])


def test_weights_special_values():
    w = special().float().repeat(30, 1)[:260]
    w[:130][~torch.isfinite(w[:130])] = 1.0
    w = w.to(BF16)
    q, s = empty(260, 272, t=E4M3), empty(3, 3, t=F32)
    _lib.quant_fp8_weights(w.to(DEV), q, s)
    want = orc.quantise_weights(w.float().numpy())
    same(f64(q), want[0]), same(f64(s), want[1])
    assert np.isnan(want[1]).any() and not np.isnan(want[1]).all()


# ------------------------------------------------------------------ norm

def run_norm(x, g, eps, r=None, h=None):
    q, s = empty(*x.shape, t=E4M3), empty(orc.blocks(x.shape[1]), len(x), t=F32)
    _lib.rmsnorm_fp8(x, g, q, s, eps, r=r, h=h)
    return q, s


def check_norm(x, r, g, eps, q, s):
    _, y = orc.norm(f64(x), None if r is None else f64(r), f64(g), float(np.float32(eps)))
    n = x.shape[1]
    top = np.stack([np.abs(y[:, i:i + 128]).max(1) for i in range(0, n, 128)])
    want = np.maximum(top / 448, orc.TINY)
    assert (np.abs(f64(s) - want) <= 2.0 ** -17 * want).all()
    u = np.abs(y) / np.repeat(want.T, 128, 1)[:, :n]
    d = np.abs(f64(q) - y / np.repeat(want.T, 128, 1)[:, :n])
    assert (d <= np.maximum(2.0 ** -4 * u, 2.0 ** -10) + 2.0 ** -16 * u).all()


@pytest.mark.parametrize("rows,hidden", [(1, 16), (5, 112), (3, 256), (4, 688), (2, 4096), (3, 4112), (1, 8192), (2, 16384), (1, 28672), (1, 32768), (700, 256)])
@pytest.mark.parametrize("resid", [False, True])
def test_norm(rows, hidden, resid):
    gen = torch.Generator(DEV).manual_seed(rows + hidden)
    rnd = lambda *n: torch.randn(n, device=DEV, generator=gen)  # noqa: E731
    x, g = (rnd(rows, hidden) * 2).to(BF16), (1 + 0.2 * rnd(hidden)).to(BF16)
    r = (rnd(rows, hidden) * 0.7).to(BF16) if resid else None
    h = torch.full_like(x, 7) if resid else None
    q, s = run_norm(x, g, 1e-5, r, h)
    check_norm(x, r, g, 1e-5, q, s)
    if resid:
        assert torch.equal(h, (x.float() + r.float()).to(BF16))


@pytest.mark.parametrize("into", ["x", "r", "none"])
def test_norm_residual_in_place_or_not_kept(into):
    x, r, g = torch.randn(40, 4096, device=DEV).to(BF16), torch.randn(40, 4096, device=DEV).to(BF16), torch.ones(4096, device=DEV).to(BF16)
    want, total = run_norm(x, g, 1e-5, r, torch.empty_like(x)), (x.float() + r.float()).to(BF16)
    h = dict(x=x, r=r, none=None)[into]
    q, s = run_norm(x, g, 1e-5, r, h)
    assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1])
    assert h is None or torch.equal(h, total)


def test_norm_of_zero_rows_and_bad_values():
    x = torch.zeros(4, 272, device=DEV)
    x[1] = torch.randn(272, device=DEV)
    x[2], x[3] = x[1], x[1]
    x[2, 7], x[3, 200] = float("nan"), float("inf")
    x, g = x.to(BF16), torch.ones(272, device=DEV).to(BF16)
    q, s = run_norm(x, g, 0.0)
    assert np.isnan(f64(s[:, [0, 2]])).all() and np.isnan(f64(q[[0, 2]])).all()  # 0 / 0, NaN
    check_norm(x[1:2], None, g, 0.0, q[1:2], s[:, 1:2])
    assert np.isnan(f64(s[1, 3])) and (f64(q[3, :128]) == 0).all()  # 1 / inf; inf / inf
    q, s = run_norm(x[:1], g, 1e-5)
    assert (f64(q) == 0).all() and (f64(s) == orc.TINY).all()


# ------------------------------------------------------------------ products

def make_rows(m, k, gen, codes="normal"):
    """8-bit rows: every code (subnormal ones, both zeros) or as quantised normal values have them."""
    if codes == "every":
        q = torch.randint(0, 256, (m, k), device=DEV, dtype=torch.uint8, generator=gen)
        q[(q & 0x7F) == 0x7F] = 0x80
        q = q.view(E4M3)
    else:
        q = (torch.randn(m, k, device=DEV, generator=gen) * 150).clamp(-448, 448).to(E4M3)
    return q


def make_scales(shape, gen, size):
    return torch.exp2(torch.rand(shape, device=DEV, generator=gen) * 8 - 4) * size


def rows64(q, s):
    return q.double() * s.double().t().repeat_interleave(128, 1)[:, :q.shape[1]]


def weights64(q, s):
    return q.double() * s.double().repeat_interleave(128, -2)[..., :q.shape[-2], :].repeat_interleave(128, -1)[..., :q.shape[-1]]


class Product:
    """Operands of one product or of a grouped one, and its check."""

    def __init__(self, m, n, k, epi, groups=0, codes="normal", seed=0):
        gen = torch.Generator(DEV).manual_seed(seed * 1000 + m + n + k)
        self.m, self.n, self.k, self.epi, self.groups = m, n, k, epi, groups
        self.two = 2 if epi >= SWIGLU else 1
        g, kb, nb = max(1, groups), orc.blocks(k), orc.blocks(n)
        self.a, self.a_s = make_rows(m, k, gen, codes), make_scales((kb, m), gen, 1 / 150)
        self.b, self.b_s = make_rows(g * self.two * n, k, gen, codes).view(g, self.two, n, k), make_scales((g, self.two, nb, kb), gen, 0.02 / 150)
        if codes == "every":
            self.a_s *= 0.3
        self.r = torch.randn(m, n, device=DEV, generator=gen).to(BF16) if epi == RESID else None
        self.c = torch.full((m, n), 5.0, device=DEV).to(E4M3 if epi == SWIGLU8 else BF16)
        self.c_s = torch.full((nb, m), 3.0, device=DEV) if epi == SWIGLU8 else None

    def run(self, off=None, c=None, c_s=None, **kw):
        c, c_s = self.c if c is None else c, self.c_s if c_s is None else c_s
        if off is None:
            _lib.gemm_fp8(self.a, self.a_s, self.b.view(-1, self.k), self.b_s.squeeze(0), c, c_s=c_s, r=self.r, epilogue=self.epi, **kw)
        else:
            _lib.gemm_fp8_grouped(self.a, self.a_s, self.b.flatten(1, 2), self.b_s, off, c, c_s=c_s, epilogue=self.epi, **kw)
        return c, c_s

    def check(self, lo=0, hi=None, e=0, cols=None):
        """Rows lo ... hi - 1 against matrix e in 64 bits."""
        at = slice(lo, self.m if hi is None else hi)
        a, w = rows64(self.a, self.a_s)[at], [weights64(self.b[e, i], self.b_s[e, i]) for i in range(self.two)]
        ref, mass = [a @ x.t() for x in w], [a.abs() @ x.abs().t() for x in w]
        err = 128 * 2.0 ** -23 + (orc.blocks(self.k) + 3) * 2.0 ** -24
        if self.two == 1:
            want, tol = ref[0], err * mass[0]
            if self.epi == RESID:
                want = want + self.r[at].double()
                tol = tol + 2.0 ** -24 * want.abs()
        else:
            gate, up = ref
            want = gate * torch.sigmoid(gate) * up
            tol = err * (1.1 * mass[0] * up.abs() + mass[1] * gate.abs() + err * mass[0] * mass[1]) + 2.0 ** -19 * want.abs()
        if self.epi != SWIGLU8:
            assert ((self.c[at].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
            return
        n = self.n
        top = torch.stack([want[:, i:i + 128].abs().amax(1) for i in range(0, n, 128)])
        far = torch.stack([tol[:, i:i + 128].amax(1) for i in range(0, n, 128)])
        s = self.c_s[:, at].double()
        assert ((s - (top / 448).clamp(min=orc.TINY)).abs() <= far / 448 + 2.0 ** -22 * s).all()
        got, u = self.c[at].double(), want / s.t().repeat_interleave(128, 1)[:, :n]
        ut = tol / s.t().repeat_interleave(128, 1)[:, :n]
        assert ((got - u).abs() <= torch.clamp(2.0 ** -4 * (u.abs() + ut), min=2.0 ** -10) + ut + 2.0 ** -20 * u.abs()).all()


SIZES = [(1, 8, 16), (1, 16, 128), (2, 136, 144), (3, 256, 256), (17, 264, 272), (64, 128, 1024), (65, 688, 256), (127, 256, 688), (128, 512, 128), (129, 520, 2064),
         (200, 1000, 400), (256, 256, 384), (300, 96, 4096), (1000, 384, 512), (1, 4096, 14336), (8, 512, 28672), (333, 2048, 1024)]


@pytest.mark.parametrize("epi", [STORE, RESID, SWIGLU, SWIGLU8])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm(m, n, k, epi):
    p = Product(m, n - n % 16 if epi == SWIGLU8 and n > 16 else max(n, 16) if epi == SWIGLU8 else n, k, epi)
    p.run()
    _lib.fp8_poll()
    p.check()


@pytest.mark.parametrize("epi", [STORE, RESID, SWIGLU, SWIGLU8])
@pytest.mark.parametrize("m,n,k", [(129, 24, 2048), (129, 520, 2064), (300, 1400, 4080), (129, 520, 4112), (260, 1040, 4096), (400, 264, 14336)])
def test_gemm_cut_along_k(m, n, k, epi):
    """Tiles for a part of the GPU: two and four CTAs a tile, in place as well."""
    p = Product(m, n - n % 16 if epi == SWIGLU8 else n, k, epi)
    p.run()
    _lib.fp8_poll()
    p.check()
    if epi == RESID:
        c = p.r.clone()
        _lib.gemm_fp8(p.a, p.a_s, p.b.view(-1, p.k), p.b_s.squeeze(0), c, r=c, epilogue=RESID)
        assert torch.equal(c, p.c)


@pytest.mark.parametrize("epi", [STORE, RESID, SWIGLU8])
@pytest.mark.parametrize("m,n,k", [(1, 10256, 1040), (40, 12304, 528), (65, 12304, 528), (20, 24592, 400), (33, 24592, 144), (17, 40016, 80)])
def test_gemm_few_rows_many_columns(m, n, k, epi):
    """Around the bounds of the kernel for few rows: two CTAs an SM, and more tiles than the GPU holds at once."""
    p = Product(m, n, k, epi)
    p.run()
    _lib.fp8_poll()
    p.check()


@pytest.mark.parametrize("epi", [STORE, SWIGLU8])
@pytest.mark.parametrize("counts,n,k", [([70, 0, 64, 33, 90], 272, 2064), ([40, 20, 33], 528, 1040), ([1, 130, 2], 144, 1040), ([16] * 16 + [0] * 4, 2064, 528)])
def test_grouped_rows_between(counts, n, k, epi):
    p = Product(sum(counts), n, k, epi, groups=len(counts))
    p.run(offsets(counts))
    _lib.fp8_poll()
    at = 0
    for e, c in enumerate(counts):
        if c:
            p.check(at, at + c, e)
        at += c


@pytest.mark.parametrize("epi", [STORE, SWIGLU8])
@pytest.mark.parametrize("m", [5, 300])
def test_gemm_of_every_code(m, epi):
    p = Product(m, 272, 528, epi, codes="every")
    p.run()
    p.check()


def test_gemm_adds_up_in_fp32():
    """Large and small products in one block, equal up to their order: a sum held in fewer bits than fp32 would lose the small ones."""
    for m in (1, 256):
        p = Product(m, 128, 1024, STORE)
        p.a_s.fill_(1.0), p.b_s.fill_(1.0)
        a, b = torch.zeros(m, 1024, device=DEV), torch.zeros(128, 1024, device=DEV)
        a[:, ::128], b[:, ::128] = 448, 448          # 448 * 448 a block, and in the next one its negative
        b[:, 128::256] = -448
        a[:, 1::2], b[:, 1::2] = 1, 1                # 512 ones
        p.a, p.b = a.to(E4M3), b.to(E4M3).view(1, 1, 128, 1024)
        p.run()
        assert (p.c.float() == 512).all()


@pytest.mark.parametrize("m", [4, 200])
@pytest.mark.parametrize("epi", [STORE, SWIGLU8])
def test_gemm_nan_scales_stay_in_their_rows_and_columns(m, epi):
    p = Product(m, 384, 272, epi)
    clean = [None if t is None else t.clone() for t in p.run()]
    p.a_s[1, 2] = float("nan")
    p.b_s[0, 0, 1, 0] = float("nan")
    p.run()
    bad = torch.zeros(m, 384, dtype=torch.bool, device=DEV)
    bad[2], bad[:, 128:256] = True, True
    assert torch.isnan(p.c.float())[bad].all() and torch.equal(p.c.float()[~bad], clean[0].float()[~bad])
    if epi == SWIGLU8:
        assert torch.isnan(p.c_s[:, 2]).all() and torch.isnan(p.c_s[1]).all() and not torch.isnan(p.c_s[[0, 2]][:, :2]).any()


@pytest.mark.parametrize("m", [3, 300])
def test_gemm_residual_in_place(m):
    p = Product(m, 264, 272, RESID)
    p.run()
    c = p.r.clone()
    _lib.gemm_fp8(p.a, p.a_s, p.b.view(-1, p.k), p.b_s.squeeze(0), c, r=c, epilogue=RESID)
    assert torch.equal(c, p.c)


@pytest.mark.parametrize("m,max_sms", [(5, 1), (5, 7), (700, 1), (700, 3), (700, 1000)])
def test_gemm_grid_limits_change_nothing(m, max_sms):
    p = Product(m, 520, 400, SWIGLU)
    want = p.run()[0].clone()
    p.run(max_sms=max_sms)
    assert torch.equal(p.c, want)


@pytest.mark.parametrize("epi", [STORE, RESID, SWIGLU, SWIGLU8])
@pytest.mark.parametrize("m,n,k", [(700, 1040, 400), (129, 4112, 144), (1030, 528, 1040)])
def test_many_tiles_a_cta(m, n, k, epi):
    """Few CTAs walk many tiles: rings, accumulators and the exchange of the largest values go on across tiles."""
    p = Product(m, n, k, epi)
    p.run(max_sms=3)
    _lib.fp8_poll()
    p.check()
    want = p.c.float().clone()
    p.run(max_sms=2)
    assert torch.equal(p.c.float(), want)


def offsets(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=I32, device=DEV)


@pytest.mark.parametrize("epi", [STORE, SWIGLU, SWIGLU8])
@pytest.mark.parametrize("counts,n,k", [([5], 264, 272), ([0, 1, 0, 130, 3, 0], 144, 400), ([128, 256, 1], 256, 128), ([0, 0, 0], 128, 128), ([300, 40, 129, 64, 2, 90], 688, 256),
                                        ([1] * 128, 80, 144), ([2, 1, 0, 3, 1, 0, 0, 1], 512, 2048), ([0] * 100 + [7] + [0] * 27, 48, 64)])
def test_grouped(counts, n, k, epi):
    """Each group with its matrix; rows before the first and behind the last group stay as they are."""
    if epi == SWIGLU8:
        n -= n % 16
    first, tail = 3, 9
    m = first + sum(counts) + tail
    p = Product(m, n, k, epi, groups=len(counts))
    p.run(offsets(counts, first))
    _lib.fp8_poll()
    at = first
    for e, c in enumerate(counts):
        if c:
            p.check(at, at + c, e)
        at += c
    for rows in (slice(0, first), slice(m - tail, m)):
        assert (p.c[rows].float() == 5).all()
        assert p.c_s is None or (p.c_s[:, rows] == 3).all()


@pytest.mark.parametrize("epi", [STORE, SWIGLU8])
def test_grouped_many_tiles_a_cta(epi):
    counts = [130, 0, 257, 3, 128, 40]
    p = Product(sum(counts), 528, 656, epi, groups=len(counts))
    p.run(offsets(counts), max_sms=3)
    at = 0
    for e, c in enumerate(counts):
        if c:
            p.check(at, at + c, e)
        at += c


@pytest.mark.parametrize("m", [40, 500])
def test_grouped_offsets_outside_and_in_disorder(m):
    """Offsets count within [0, m], one below the one before it as that one."""
    p = Product(m, 144, 272, STORE, groups=6)
    p.run(torch.tensor([-5, 10, 4, 20, m + 100, 7, 2147483647], dtype=I32, device=DEV))
    for e, (lo, hi) in enumerate([(0, 10), (10, 10), (10, 20), (20, m), (m, m), (m, m)]):
        if hi > lo:
            p.check(lo, hi, e)


@pytest.mark.parametrize("m", [6, 600])
def test_grouped_nan_of_another_group_does_not_spread(m):
    p = Product(m, 144, 272, STORE, groups=3)
    off = offsets([m // 3] * 3)
    want = p.run(off)[0].clone()
    p.a_s[:, m // 3:2 * (m // 3)] = float("nan")
    p.b_s[1] = float("nan")
    p.run(off)
    keep = torch.ones(m, dtype=torch.bool, device=DEV)
    keep[m // 3:2 * (m // 3)] = False
    assert torch.equal(p.c[keep], want[keep]) and torch.isnan(p.c[~keep].float()).all()


@pytest.mark.parametrize("call", ["norm", "quant", "weights", "gemm", "grouped"])
def test_no_rows(call):
    e = lambda *n, t=BF16: empty(*n, t=t)  # noqa: E731
    if call == "norm":
        _lib.rmsnorm_fp8(e(0, 64), e(64), e(0, 64, t=E4M3), e(1, 0, t=F32), 1e-5)
    elif call == "quant":
        _lib.quant_fp8(e(0, 64), e(0, 64, t=E4M3), e(1, 0, t=F32))
        q, s = quant(e(0, 64), torch.zeros(2, dtype=I32, device=DEV))  # nothing to take rows from
        assert (f64(q) == 0).all() and (f64(s) == orc.TINY).all()
    elif call == "weights":
        _lib.quant_fp8_weights(e(0, 64, 64), e(0, 64, 64, t=E4M3), e(0, 1, 1, t=F32))
    elif call == "gemm":
        _lib.gemm_fp8(e(0, 64, t=E4M3), e(1, 0, t=F32), e(8, 64, t=E4M3), e(1, 1, t=F32), e(0, 8))
    else:
        _lib.gemm_fp8_grouped(e(0, 64, t=E4M3), e(1, 0, t=F32), e(2, 8, 64, t=E4M3), e(2, 1, 1, t=F32), offsets([0, 0]), e(0, 8))
    torch.cuda.synchronize()


# ------------------------------------------------------------------ streams, graphs, far offsets

@pytest.mark.parametrize("m,groups", [(9, 0), (300, 0), (9, 3), (600, 3)])
def test_two_streams_at_once_and_a_graph(m, groups):
    """Calls that run at once share nothing, and a captured call gives what a single one does, bit for bit."""
    ps = [Product(m, 528, 1040, SWIGLU8, groups=groups, seed=i) for i in range(2)]
    off = offsets([m // 3] * 3) if groups else None
    want = [[t.clone() for t in p.run(off)] for p in ps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[[torch.full_like(t.float(), 5 if t.dtype == E4M3 else 3).to(t.dtype) for t in w] for _ in range(6)] for w in want]
    torch.cuda.synchronize()
    for i in range(6):
        for p, o, st in zip(ps, outs, streams):
            p.run(off, *o[i], stream=st)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for c, s in o:
            assert torch.equal(c.view(torch.uint8), w[0].view(torch.uint8)) and torch.equal(s, w[1])
    p, w = ps[0], want[0]
    c, s = torch.zeros_like(p.c.float()).to(E4M3), torch.zeros_like(p.c_s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(off, c, s)
    rows = slice(0, m // 3 * 3)
    for _ in range(3):
        c.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c[rows].view(torch.uint8), w[0][rows].view(torch.uint8)) and torch.equal(s[:, rows], w[1][:, rows])
    if groups:  # the offsets are read at each replay
        off.copy_(offsets([0, m // 3, m // 3]))
        graph.replay()
        p.run(off)
        torch.cuda.synchronize()
        assert torch.equal(c[:m // 3 * 2].view(torch.uint8), p.c[:m // 3 * 2].view(torch.uint8))


@pytest.mark.parametrize("m", [1, 40, 200, 700])
def test_a_chain_over_the_same_buffers(m):
    """Each call reads what the one ahead wrote to buffers that were read before: one after the other without a wait, captured, and with a wait after each call."""
    n, f = 1024, 528
    up, down = Product(m, f, n, SWIGLU8, seed=5), Product(m, n, f, RESID, seed=6)
    up.b_s.mul_(0.05), down.b_s.mul_(0.05)
    x0 = torch.randn(m, n, device=DEV).bfloat16()
    g = torch.ones(n, device=DEV, dtype=BF16)
    x, h = x0.clone(), torch.zeros_like(x0)
    q, s = torch.zeros(m, n, device=DEV).to(E4M3), torch.zeros(n // 128, m, device=DEV)
    c, c_s = torch.zeros(m, f, device=DEV).to(E4M3), torch.zeros((f + 127) // 128, m, device=DEV)

    def pair(out, res):
        return [lambda: _lib.gemm_fp8(q, s, up.b.view(-1, n), up.b_s.squeeze(0), c, c_s=c_s, epilogue=SWIGLU8),
                lambda: _lib.gemm_fp8(c, c_s, down.b.view(-1, f), down.b_s.squeeze(0), out, r=res, epilogue=RESID)]

    calls = [lambda: _lib.rmsnorm_fp8(x, g, q, s, 1e-5, r=x0, h=h), *pair(h, h), lambda: _lib.quant_fp8(h, q, s), *pair(x, x0)] * 8

    def layers(wait):
        for call in calls:
            call()
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return x.clone(), h.clone()

    want = layers(True)
    assert torch.isfinite(want[0]).all() and not torch.equal(want[0], x0)
    for _ in range(5):
        x.copy_(x0)
        assert all(torch.equal(a, b) for a, b in zip(layers(False), want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.copy_(x0)
        for call in calls:
            call()
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(h, want[1])
    _lib.fp8_poll()


@pytest.mark.parametrize("m,n,k,epi", [(129, 528, 4112, SWIGLU), (129, 528, 4112, SWIGLU8), (257, 528, 2064, SWIGLU8), (130, 520, 4112, RESID), (1, 528, 14336, SWIGLU), (3, 1040, 8192, STORE)])
def test_clusters_whose_rows_end_early_beside_others(m, n, k, epi):
    """CTAs of a cluster that store little end while peers still read their sums, on two streams that fill each other's SMs: the same bits at each call."""
    ps = [Product(m, n, k, epi, seed=i) for i in (7, 8)]
    want = [p.run()[0].float().clone() for p in ps]
    ps[0].check(), ps[1].check()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[(torch.zeros_like(p.c.float()).to(p.c.dtype), None if p.c_s is None else torch.zeros_like(p.c_s)) for _ in range(40)] for p in ps]
    torch.cuda.synchronize()
    for i in range(40):
        for p, o, st in zip(ps, outs, streams):
            p.run(None, *o[i], stream=st)
    torch.cuda.synchronize()
    _lib.fp8_poll()
    for w, o in zip(want, outs):
        assert all(torch.equal(c.float(), w) for c, _ in o)


def test_two_threads_at_once():
    """Calls from two host threads, each on a stream of its own."""
    import threading
    ps = [Product(9, 528, 1040, SWIGLU8, seed=3), Product(300, 520, 2064, STORE, seed=4)]
    want = [p.run()[0].float().clone() for p in ps]
    outs, errors = [[], []], []

    def work(i):
        try:
            st, p = torch.cuda.Stream(), ps[i]
            for _ in range(30):
                c = torch.zeros_like(p.c.float()).to(p.c.dtype)
                st.wait_stream(torch.cuda.current_stream())
                outs[i].append(p.run(None, c, None if p.c_s is None else torch.zeros_like(p.c_s), stream=st)[0])
            st.synchronize()
        except Exception as e:  # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors
    for i in range(2):
        assert len(outs[i]) == 30 and all(torch.equal(c.float(), want[i]) for c in outs[i])


def test_results_repeat_bit_for_bit():
    for m, k in ((1, 14336), (40, 8192), (700, 1024)):
        p = Product(m, 1024, k, STORE)
        want = p.run()[0].clone()
        for _ in range(20):
            assert torch.equal(p.run()[0], want)


def test_weights_past_32_bits():
    """More than 2^32 bytes of experts' matrices: the last one's rows."""
    n, k, groups = 8192, 8192, 65
    b = torch.zeros(groups, n, k, dtype=torch.uint8, device=DEV).view(E4M3)
    b_s = torch.full((groups, 64, 64), 2.0 ** -8, device=DEV)
    for m in (5, 200):
        p = Product(m, n, k, STORE)
        b[-1] = p.b[0, 0]
        c = empty(m, n)
        _lib.gemm_fp8_grouped(p.a, p.a_s, b, b_s, torch.tensor([0] * groups + [m], dtype=I32, device=DEV), c)
        p.c, p.b_s = c, b_s[:1, None]
        p.check()


def test_rows_past_32_bits():
    """Outputs, rows and quantised values at offsets past 2^32 bytes."""
    m, n, k = 140000, 16384, 128
    p = Product(m, n, k, STORE)
    p.run()
    for lo in (0, 131070, m - 130):
        p.check(lo, lo + 130)
    x = torch.randn(m, n, device=DEV, dtype=BF16)
    q, s = quant(x)
    want = orc.quantise_rows(x[-2:].float().cpu().numpy())
    same(f64(q[-2:]), want[0]), same(f64(s[:, -2:]), want[1])


def test_binding_refuses_tensors_of_another_place():
    p = Product(3, 144, 272, STORE)
    with pytest.raises(ValueError, match="cpu"):
        p.b = p.b.cpu()
        p.run()


@pytest.mark.parametrize("limit", [1, 500, 2000, 20000])
@pytest.mark.parametrize("m,n,epi,groups", [(5, 1024, STORE, 0), (64, 512, SWIGLU8, 0), (300, 512, RESID, 0), (700, 5200, SWIGLU8, 0), (900, 528, STORE, 3), (12, 528, SWIGLU, 3)])
def test_limits_shorter_than_the_waits(m, n, epi, groups, limit):
    """A wait that gives up is reported once, or nothing gave up and the result is right; the next call is as ever."""
    p = Product(m, n, 2064, epi, groups=groups)
    short_limit(p, limit, offsets([m // 3] * 3) if groups else None, m // 3 * 3 if groups else m)


@pytest.mark.parametrize("limit", [1, 500, 2000, 20000])
@pytest.mark.parametrize("epi", [RESID, SWIGLU, SWIGLU8])
def test_limits_shorter_than_the_waits_of_four_ctas(epi, limit):
    short_limit(Product(300, 528, 4112, epi), limit, None, 300)


def short_limit(p, limit, off, rows):
    want = p.run(off)[0].float().clone()
    _lib.fp8_poll()
    try:
        _lib.fp8_set_timeout(limit)
        p.run(off)
        try:
            _lib.fp8_poll()
            assert torch.equal(p.c.float()[:rows], want[:rows])
        except _lib.NanoflowError as e:
            assert e.code == _lib.NF_ERR_TIMEOUT
    finally:
        _lib.fp8_set_timeout(2_000_000_000)
    _lib.fp8_poll()
    p.run(off)
    _lib.fp8_poll()
    assert torch.equal(p.c.float()[:rows], want[:rows])


def _told():
    try:
        _lib.fp8_poll()
        return False
    except _lib.NanoflowError as e:
        assert e.code == _lib.NF_ERR_TIMEOUT
        return True


def _in_a_thread(f):
    import threading
    out = []
    t = threading.Thread(target=lambda: out.append(f()))
    t.start()
    t.join()
    return out[0]


@pytest.mark.parametrize("m,n,k", [(900, 5200, 2064), (64, 4096, 14336)])
def test_polls_of_several_threads_take_no_report_from_one_another(m, n, k):
    """A product that gave up is reported to its caller although another thread's poll came first, to each thread once."""
    p = Product(m, n, k, STORE)
    p.run()
    _told()
    for _ in range(20):
        try:
            _lib.fp8_set_timeout(1)
            p.run()
        finally:
            _lib.fp8_set_timeout(2_000_000_000)
        assert not _in_a_thread(lambda: (_told(), _told()))[1]
        mine = _told()
        if mine:
            break
    assert mine  # a limit of a nanosecond: some wait of 20 calls ran out
    assert not _told()

    def product_then_poll():  # a thread that begins with a product is not told of what was reported before
        c = torch.zeros_like(p.c)
        _lib.gemm_fp8(p.a, p.a_s, p.b.view(-1, p.k), p.b_s.squeeze(0), c)
        return _told()

    assert not _in_a_thread(product_then_poll)
    p.run()
    assert not _told()
    p.check()


def test_a_poll_inside_a_capture_is_refused_and_the_capture_goes_on():
    p = Product(5, 528, 1040, STORE)
    want = p.run()[0].clone()
    _told()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(_lib.NanoflowError, match="captured") as e:
            _lib.fp8_poll()
        p.run()
    assert e.value.code == _lib.NF_ERR_INVALID_ARG
    p.c.zero_()
    graph.replay()
    _lib.fp8_poll()
    assert torch.equal(p.c, want)


def test_first_call_of_a_process_in_a_capture():
    """Nothing is allocated or looked up that a capture forbids."""
    code = """
import torch
from nano_intra_device_gb300 import _lib
e = torch.float8_e4m3fn
x = torch.randn(200, 256, device="cuda").bfloat16()
q, s, c = torch.zeros(200, 256, device="cuda").to(e), torch.zeros(2, 200, device="cuda"), torch.zeros(200, 128, device="cuda").bfloat16()
w, ws, d = torch.zeros(128, 256, device="cuda").to(e), torch.ones(1, 2, device="cuda"), torch.ones(3, 128, device="cuda").bfloat16()
w.view(torch.uint8).fill_(0x38)  # ones
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    _lib.quant_fp8(x, q, s)
    _lib.gemm_fp8(q, s, w, ws, c)
    _lib.gemm_fp8(q[:3], s[:, :3].contiguous(), w, ws, d)
g.replay()
torch.cuda.synchronize()
_lib.fp8_poll()
want = x.float().sum(1, keepdim=True)
assert (c.float() - want).abs().max() < 4, (c.float() - want).abs().max()
print("captured")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_first_cut_of_a_process_in_a_capture(tmp_path):
    """K long enough for every cut: clusters are counted and launched for the first time inside a capture, with the results of calls outside one."""
    code = """
import sys
import torch
from nano_intra_device_gb300 import _lib
e = torch.float8_e4m3fn
gen = torch.Generator("cuda").manual_seed(1)
def case(m, n, k, epi, top=1e9):  # without a limit a few codes are NaN (beyond 464), and their rows or columns
    two = 2 if epi >= 2 else 1
    a = (torch.randn(m, k, device="cuda", generator=gen) * 100).clamp(-top, top).to(e)
    b = (torch.randn(two * n, k, device="cuda", generator=gen) * 100).clamp(-top, top).to(e)
    a_s, b_s = torch.rand(k // 128, m, device="cuda", generator=gen) / 100, torch.rand(two, (n + 127) // 128, k // 128, device="cuda", generator=gen) / 100
    c = torch.zeros(m, n, device="cuda").to(e if epi == 3 else torch.bfloat16)
    return dict(a=a, a_s=a_s, b=b, b_s=b_s, c=c, c_s=torch.zeros((n + 127) // 128, m, device="cuda") if epi == 3 else None, epilogue=epi)
cases = [case(200, 528, 4096, 0), case(200, 528, 2048, 3), case(3, 528, 4096, 0), case(3, 528, 4096, 2)]
cases += [case(200, 528, 4096, 0, 448), case(200, 528, 2048, 3, 448), case(3, 528, 4096, 0, 448), case(3, 528, 4096, 2, 448)]
if sys.argv[1] == "captured":
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in cases:
            _lib.gemm_fp8(**c)
    g.replay()
else:
    for c in cases:
        _lib.gemm_fp8(**c)
torch.cuda.synchronize()
_lib.fp8_poll()
for i, c in enumerate(cases):
    b = c["b"].float().view(-1, c["c"].shape[1], c["a"].shape[1])
    w = [x * s.repeat_interleave(128, 0)[:len(x)].repeat_interleave(128, 1) for x, s in zip(b.double(), c["b_s"].double())]
    y = [(c["a"].double() * c["a_s"].double().t().repeat_interleave(128, 1)) @ x.t() for x in w]
    if c["epilogue"] >= 2:
        y = [y[0] * torch.sigmoid(y[0]) * y[1]]
    got = c["c"].double() * (c["c_s"].double().t().repeat_interleave(128, 1)[:, :c["c"].shape[1]] if c["c_s"] is not None else 1)
    nan = torch.isnan(y[0])
    assert i < 4 or not nan.any()
    if c["epilogue"] == 3:  # a NaN makes its block of 128 NaN
        nan = torch.cat([p.any(1, keepdim=True).expand_as(p) for p in nan.split(128, 1)], 1)
    assert torch.equal(torch.isnan(got), nan)
    d, want = (got - y[0])[~nan], y[0][~nan]
    assert d.norm() <= 2.0 ** -4 * want.norm(), d.norm() / want.norm()
torch.save([c["c"].float().cpu() for c in cases], sys.argv[2])
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    outs = []
    for how in ("captured", "called"):
        out = tmp_path / how
        r = subprocess.run([sys.executable, "-c", code, how, str(out)], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        outs.append(torch.load(out))
    # equal bits, so the same cuts: a cut left out would add up in another order
    assert all(torch.equal(a.nan_to_num(1e9), b.nan_to_num(1e9)) for a, b in zip(*outs))


# ------------------------------------------------------------------ products cut along K

CUT = [(200, 528, 2064), (200, 528, 4112)]  # tiles that leave room for two CTAs each, and for four (16 and 32 blocks of K)


@pytest.mark.parametrize("epi", [STORE, RESID, SWIGLU, SWIGLU8])
@pytest.mark.parametrize("m,n,k", CUT)
def test_cut_products_repeat_in_a_graph_and_on_two_streams(m, n, k, epi):
    ps = [Product(m, n, k, epi, seed=i) for i in (11, 12)]
    want = [p.run()[0].float().clone() for p in ps]
    ps[0].check(), ps[1].check()
    for _ in range(20):
        assert torch.equal(ps[0].run()[0].float(), want[0])
    new = lambda p: (torch.zeros_like(p.c.float()).to(p.c.dtype), None if p.c_s is None else torch.zeros_like(p.c_s))  # noqa: E731
    outs, streams = [[new(p) for _ in range(10)] for p in ps], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(10):
        for p, o, st in zip(ps, outs, streams):
            p.run(None, *o[i], stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(c.float(), w) for w, o in zip(want, outs) for c, _ in o)
    out = new(ps[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            ps[0].run(None, *out)
    for _ in range(3):
        out[0].view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0].float(), want[0])
    _lib.fp8_poll()


@pytest.mark.parametrize("m,k", [(200, 2048), (200, 4096), (40, 4096)])
def test_a_chain_of_cut_products_over_the_same_buffers(m, k):
    """Each call reads what the one ahead wrote, without a wait and captured, as with a wait after each."""
    up, down = Product(m, k, k, SWIGLU8, seed=13), Product(m, k, k, RESID, seed=14)
    up.b_s.mul_(0.02), down.b_s.mul_(0.02)
    x0 = torch.randn(m, k, device=DEV).bfloat16()
    x, g = x0.clone(), torch.ones(k, device=DEV, dtype=BF16)
    q, s = torch.zeros(m, k, device=DEV).to(E4M3), torch.zeros(k // 128, m, device=DEV)
    c, c_s = torch.zeros(m, k, device=DEV).to(E4M3), torch.zeros(k // 128, m, device=DEV)
    calls = [lambda: _lib.rmsnorm_fp8(x, g, q, s, 1e-5),
             lambda: _lib.gemm_fp8(q, s, up.b.view(-1, k), up.b_s.squeeze(0), c, c_s=c_s, epilogue=SWIGLU8),
             lambda: _lib.gemm_fp8(c, c_s, down.b.view(-1, k), down.b_s.squeeze(0), x, r=x, epilogue=RESID)] * 6

    def layers(wait):
        x.copy_(x0)
        for call in calls:
            call()
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return x.clone()

    want = layers(True)
    assert torch.isfinite(want).all() and not torch.equal(want, x0)
    for _ in range(5):
        assert torch.equal(layers(False), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(x0)
        for call in calls:
            call()
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)
    _lib.fp8_poll()


@pytest.mark.parametrize("epi", [STORE, RESID, SWIGLU, SWIGLU8])
@pytest.mark.parametrize("m,n,k", CUT)
def test_cut_products_under_limits_of_the_grid(m, n, k, epi):
    """Limits that leave the cut in four, in two and none; with none the sums of K's parts are one sum."""
    p = Product(m, n, k, epi)
    for max_sms in (0, 151, 80, 40, 20, 10, 1):
        p.c.view(torch.uint8).zero_()
        p.run(max_sms=max_sms)
        _lib.fp8_poll()
        p.check()


@pytest.mark.parametrize("epi", [STORE, SWIGLU8])
@pytest.mark.parametrize("m,n,k", CUT)
def test_cut_products_of_every_code(m, n, k, epi):
    p = Product(m, n, k, epi, codes="every")
    p.run()
    p.check()


@pytest.mark.parametrize("k", [2048, 4096])
def test_cut_products_add_up_in_fp32(k):
    """As test_gemm_adds_up_in_fp32, with the large products and their negatives in every CTA's part of K."""
    p = Product(200, 128, k, STORE)
    p.a_s.fill_(1.0), p.b_s.fill_(1.0)
    a, b = torch.zeros(200, k, device=DEV), torch.zeros(128, k, device=DEV)
    a[:, ::128], b[:, ::128] = 448, 448
    b[:, 128::256] = -448
    a[:, 1::2], b[:, 1::2] = 1, 1
    p.a, p.b = a.to(E4M3), b.to(E4M3).view(1, 1, 128, k)
    p.run()
    assert (p.c.float() == k // 2).all()


@pytest.mark.parametrize("epi", [STORE, SWIGLU, SWIGLU8])
@pytest.mark.parametrize("k", [2064, 4112])
def test_cut_products_keep_nan_scales_in_their_rows_and_columns(epi, k):
    """A NaN in the part of K of one CTA, for a row in the columns or rows that another one finishes."""
    p = Product(200, 384, k, epi)
    clean = [None if t is None else t.clone() for t in p.run()]
    p.a_s[1, 2] = p.a_s[-1, 70] = float("nan")
    p.b_s[0, 0, 1, -1] = float("nan")
    p.run()
    bad = torch.zeros(200, 384, dtype=torch.bool, device=DEV)
    bad[[2, 70]], bad[:, 128:256] = True, True
    assert torch.isnan(p.c.float())[bad].all() and torch.equal(p.c.float()[~bad], clean[0].float()[~bad])
    if epi == SWIGLU8:
        rest = [i for i in range(200) if i not in (2, 70)]
        assert torch.isnan(p.c_s[:, [2, 70]]).all() and torch.isnan(p.c_s[1]).all() and torch.equal(p.c_s[[0, 2]][:, rest], clean[1][[0, 2]][:, rest])


@pytest.mark.parametrize("m", [3, 200])
def test_cut_products_with_infinite_sums(m):
    """Sums that leave fp32's range in one CTA's part of K: infinities in their rows, the others as ever."""
    p = Product(m, 384, 4096, STORE)
    p.a = p.a.float().abs().to(E4M3)
    p.b = p.b.float().abs().to(E4M3)
    clean = p.run()[0].clone()
    p.a_s[5, 1] = 1e33  # times 223 and a block's sum of some 10^6
    p.b_s[0, 0, :, 5] = 1e5 / 448
    rest = [i for i in range(m) if i != 1]
    want = p.run()[0].clone()
    assert torch.isinf(want[1]).all() and torch.isfinite(clean).all() and torch.isfinite(want[rest]).all()
    p.a_s[5, 1] = 1 / 150
    p.run()
    p.check()
    assert torch.equal(p.c[rest], want[rest])


# ------------------------------------------------------------------ together

def quant_rows64(y):
    """Oracle codes and scales of float64 values rounded to fp32."""
    return orc.quantise_rows(y.astype(np.float32))


@pytest.mark.parametrize("tokens", [1, 37, 260])
def test_the_ffn_of_a_layer(tokens):
    """The small layer's second half in 8 bits: norm with the residual, gate and up, down and its residual, as
    one captured graph; each stage against float64 from the stage before."""
    hidden, ffn = 256, 688
    gen = torch.Generator(DEV).manual_seed(tokens)
    rnd = lambda *n, std=1.0: (torch.randn(n, device=DEV, generator=gen) * std).to(BF16)  # noqa: E731
    x, o, g = rnd(tokens, hidden), rnd(tokens, hidden, std=0.5), 1 + rnd(hidden, std=0.1)
    wgu, wd = rnd(2, ffn, hidden, std=0.05), rnd(hidden, ffn, std=0.05)
    q_gu, s_gu, q_d, s_d = empty(2, ffn, hidden, t=E4M3), empty(2, 6, 2, t=F32), empty(hidden, ffn, t=E4M3), empty(2, 6, t=F32)
    _lib.quant_fp8_weights(wgu, q_gu, s_gu)
    _lib.quant_fp8_weights(wd, q_d, s_d)
    h, n2, n2_s = empty(tokens, hidden), empty(tokens, hidden, t=E4M3), empty(2, tokens, t=F32)
    a, a_s, y = empty(tokens, ffn, t=E4M3), empty(6, tokens, t=F32), empty(tokens, hidden)

    def step():
        _lib.rmsnorm_fp8(x, g, n2, n2_s, 1e-5, r=o, h=h)
        _lib.gemm_fp8(n2, n2_s, q_gu.view(2 * ffn, hidden), s_gu, a, c_s=a_s, epilogue=SWIGLU8)
        _lib.gemm_fp8(a, a_s, q_d, s_d, y, r=h, epilogue=RESID)

    step()
    first = [t.clone() for t in (h, n2_s, a_s, y)]
    check_norm(x, o, g, 1e-5, n2, n2_s)
    p = Product(tokens, ffn, hidden, SWIGLU8)
    p.a, p.a_s, p.b, p.b_s, p.c, p.c_s = n2, n2_s, q_gu[None], s_gu[None], a, a_s
    p.check()
    p = Product(tokens, hidden, ffn, RESID)
    p.a, p.a_s, p.b, p.b_s, p.r, p.c = a, a_s, q_d[None, None], s_d[None, None], h, y
    p.check()
    # the whole beside the same in float64 without 8 bits: each of the three quantised operands errs by
    # 2^-4 of a value at most, uniformly spread, so by some 2^-4 / sqrt(3) in the root mean square
    hh, n64 = orc.norm(f64(x), f64(o), f64(g), 1e-5)
    w = f64(wgu)
    far = f64(y) - hh - orc.swiglu(n64 @ w[0].T, n64 @ w[1].T) @ f64(wd).T
    assert np.sqrt((far ** 2).mean()) <= 0.1 * np.sqrt(((f64(y) - hh) ** 2).mean())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (h, n2_s, a_s, y):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for t, w in zip((h, n2_s, a_s, y), first):
        assert torch.equal(t, w)


@pytest.mark.parametrize("tokens", [1, 19, 300])
def test_the_experts_of_a_layer(tokens):
    """Top-2 of 4 experts in 8 bits: the tokens' rows in the experts' order, gate and up, down, and the
    weighted sum; against float64 of the same 8-bit operands, stage by stage."""
    hidden, ffn, experts = 256, 688, 4
    gen = torch.Generator(DEV).manual_seed(tokens)
    rnd = lambda *n, std=1.0: (torch.randn(n, device=DEV, generator=gen) * std).to(BF16)  # noqa: E731
    x, g = rnd(tokens, hidden), 1 + rnd(hidden, std=0.1)
    wgu, wd = rnd(experts, 2, ffn, hidden, std=0.05), rnd(experts, hidden, ffn, std=0.05)
    q_gu, s_gu, q_d, s_d = empty(experts, 2, ffn, hidden, t=E4M3), empty(experts, 2, 6, 2, t=F32), empty(experts, hidden, ffn, t=E4M3), empty(experts, 2, 6, t=F32)
    _lib.quant_fp8_weights(wgu, q_gu, s_gu)
    _lib.quant_fp8_weights(wd, q_d, s_d)
    logits = torch.randn(tokens, experts, device=DEV, generator=gen)
    top, chosen = logits.topk(2, dim=1)
    order = chosen.flatten().argsort(stable=True)
    token, off = (order // 2).int(), offsets(torch.bincount(chosen.flatten(), minlength=experts).cpu().numpy())
    rows = 2 * tokens
    n2, q, s = empty(tokens, hidden), empty(rows, hidden, t=E4M3), empty(2, rows, t=F32)
    a, a_s, part = empty(rows, ffn, t=E4M3), empty(6, rows, t=F32), empty(rows, hidden)
    _lib.rmsnorm(x, g, n2, 1e-5)
    _lib.quant_fp8(n2, q, s, index=token)
    _lib.gemm_fp8_grouped(q, s, q_gu.view(experts, 2 * ffn, hidden), s_gu, off, a, c_s=a_s, epilogue=SWIGLU8)
    _lib.gemm_fp8_grouped(a, a_s, q_d, s_d, off, part)
    _lib.fp8_poll()
    want = orc.quantise_rows(n2[token.long()].float().cpu().numpy())
    same(f64(q), want[0]), same(f64(s), want[1])
    bounds = off.tolist()
    up, down = Product(rows, ffn, hidden, SWIGLU8), Product(rows, hidden, ffn, STORE)
    up.a, up.a_s, up.b, up.b_s, up.c, up.c_s = q, s, q_gu, s_gu, a, a_s
    down.a, down.a_s, down.b, down.b_s, down.c = a, a_s, q_d[:, None], s_d[:, None], part
    for e in range(experts):
        if bounds[e + 1] > bounds[e]:
            up.check(bounds[e], bounds[e + 1], e), down.check(bounds[e], bounds[e + 1], e)
    y = torch.zeros(tokens, hidden, device=DEV).index_add_(0, token.long(), part.float() * top.softmax(1).flatten()[order][:, None])
    assert torch.isfinite(y).all()
