"""The 8-bit operators without a GPU: the oracle's format, refusals of the C entries and of the binding."""
import numpy as np
import pytest
import torch

from nano_intra_device_gb300 import _lib
from oracle import fp8 as orc

P16 = 1 << 20  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def _refused(code):
    assert code == _lib.NF_ERR_INVALID_ARG
    return _lib.lib().nf_last_error().decode()


# ------------------------------------------------------------------ the oracle

def test_code_values_are_torchs():
    """Every e4m3 value stays, its neighbours' midpoints go to the even code, and random values go where torch's conversion takes them."""
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(orc.code_values(every), every)
    mid = (every[1:] + every[:-1]) / 2
    r = np.random.default_rng(0).standard_normal(20000) * 10.0 ** np.random.default_rng(1).uniform(-4, 2, 20000)
    for x in (mid, -mid, np.clip(r, -448, 448)):
        x = x.astype(np.float32)
        assert np.array_equal(orc.code_values(x.astype(np.float64)), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())
    assert np.isnan(orc.code_values(np.array([np.nan]))).all() and orc.code_values(np.array([1e9]))[0] == 448


def test_blocks_of_representable_values_are_exact():
    r = np.random.default_rng(2)
    y = orc.E4M3[r.integers(0, 127, (5, 300))].astype(np.float32) * np.float32(2.0 ** -5)
    y[:, ::128] = 448 * 2.0 ** -5
    q, s = orc.quantise_rows(y)
    assert s.shape == (3, 5) and (s == 2.0 ** -5).all() and np.array_equal(orc.rows_of(q, s), y)
    w, ws = orc.quantise_weights(y)
    assert ws.shape == (1, 3) and np.array_equal(orc.weights_of(w, ws), y)


def test_special_blocks():
    y = np.zeros((4, 130), np.float32)
    y[1, 3], y[2, 129], y[3, 5] = np.nan, np.inf, 1e-44
    q, s = orc.quantise_rows(y)
    assert s[0, 0] == orc.TINY and (q[0] == 0).all()
    assert np.isnan(s[0, 1]) and np.isnan(q[1, :128]).all() and (q[1, 128:] == 0).all()
    assert np.isnan(s[1, 2]) and not np.isnan(q[2, :128]).any()
    assert s[0, 3] == orc.TINY and (q[3] == 0).all()


def test_quantised_values_are_within_half_a_step():
    """Codes are off by half a step (2^-4 of a value, 2^-10 of the scale near zero), beside the quotient's rounding to fp32."""
    y = (np.random.default_rng(3).standard_normal((7, 400)) * 3).astype(np.float32)
    q, s = orc.quantise_rows(y)
    u = y.astype(np.float64) / np.repeat(s.T, 128, 1)[:, :400]
    assert (np.abs(q - u) <= np.maximum(2.0 ** -4 * np.abs(u), 2.0 ** -10) * (1 + 2.0 ** -20)).all()
    assert np.abs(q).max() == 448


def test_norm_of_the_oracle():
    x = np.array([[3.0, -4.0]])
    h, y = orc.norm(x, None, np.array([2.0, 1.0]), 0.0)
    assert np.allclose(y, [[2 * 3 / np.sqrt(12.5), -4 / np.sqrt(12.5)]]) and h is x
    h, y2 = orc.norm(x / 2, x / 2, np.array([2.0, 1.0]), 0.0)
    assert np.array_equal(h, x) and np.allclose(y, y2)
    assert orc.swiglu(np.array([0.0, -1e4]), np.array([5.0, 1.0])).tolist() == [0.0, 0.0]


# ------------------------------------------------------------------ refusals

def test_norm_refusals(L):
    def call(**kw):
        a = dict(x=P16, r=P16, g=P16, h=P16, q=P16, s=P16, rows=3, n=256, eps=1e-5) | kw
        return L.nf_rmsnorm_fp8(a["x"], a["r"], a["g"], a["h"], a["q"], a["s"], a["rows"], a["n"], a["eps"], None)
    for k in ("x", "g", "q", "s"):
        assert "NULL" in _refused(call(**{k: None}))
    for bad in (dict(rows=-1), dict(n=0), dict(n=-16), dict(n=8), dict(n=250), dict(n=32784), dict(eps=-1.0), dict(eps=float("nan")),
                dict(x=P16 + 8), dict(r=P16 + 2), dict(g=P16 + 4), dict(h=P16 + 8), dict(q=P16 + 8), dict(s=P16 + 2), dict(r=None)):
        _refused(call(**bad))
    assert call(rows=0, x=None) == _lib.NF_OK


def test_quant_refusals(L):
    def call(**kw):
        a = dict(x=P16, src=3, index=None, q=P16, s=P16, rows=3, n=256) | kw
        return L.nf_quant_fp8(a["x"], a["src"], a["index"], a["q"], a["s"], a["rows"], a["n"], None)
    for k in ("x", "q", "s"):
        assert "NULL" in _refused(call(**{k: None}))
    for bad in (dict(rows=-1), dict(src=-1, index=P16), dict(src=4), dict(n=0), dict(n=24), dict(n=40000), dict(x=P16 + 2), dict(q=P16 + 4),
                dict(index=P16 + 2), dict(s=P16 + 1)):
        _refused(call(**bad))
    assert call(rows=0, src=0) == _lib.NF_OK and call(rows=0, src=7, index=P16) == _lib.NF_OK


def test_weights_refusals(L):
    def call(**kw):
        a = dict(w=P16, q=P16, s=P16, mats=2, rows=200, n=256) | kw
        return L.nf_quant_fp8_weights(a["w"], a["q"], a["s"], a["mats"], a["rows"], a["n"], None)
    for k in ("w", "q", "s"):
        assert "NULL" in _refused(call(**{k: None}))
    for bad in (dict(mats=-1), dict(rows=0), dict(n=0), dict(n=24), dict(w=P16 + 8), dict(q=P16 + 8), dict(s=P16 + 2),
                dict(mats=1 << 30, rows=1 << 20, n=1 << 20)):
        _refused(call(**bad))
    assert call(mats=0) == _lib.NF_OK


@pytest.mark.parametrize("grouped", [False, True])
def test_gemm_refusals(L, grouped):
    def call(**kw):
        a = dict(a=P16, a_s=P16, b=P16, b_s=P16, off=P16, groups=4, c=P16, c_s=P16, r=P16, m=3, n=256, k=256, epi=0, sms=0) | kw
        if grouped:
            return L.nf_gemm_fp8_grouped(a["a"], a["a_s"], a["b"], a["b_s"], a["off"], a["groups"], a["c"], a["c_s"], a["m"], a["n"], a["k"],
                                         a["epi"], a["sms"], None)
        return L.nf_gemm_fp8(a["a"], a["a_s"], a["b"], a["b_s"], a["c"], a["c_s"], a["r"], a["m"], a["n"], a["k"], a["epi"], a["sms"], None)
    for k in ("a", "a_s", "b", "b_s", "c"):
        assert "NULL" in _refused(call(**{k: None}))
    assert "NULL" in _refused(call(c_s=None, epi=_lib.NF_EPI_SWIGLU_FP8))
    for bad in (dict(m=-1), dict(n=0), dict(n=4), dict(n=252), dict(k=0), dict(k=8), dict(k=250), dict(epi=-1), dict(epi=4), dict(sms=-1),
                dict(n=264, epi=_lib.NF_EPI_SWIGLU_FP8), dict(a=P16 + 8), dict(b=P16 + 8), dict(c=P16 + 8), dict(a_s=P16 + 2), dict(b_s=P16 + 2),
                dict(m=0x7fffffff), dict(n=0x7ffffff8), dict(k=0x7ffffff0)):
        _refused(call(**bad))
    if grouped:
        assert "NULL" in _refused(call(off=None))
        for bad in (dict(groups=0), dict(groups=129), dict(epi=_lib.NF_EPI_RESID), dict(off=P16 + 2)):
            _refused(call(**bad))
    else:
        assert "NULL" in _refused(call(r=None, epi=_lib.NF_EPI_RESID))
        _refused(call(r=P16 + 8, epi=_lib.NF_EPI_RESID))
    assert call(m=0) == _lib.NF_OK


def test_timeout_refusals(L):
    for bad in (0, -1, 10 ** 10 + 1):
        assert "timeout_ns" in _refused(L.nf_fp8_set_timeout(bad))
    assert L.nf_fp8_set_timeout(2 * 10 ** 9) == _lib.NF_OK


def test_the_bf16_product_refuses_the_8_bit_epilogue(L):
    _refused(L.nf_gemm(P16, P16, P16, None, 8, 16, 16, _lib.NF_EPI_SWIGLU_FP8, 0, None))


# ------------------------------------------------------------------ the binding

E, F, H, I = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32


def z(*n, t=H):
    return torch.zeros(n, dtype=t)


CALLS = {
    "norm": (_lib.rmsnorm_fp8, dict(x=z(3, 272), g=z(272), q=z(3, 272, t=E), s=z(3, 3, t=F), eps=1e-5, r=z(3, 272), h=z(3, 272))),
    "quant": (_lib.quant_fp8, dict(x=z(3, 272), q=z(5, 272, t=E), s=z(3, 5, t=F), index=z(5, t=I))),
    "weights": (_lib.quant_fp8_weights, dict(w=z(2, 130, 272), q=z(2, 130, 272, t=E), s=z(2, 2, 3, t=F))),
    "gemm": (_lib.gemm_fp8, dict(a=z(3, 272, t=E), a_s=z(3, 3, t=F), b=z(136, 272, t=E), b_s=z(2, 3, t=F), c=z(3, 136), r=z(3, 136), epilogue=_lib.NF_EPI_RESID)),
    "swiglu8": (_lib.gemm_fp8, dict(a=z(3, 272, t=E), a_s=z(3, 3, t=F), b=z(288, 272, t=E), b_s=z(2, 2, 3, t=F), c=z(3, 144, t=E), c_s=z(2, 3, t=F),
                                    epilogue=_lib.NF_EPI_SWIGLU_FP8)),
    "grouped": (_lib.gemm_fp8_grouped, dict(a=z(3, 272, t=E), a_s=z(3, 3, t=F), b=z(4, 136, 272, t=E), b_s=z(4, 2, 3, t=F), group_off=z(5, t=I), c=z(3, 136))),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_binding_refuses_other_types_sizes_and_strides(name):
    call, good = CALLS[name]
    with pytest.raises(ValueError, match="CUDA device"):  # right, but for where they are
        call(**good)
    for k, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)
        for bad in (t.double() if t.dtype == F else t.float(), wide, wide[..., ::2]):
            with pytest.raises(ValueError):
                call(**(good | {k: bad}))


def test_binding_wants_the_scales_of_an_8_bit_output():
    call, good = CALLS["swiglu8"]
    with pytest.raises(ValueError, match="c_s"):
        call(**(good | dict(c_s=None)))


def _other_way_round(t):
    """Contiguous, with as many elements, rows and columns of the last two dimensions exchanged."""
    return t.view(t.shape[:-2] + (t.shape[-1], t.shape[-2]))


@pytest.mark.parametrize("name,k", [(n, k) for n, (_, good) in CALLS.items() for k, t in good.items() if isinstance(t, torch.Tensor) and t.dim() > 1])
def test_binding_refuses_the_other_way_round(name, k):
    """Scales [rows, blocks], weights [K, N] and the like have the right count and would give wrong results."""
    call, good = CALLS[name]
    big = dict(good)
    if name in ("gemm", "swiglu8", "grouped"):  # (three rows and three blocks of K would be the same either way)
        big |= dict(a=z(4, 272, t=E), a_s=z(3, 4, t=F), c=z(4, good["c"].shape[1], t=good["c"].dtype))
        big |= dict(r=z(4, 136)) if name == "gemm" else dict(c_s=z(2, 4, t=F)) if name == "swiglu8" else {}
    if name == "norm":
        big |= {n: z(4, 272, t=good[n].dtype) for n in ("x", "q", "r", "h")} | dict(s=z(3, 4, t=F))
    with pytest.raises(ValueError, match="CUDA device"):
        call(**big)
    with pytest.raises(ValueError) as e:
        call(**(big | {k: _other_way_round(big[k])}))
    assert "CUDA device" not in str(e.value)


def test_binding_takes_every_naming_of_the_same_rows():
    """One row's scales in either order and matrices stacked as one are the same memory."""
    call, good = CALLS["swiglu8"]
    one = good | dict(a=z(1, 272, t=E), a_s=z(1, 3, t=F), c=z(1, 144, t=E), c_s=z(2, t=F))
    for more in ({}, dict(b=z(2, 144, 272, t=E)), dict(b_s=z(4, 3, t=F))):
        with pytest.raises(ValueError, match="CUDA device"):
            call(**(one | more))


# ------------------------------------------------------------------ host code

def run_host_code(tmp_path, code):
    """Compile a program against csrc/ with the host compiler and return what it prints."""
    import os
    import subprocess
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(code)
    csrc = os.path.join(os.path.dirname(_lib.__file__), "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60).stdout


def test_answers_are_kept_by_device_and_failures_are_not(tmp_path):
    out = run_host_code(tmp_path, """
#include "by_device.h"
#include <cstdio>
int asked = 0;
int main() {
  static nf::ByDevice<9> kept;
  auto get = [](int dev, int which, int says, int code) {
    int n = -1;
    const int e = kept.get(dev, which, &n, [&](int* a) { ++asked; *a = says; return code; });
    std::printf("%d:%d:%d ", e, e ? -1 : n, asked);
  };
  get(0, 2, 36, 0), get(0, 2, 99, 0);  // asked once
  get(1, 2, 33, 0), get(0, 2, 99, 0), get(1, 2, 99, 0);  // another device has its own
  get(0, 4, 18, 700), get(0, 4, 17, 0), get(0, 4, 99, 0);  // a failure is told and not kept
  get(0, 8, 0, 0), get(0, 8, 99, 0);  // none fits: an answer too
  get(64, 2, 5, 0), get(64, 2, 6, 0);  // a device beyond those counted is asked every time
}
""")
    assert out.split() == ["0:36:1", "0:36:1", "0:33:2", "0:36:2", "0:33:2", "700:-1:3", "0:17:4", "0:17:4", "0:0:5", "0:0:5", "0:5:6", "0:6:7"]


def test_no_kernel_keeps_occupancy_by_process():
    """Each query of a device's occupancy goes through the answers kept by device."""
    import glob
    import os
    for path in glob.glob(os.path.join(os.path.dirname(_lib.__file__), "csrc", "*.cu")):
        text = open(path).read()
        assert text.count("cudaOccupancyMaxActiveClusters(") == text.count("kept.get("), path


# (M, N, K, groups, SwiGLU) and the us measured by the kernel of few rows and by tiles, on 152 SMs
MEASURED = [
    (64, 8192, 4096, 1, 0, 10.8, 15.6), (128, 8192, 4096, 1, 0, 13.2, 15.8), (128, 2048, 4096, 1, 1, 11.3, 12.7), (64, 4096, 4096, 1, 1, 12.0, 14.5),
    (128, 4096, 4096, 1, 1, 15.4, 14.6), (64, 14336, 4096, 1, 0, 14.8, 16.9), (128, 14336, 4096, 1, 0, 19.5, 17.4), (16, 28672, 4096, 1, 0, 23.2, 30.5),
    (32, 28672, 4096, 1, 0, 23.5, 23.4), (64, 28672, 4096, 1, 0, 25.1, 23.8), (16, 128256, 4096, 1, 0, 89, 96), (32, 128256, 4096, 1, 0, 97, 89),
    (512, 1024, 4096, 8, 0, 13.5, 19.0), (256, 512, 4096, 8, 1, 12.5, 19.4), (512, 512, 4096, 8, 1, 21.9, 19.5), (256, 2048, 4096, 8, 0, 16.4, 20.0),
    (64, 14336, 4096, 8, 1, 139, 140), (256, 14336, 4096, 8, 1, 165, 142), (512, 2048, 2048, 64, 0, 58, 48), (128, 768, 2048, 64, 0, 25.5, 24.0),
    (64, 2048, 1024, 64, 0, 28.1, 21.9), (32, 2048, 1024, 64, 0, 18.4, 16.2), (128, 1024, 1024, 128, 0, 30.4, 23.0), (16, 8192, 1024, 16, 0, 24.9, 21.1),
    (64, 2048, 2048, 64, 0, 40.3, 36.8), (63, 2048, 2048, 64, 0, 41.1, 37.9), (48, 2048, 2048, 64, 0, 32.8, 33.9), (32, 2048, 2048, 64, 0, 26.9, 26.6),
    (64, 768, 2048, 64, 0, 15.8, 16.1), (48, 768, 2048, 64, 0, 13.9, 17.6), (64, 512, 2048, 128, 0, 14.4, 15.8), (8, 8192, 2048, 8, 0, 15.6, 17.9),
    (64, 1024, 4096, 64, 0, 41.4, 44.4), (64, 768, 2048, 64, 1, 25.5, 29.7), (16, 2048, 2048, 16, 1, 17.6, 26.8), (8, 8192, 4096, 8, 0, 25.0, 32.9),
]


def test_the_choice_of_kernel_agrees_with_what_was_measured(tmp_path):
    """At every size that the rule's comment gives, the side that it takes is the faster one, or within 6 % of it."""
    cases = ", ".join(f"{{{m}, {n}, {k}, {g}, {two}}}" for m, n, k, g, two, _, _ in MEASURED)
    out = run_host_code(tmp_path, """
#include "fp8_choice.h"
#include <cstdio>
int main() {
  const int cases[][5] = {%s};
  for (const auto& c : cases) std::printf("%%d ", nf::few_rows(c[0], c[1], c[2], c[3], c[4] != 0, 152));
  std::printf("%%d", nf::few_rows(0x7fffffff - 256, 0x7ffffff0, 16, 1, false, 152));
}
""" % cases)
    *few, large = [int(x) for x in out.split()]
    wrong = [(c, x) for c, x in zip(MEASURED, few) if (c[5] if x else c[6]) > 1.06 * min(c[5:])]
    assert not wrong and large == 0
