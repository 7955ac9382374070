"""Host-side checks of the 8-bit (W8A8) calls: argument errors are rejected
before any CUDA call (made-up addresses, no GPU touched), the Python wrappers
refuse tensors that do not fit, and the plain forms the GPU tests compare with
agree with the 64-bit mathematics."""
import ctypes as C
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import int8_ref as ref
from vector_quantization_codec_b200 import qamw

FAKE = 0x7F0000000000  # a 16-byte aligned address that is never dereferenced
L = qamw.lib()
BF16, F32 = qamw.QAMW_DTYPE_BF16, qamw.QAMW_DTYPE_F32
INVALID, SHAPE, ALIGN, OK = (qamw.QAMW_ERR_INVALID, qamw.QAMW_ERR_SHAPE, qamw.QAMW_ERR_ALIGN,
                             qamw.QAMW_OK)


def _encode(fn, x=FAKE, dtype=BF16, rows=4, d=128, s=FAKE, q=FAKE, scale=FAKE):
    return getattr(L, fn)(x, dtype, rows, d, s, q, scale, None, None)


@pytest.mark.parametrize("fn", ["qamw_int8_encode_weights", "qamw_int8_encode_tokens"])
@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
    (dict(rows=-1), SHAPE), (dict(d=0), SHAPE), (dict(d=100), SHAPE), (dict(d=-64), SHAPE),
    (dict(d=32768 + 64), SHAPE),
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID),
    (dict(x=FAKE + 8), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(scale=FAKE + 2), ALIGN),
    (dict(s=FAKE + 8), ALIGN),
    (dict(rows=0, x=None, q=None, scale=None, s=None), OK),  # nothing to do
])
def test_encode_argument_errors(fn, kw, rc):
    assert _encode(fn, **kw) == rc


def _norm(x=FAKE, res=FAKE, dtype=BF16, gain=FAKE, eps=1e-5, rows=4, d=128, s=FAKE, out=FAKE,
          q=FAKE, scale=FAKE):
    return L.qamw_rmsnorm_int8(x, res, dtype, gain, eps, rows, d, s, out, q, scale, None, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=7), INVALID), (dict(rows=-3), SHAPE), (dict(d=96), SHAPE), (dict(d=65536), SHAPE),
    (dict(eps=0.0), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(eps=1e-39), INVALID),
    (dict(x=None), INVALID), (dict(gain=None), INVALID), (dict(q=None), INVALID),
    (dict(scale=None), INVALID),
    (dict(res=None), INVALID), (dict(out=None), INVALID),  # one without the other
    (dict(x=FAKE + 4), ALIGN), (dict(res=FAKE + 2), ALIGN), (dict(gain=FAKE + 2), ALIGN),
    (dict(out=FAKE + 8), ALIGN), (dict(q=FAKE + 4), ALIGN), (dict(s=FAKE + 2), ALIGN),
    (dict(scale=FAKE + 1), ALIGN),
    (dict(rows=0, x=None, res=None, out=None, gain=None, q=None, scale=None), OK),
])
def test_norm_argument_errors(kw, rc):
    assert _norm(**kw) == rc


def _gemm(x=FAKE, xs=FAKE, ntok=4, w=FAKE, ws=FAKE, d_out=8, d_in=128, y=FAKE, dtype=BF16):
    return L.qamw_int8_gemm(x, xs, ntok, w, ws, d_out, d_in, y, dtype, None, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=2), INVALID), (dict(ntok=-1), INVALID), (dict(ntok=65537), INVALID),
    (dict(d_out=-1), SHAPE), (dict(d_in=0), SHAPE), (dict(d_in=32), SHAPE), (dict(d_in=100), SHAPE),
    (dict(d_in=32768 + 64), SHAPE),
    (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(w=None), INVALID),
    (dict(ws=None), INVALID), (dict(y=None), INVALID),
    (dict(x=FAKE + 8), ALIGN), (dict(w=FAKE + 4), ALIGN), (dict(xs=FAKE + 2), ALIGN),
    (dict(ws=FAKE + 1), ALIGN), (dict(y=FAKE + 1), ALIGN), (dict(y=FAKE + 2, dtype=F32), ALIGN),
    (dict(ntok=0, x=None, xs=None, y=None), OK), (dict(d_out=0, w=None, ws=None, y=None), OK),
])
def test_gemm_argument_errors(kw, rc):
    assert _gemm(**kw) == rc


def test_wrappers_refuse_tensors_that_are_not_on_a_gpu():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for fn in (qamw.qamw_int8_encode_tokens, qamw.qamw_int8_encode_weights):
        with pytest.raises(ValueError):
            fn(x)
    with pytest.raises(ValueError):
        qamw.qamw_rmsnorm_int8(x, torch.ones(64, dtype=torch.bfloat16))
    q = torch.zeros((2, 64), dtype=torch.int8)
    with pytest.raises(ValueError):
        qamw.qamw_int8_gemm(q, torch.ones(2), q, torch.ones(2))


@pytest.mark.parametrize("kind", ["weights", "tokens", "norm"])
def test_stated_fp32_steps_follow_the_mathematics(kind):
    """rows32 against rows64: at most two roundings in v and in a, one in 127 / a and one in the
    product, so 127 v / a is off by at most 127 * 6 * 2^-24 < 5e-5 and q by 0.5 + 5e-5."""
    g = np.random.default_rng(5)
    h = (g.standard_normal((9, 320)) * g.lognormal(0, 2, (1, 320))).astype(np.float32)
    h[3] = 0
    h[4] *= np.float32(1e-20)
    s = g.lognormal(0, 0.5, 320).astype(np.float16)
    gain = (1 + 0.2 * g.standard_normal(320)).astype(np.float32) if kind == "norm" else None
    q, scale, _ = ref.rows32(h, ref.factors32(320, s, gain, divide=kind != "weights"))
    u, scale64 = ref.rows64(h, s, gain, divide=kind != "weights")
    assert np.abs(q - u).max() <= 0.5 + 5e-5
    assert (np.abs(scale - scale64) <= 3 * ref.U32 * scale64 * (1 + 1e-6)).all()
    assert (np.abs(q).max(axis=1) == np.where(scale > 0, 127, 0)).all()


def test_gemm_c_types_take_null():
    assert L.qamw_int8_gemm(None, None, 0, None, None, 0, 64, None, F32, None, None) == OK
    assert isinstance(L, C.CDLL)


@pytest.mark.parametrize("tries,st,eps,rc", [(0, None, 1e-5, INVALID), ((1 << 18) + 1, FAKE, 1e-5, INVALID),
                                             (0, FAKE, 0.0, INVALID)])
def test_giving_up_check_argument_errors(tries, st, eps, rc):
    assert L.qamw_selftest_rmsnorm_int8(tries, FAKE, FAKE, BF16, FAKE, eps, 4, 128, None, FAKE, FAKE, FAKE,
                                        st, None) == rc


@pytest.mark.parametrize("shape", [(65536, 1 << 30, 32768), (65536, 1 << 30, 64), (1, 1 << 30, 64),
                                   (65536, 1, 32768), (12000, 1 << 30, 32768)], ids=str)
def test_products_of_the_largest_sizes_get_a_plan(shape):
    """The largest sizes that the call allows are planned (and then fail to launch: the child sees no
    GPU), whatever their estimated time."""
    ntok, d_out, d_in = shape
    code = ("from vector_quantization_codec_b200 import qamw\n"
            f"rc = qamw.lib().qamw_int8_gemm({FAKE}, {FAKE}, {ntok}, {FAKE}, {FAKE}, {d_out}, {d_in}, {FAKE}, "
            f"{BF16}, None, None)\nassert rc == {qamw.QAMW_ERR_CUDA}, rc\n")
    r = subprocess.run([sys.executable, "-c", code], env={**os.environ, "CUDA_VISIBLE_DEVICES": ""},
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)


CACHE_MAIN = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "launch_cache.h"
using namespace qamw;
int main() {
  static LaunchCache cache;
  static char kernels[8];
  // every width of every kernel, as several threads meet them in different orders
  const auto key = [](int i) {
    return LaunchKey{i % 2, &kernels[i % 8], 32 * (1 + i % 32), (size_t)(64 * (i / 8))};
  };
  const int n = 4096;
  std::vector<std::thread> threads;
  for (int t = 0; t < 4; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < n; ++i) {
        const int j = (i * 7 + t * 1000) % n;
        int v;
        if (!cache.get(key(j), &v)) cache.put(key(j), j);
      }
    });
  for (auto& t : threads) t.join();
  for (int i = 0; i < n; ++i) {
    int v = -1;
    if (!cache.get(key(i), &v) || v != i) return printf("key %d: %d\n", i, v), 1;
  }
  int v;
  return cache.get(LaunchKey{2, kernels, 32, 0}, &v) ? 2 : 0;
}
"""


def test_launch_facts_of_every_width_are_kept(tmp_path):
    """What a call looks up once per kernel and width stays looked up, however many there are."""
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(CACHE_MAIN)
    csrc = os.path.join(os.path.dirname(os.path.abspath(qamw.__file__)), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", csrc, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout)


def test_a_refused_stream_leaves_the_device_as_it_was(monkeypatch):
    """The wrappers make the tensors' device current before they look at the stream: an argument that
    is no stream must not leave it so."""
    entered = []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)

        def __exit__(self, *exc):
            entered.pop()

    monkeypatch.setattr(qamw.torch.cuda, "device", Device)
    for stream in ("no stream", object(), [1]):
        with pytest.raises((TypeError, ValueError)):
            qamw._enter(3, stream)
        assert not entered


def test_giving_up_checks_refuse_tensors_that_are_not_on_a_gpu():
    x, q, one = torch.zeros((2, 64)), torch.zeros((2, 64), dtype=torch.int8), torch.ones(2)
    st = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        qamw.qamw_selftest_rmsnorm_int8(0, x, x[0], None, q, one, st)
    with pytest.raises(ValueError):
        qamw.qamw_selftest_int8_gemm(q, one, q, one, torch.zeros((2, 2)), st)


def test_giving_up_check_of_the_product_argument_errors():
    S = L.qamw_selftest_int8_gemm
    assert S(FAKE, FAKE, 4, FAKE, FAKE, 8, 128, FAKE, BF16, None, None) == INVALID
    assert S(FAKE, FAKE, 4, FAKE, FAKE, 8, 100, FAKE, BF16, FAKE, None) == SHAPE
    assert S(FAKE + 8, FAKE, 4, FAKE, FAKE, 8, 128, FAKE, BF16, FAKE, None) == ALIGN
