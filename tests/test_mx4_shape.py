"""Host checks of the rule that selects a 4-bit product's kernel form (csrc/mx4_shape.hpp, compiled
here by itself): every selected form is built, every built form is selected by a size that the GPU
tests run, and by no other size than the rule says.  Runs without a GPU."""
import ctypes
import os
import subprocess

import pytest

from tests.mx4_forms import FORMS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"f32": 0, "bf16": 1, "fp8": 2}

SOURCE = r"""
#include "mx4_shape.hpp"
using namespace sffn;
extern "C" void shape(int x, int64_t nb, int64_t kb, int64_t T, int* o) {
  const Mx4Shape s = mx4_shape(x, nb, kb, T);
  o[0] = s.tt, o[1] = s.rb, o[2] = s.ks;
}
extern "C" int built(int x, int tt, int rb, int ks) { return mx4_built(x, tt, rb, ks); }
// The number of sizes whose form is not built: row blocks one by one, then in small steps up to the
// most that a call takes; the same for blocks of columns.
extern "C" int64_t unbuilt(int64_t* seen) {
  int64_t bad = 0;
  const int64_t tokens[] = {1, 16, 17, 32, 33, 48, 49, 64, 65, 96, 97, 113, 128, 129, 200, 513, 1025, 32768, 1 << 20};
  for (int64_t T : tokens)
    for (int64_t nb = 1; nb <= 1 << 22; nb += nb < 7000 ? 1 : nb / 100)
      for (int64_t kb = 1; kb <= 1 << 23 && nb * kb < 1 << 25; kb += kb < 70 ? 1 : kb / 10)
        for (int x = 0; x < 3; ++x) {
          const Mx4Shape s = mx4_shape(x, nb, kb, T);
          bad += !mx4_built(x, s.tt, s.rb, s.ks);
          ++seen[x];
        }
  return bad;
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx4_shape")
    (d / "rule.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "activation_sparse_transformer_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + csrc,
                    str(d / "rule.cpp"), "-o", str(d / "rule.so")], check=True)
    L = ctypes.CDLL(str(d / "rule.so"))
    L.shape.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int)]
    L.unbuilt.restype = ctypes.c_int64
    return L


def test_tested_sizes_select_their_forms(rule):
    o = (ctypes.c_int * 3)()
    for kind, T, N, K, form in FORMS:
        rule.shape(TYPES[kind], -(-N // 16), -(-K // 128), T, o)
        assert tuple(o) == form, (kind, T, N, K)
        assert N % 16 and K % 128 and T % 16


def test_every_built_form_is_tested(rule):
    built = {(kind, tt, rb, ks) for kind, x in TYPES.items() for tt in range(1, 5) for rb in range(1, 5)
             for ks in (2, 4, 8) if rule.built(x, tt, rb, ks)}
    assert built == {(kind, *form) for kind, _, _, _, form in FORMS}
    assert len(built) == len(FORMS)


def test_every_selected_form_is_built(rule):
    seen = (ctypes.c_int64 * 3)()
    assert rule.unbuilt(seen) == 0
    assert min(seen) > 10 ** 7
