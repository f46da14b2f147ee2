"""Host checks of the rule that selects the kernel form of a product of 4-bit tokens
(csrc/mx4_matmul_form.hpp, compiled here by itself): the sizes that the GPU tests run select their
forms, every form is among them, and every size that a call takes selects one.  Runs without a GPU."""
import ctypes
import os
import subprocess

import pytest

from tests.mx4_matmul_forms import FORMS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "mx4_matmul_form.hpp"
using namespace sffn;
extern "C" int form(int64_t nb, int64_t kb, int64_t T, int rounding, int y_f32) {
  return mx4_matmul_form(nb, kb, T, rounding, y_f32);
}
extern "C" int forms() { return MX4_FORMS; }
// Sizes whose form is none of those for their number of tokens: row blocks one by one, then in small
// steps up to the most that a call takes; the same for blocks of columns.
extern "C" int64_t wrong(int64_t* seen) {
  int64_t bad = 0;
  const int64_t tokens[] = {1, 15, 16, 17, 32, 33, 64, 65, 128, 129, 513, 4096, 32768, 1 << 20};
  for (int64_t T : tokens)
    for (int64_t nb = 1; nb <= 1 << 22; nb += nb < 5000 ? 1 : nb / 100)
      for (int64_t kb = 1; kb <= 1 << 21 && nb * kb < 1 << 25; kb += kb < 70 ? 1 : kb / 10) {
        const int f = mx4_matmul_form(nb, kb, T, false, T & nb & 1), r = mx4_matmul_form(nb, kb, T, true, nb & 1);
        if (T <= 16) bad += f > MX4_FEW_16x2 || r > MX4_FEW_16x4;
        else if (T <= 32) bad += f != MX4_FEW_32x1 && f != MX4_FEW_32x2;
        else bad += f < MX4_FEW_32x2 || f >= MX4_FORMS || (f == MX4_FEW_32x2 && T > 64);
        ++*seen;
      }
  return bad;
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx4_matmul_form")
    (d / "rule.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "activation_sparse_transformer_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + csrc,
                    str(d / "rule.cpp"), "-o", str(d / "rule.so")], check=True)
    L = ctypes.CDLL(str(d / "rule.so"))
    L.form.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2
    L.wrong.restype = ctypes.c_int64
    return L


def test_tested_sizes_select_their_forms(rule):
    for y_f32 in (0, 1):  # the same form for both types of results
        got = [(r, T, N, K, rule.form(-(-N // 16), -(-K // 128), T, r, y_f32)) for r, T, N, K, _ in FORMS]
        assert got == FORMS
    assert all(N % 16 and K % 128 and T % 16 for _, T, N, K, _ in FORMS)


def test_every_form_is_tested(rule):
    assert {f for _, _, _, _, f in FORMS} == set(range(rule.forms()))
    assert {f for r, _, _, _, f in FORMS if r} == {0, 1, 2}


def test_every_size_selects_a_form(rule):
    seen = ctypes.c_int64()
    assert rule.wrong(ctypes.byref(seen)) == 0 and seen.value > 10 ** 6
