"""Host checks of the rules by which the layer norm and its gradient share rows (csrc/layer_norm_shape.hpp,
compiled here by itself): every row's vectors have a lane, launches stay within their limits, and the
sizes that the GPU tests run take every form of the gradient.  Runs without a GPU."""
import ctypes
import os
import subprocess

import pytest

from tests.layer_norm_shapes import SIZES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "layer_norm_shape.hpp"
using namespace sffn;
// lanes, waves, vectors a lane, rows a workgroup, whether the row groups sum columns, workgroups of rows
extern "C" void form(int64_t rows, int32_t d, int64_t* out) {
  const ln_grad::GradShape g = ln_grad::grad_shape(d);
  const int64_t v[] = {g.row.lanes, g.row.waves, g.row.nv, g.rows, ln_grad::sums_in_rows(rows, d),
                       ln_grad::row_groups(rows, d)};
  for (int i = 0; i < 6; ++i) out[i] = v[i];
}
// Lengths whose vectors have no lane, or whose workgroups do not fit what the kernels assume.
extern "C" int wrong() {
  int bad = 0;
  const int64_t counts[] = {1, 2, 37, 1024, 1025, 100000, 1 << 30};
  for (int32_t d = 1; d <= 32768; ++d) {
    for (int wide = 0; wide < 2; ++wide) {
      const RowShape r = row_shape(d, wide);
      const int lanes = r.lanes > 0 ? r.lanes : 64 * r.waves;
      bad += r.nv < 1 || r.nv > 4 || lanes * r.nv * 8 < d || r.waves > 16 || (r.lanes > 0 && r.nv > 1);
      bad += r.lanes > 0 && rows_of(r.lanes) * r.lanes != 64 * r.waves;
    }
    const ln_grad::GradShape g = ln_grad::grad_shape(d);
    const int lanes = g.row.lanes > 0 ? g.row.lanes : 64 * g.row.waves;
    bad += lanes * g.row.nv * 8 < d || g.threads() > 1024 || g.threads() % 64 != 0 || g.threads() != g.rows * lanes;
    bad += g.threads() < 32 || (g.row.nv > 1 && (g.row.lanes != 1024 || g.rows != 1));
    for (int64_t rows : counts) {
      const int64_t n = ln_grad::row_groups(rows, d), parts = ln_grad::sum_parts(rows, d);
      const bool sums = ln_grad::sums_in_rows(rows, d);
      bad += n < 1 || n > (sums ? 256 : 1 << 20) || (sums && (d > 16384 || g.row.nv > 2));
      bad += parts < 1 || parts > 64 || (ln_grad::few_rows(rows, d) && parts != 1);
    }
  }
  return bad;
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("layer_norm_shape")
    (d / "rule.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "activation_sparse_transformer_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + csrc,
                    str(d / "rule.cpp"), "-o", str(d / "rule.so")], check=True)
    return ctypes.CDLL(str(d / "rule.so"))


def _form(rule, rows, d):
    """(lanes, waves, vectors a lane, columns summed in registers), rows of a workgroup, workgroups"""
    v = (ctypes.c_int64 * 6)()
    rule.form(ctypes.c_int64(rows), ctypes.c_int32(d), v)
    return (v[0], v[1], v[2], bool(v[4])), v[3], v[5]


def test_every_length_fits(rule):
    assert rule.wrong() == 0


def test_every_form_of_the_gradient_is_tested(rule):
    forms = {_form(rule, rows, d)[0] for rows in (1, 5000) for d in range(1, 32769)}
    assert {_form(rule, rows, d)[0] for many, few, d in SIZES for rows in (many, few)} == forms


def test_many_rows_take_several_turns(rule):
    """The many rows of a size are more than the workgroups take at once, and leave some without a row in the
    last turn or end inside a workgroup's rows; the few are summed in the same launch."""
    for many, few, d in SIZES:
        (_, _, _, sums), rpb, groups = _form(rule, many, d)
        assert sums == (d <= 16384)
        if sums:
            assert many > groups * rpb and many % (groups * rpb) != 0
        assert not _form(rule, few, d)[0][3]
    assert sum(d % 8 == 0 for _, _, d in SIZES) == 3
