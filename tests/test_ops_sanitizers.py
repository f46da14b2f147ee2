"""Host-side AddressSanitizer build of the library under the argument checks of the operators
around the layer (CPU only)."""
import glob

import pytest

from tests.test_sanitizers import _child_pytest


def test_operators_host_code_under_asan(tmp_path):
    from activation_sparse_transformer_amd import build as hip_build
    rt = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    if not rt:
        pytest.skip("clang's AddressSanitizer runtime is not installed")
    lib = hip_build.build(out=str(tmp_path / "libsparse_ffn_asan.so"),
                          extra=("-Xarch_host", "-fsanitize=address",
                                 "-Xarch_host", "-fno-omit-frame-pointer", "-g"))
    _child_pytest({"LD_PRELOAD": rt[-1], "SFFN_LIB": lib}, ["tests/test_ops_abi.py"])
