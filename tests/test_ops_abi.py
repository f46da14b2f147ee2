"""Host-only checks of include/ffn_ops.h: every declared call is exported, wrapped and commented,
constants agree with the binding, and bad arguments are refused before anything reaches the GPU.
Runs without a GPU."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ffn_ops.h")
A = 0x1000  # stands for a device pointer; never followed
OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def ops():
    import activation_sparse_transformer_amd as sffn
    from activation_sparse_transformer_amd import ffn_ops
    if not os.path.exists(sffn.LIB_PATH):
        pytest.fail("libsparse_ffn.so is not built (run __graft_entry__.build())")
    return ffn_ops


def test_header_matches_library_and_binding(ops):
    text = open(HEADER).read()
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\bsffn_status_t\s+([a-z0-9_]+)\s*\(", code)))
    assert names == sorted(ops.exported_names())
    L = ctypes.CDLL(__import__("activation_sparse_transformer_amd").LIB_PATH)
    for n in names:
        assert hasattr(L, n), n
        assert re.search(r"\*/\s*sffn_status_t\s+" + n + r"\s*\(", text), n
    defs = dict(re.findall(r"#define\s+(SFFN_[A-Z0-9_]+)\s+([0-9]+)", code))
    assert defs == {"SFFN_E4M3": str(ops.SFFN_E4M3), "SFFN_NORM_MAX_D": str(ops.NORM_MAX_D),
                    "SFFN_MX4_GROUP": str(ops.MX4_GROUP), "SFFN_ADAMW_BLOCK": str(ops.ADAMW_BLOCK)}
    assert ctypes.sizeof(ops.AdamwTensorC) == 64 and ctypes.sizeof(ops.AdamwHyperC) == 48


NORM = dict(dtype=BF16, gain_dtype=BF16, x=A, x_stride=64, residual=A, residual_stride=64, gain=A,
            eps=1e-6, rows=0, d=64, y=A, stat=A, h=A)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), ({"dtype": 7}, INVALID), ({"dtype": E4M3}, INVALID), ({"gain_dtype": E4M3}, INVALID),
    ({"dtype": F32, "gain_dtype": BF16}, INVALID), ({"gain_dtype": F32}, OK),
    ({"d": 0}, INVALID), ({"d": -1}, INVALID), ({"d": 32769}, UNSUPPORTED), ({"rows": -1}, INVALID),
    ({"eps": -1e-6}, INVALID), ({"eps": float("nan")}, INVALID), ({"residual": None}, INVALID),
    ({"rows": 2, "x": None}, INVALID), ({"rows": 2, "x_stride": 63}, INVALID),
    ({"rows": 2, "residual_stride": 0}, INVALID), ({"rows": 2, "gain": None}, INVALID),
    ({"rows": 2, "y": None}, INVALID), ({"rows": 2, "x": A + 1}, INVALID),
    ({"rows": 2, "h": A + 1}, INVALID), ({"rows": 2, "stat": A + 2}, INVALID),
    ({"rows": 2, "gain": A + 1}, INVALID),
])
def test_norm_arguments(ops, kw, status):
    a = dict(NORM, **kw)
    for fn in ("sffn_rms_norm", "sffn_rms_norm_fp8"):
        assert getattr(ops._lib(), fn)(*a.values(), None) == status, fn


def test_norm_fp8_needs_scales(ops):
    a = dict(NORM, rows=2, stat=None)
    assert ops._lib().sffn_rms_norm_fp8(*a.values(), None) == INVALID


GRAD = dict(dtype=BF16, gain_dtype=F32, dy=A, dy_stride=64, h=A, h_stride=64, gain=A, rstd=A, dres=A,
            dres_stride=64, rows=5000, d=64, dx=A, dgain=A, ws=A, nb=1 << 30)


@pytest.mark.parametrize("kw,status", [
    ({"rows": 0, "dgain": None}, OK), ({"dtype": 5}, INVALID), ({"rows": -2}, INVALID),
    ({"d": 40000}, UNSUPPORTED), ({"dy": None}, INVALID), ({"h": None}, INVALID),
    ({"h_stride": 32}, INVALID), ({"dres_stride": 32}, INVALID), ({"rstd": None}, INVALID),
    ({"dx": None}, INVALID), ({"ws": None}, INVALID), ({"ws": A + 8}, INVALID), ({"nb": 16}, INVALID),
    ({"dx": A + 1}, INVALID), ({"dgain": A + 1}, INVALID),
])
def test_norm_backward_arguments(ops, kw, status):
    a = dict(GRAD, **kw)
    assert ops._lib().sffn_rms_norm_backward(*a.values(), None) == status


def test_norm_workspace(ops):
    f, n = ops._lib(), ctypes.c_size_t()
    for rows in (0, 1, 4, 1000, 100000, 1 << 30):
        assert f.sffn_rms_norm_backward_workspace(rows, 2048, ctypes.byref(n)) == OK
        assert n.value % (2048 * 4) == 0 and n.value <= 1024 * 2048 * 4
        assert (n.value == 0) == (rows <= 4)  # few rows are summed in the same launch
    assert f.sffn_rms_norm_backward_workspace(4, 2048, None) == INVALID


@pytest.mark.parametrize("kw,status", [
    ({"T": 0}, OK), ({"N": 0}, OK), ({"N": -1}, INVALID), ({"K": 0}, INVALID), ({"T": -1}, INVALID),
    ({"T": (1 << 20) + 1}, UNSUPPORTED), ({"N": 1 << 30, "K": 1 << 20}, UNSUPPORTED),
    ({"K": (1 << 30) + 1, "N": 1}, UNSUPPORTED), ({"N": (1 << 26) + 1, "K": 1}, UNSUPPORTED), ({"x_dtype": 3}, INVALID), ({"y_dtype": E4M3}, INVALID),
    ({"x_dtype": E4M3, "x_scale": None}, INVALID), ({"tiled": None}, INVALID), ({"tiled": A + 8}, INVALID),
    ({"x": None}, INVALID), ({"x_stride": 63}, INVALID), ({"y": None}, INVALID), ({"y": A + 1}, INVALID),
    ({"bias": A + 2}, INVALID), ({"x": A + 1}, INVALID),
])
def test_mx4_linear_arguments(ops, kw, status):
    a = dict(tiled=A, N=48, K=64, x_dtype=BF16, x=A, x_stride=64, x_scale=A, T=3, bias=A, relu=1,
             y_dtype=F32, y=A)
    a.update(kw)
    assert ops._lib().sffn_mx4_linear(*a.values(), None) == status


def test_mx4_weights_arguments(ops):
    f, n = ops._lib(), ctypes.c_size_t()
    assert f.sffn_mx4_bytes(33, 129, ctypes.byref(n)) == OK and n.value == 3 * 2 * 1088
    assert f.sffn_mx4_bytes(33, 129, None) == INVALID
    assert f.sffn_mx4_tile(None, A, 16, 32, A, None) == INVALID
    assert f.sffn_mx4_tile(A, A, 16, 32, A + 4, None) == INVALID
    assert f.sffn_mx4_tile(A, A, 0, 32, None, None) == OK
    assert f.sffn_mx4_quantize(E4M3, A, 32, 16, 32, A, A, None) == INVALID
    assert f.sffn_mx4_quantize(F32, A, 31, 16, 32, A, A, None) == INVALID
    assert f.sffn_mx4_quantize(F32, A, 32, 16, 32, A, None, None) == INVALID
    assert f.sffn_mx4_quantize(F32, None, 32, 16, 32, A, A, None) == INVALID
    assert f.sffn_mx4_quantize(F32, None, 32, 0, 32, None, None, None) == OK


TENSOR = dict(param=A, grad=A, master=None, m=A, v=A, m_scale=A, v_scale=A, n=300)
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)


@pytest.mark.parametrize("kw,hyper,types,status", [
    ({"n": 0}, {}, (F32, F32, 32), OK), ({"n": 0, "param": None, "m": None}, {}, (F32, F32, 8), OK),
    ({}, {}, (E4M3, F32, 32), INVALID), ({}, {}, (F32, E4M3, 32), INVALID), ({}, {}, (F32, F32, 16), INVALID),
    ({"n": -1}, {}, (F32, F32, 32), INVALID), ({"param": None}, {}, (F32, F32, 32), INVALID),
    ({"grad": None}, {}, (F32, F32, 32), INVALID), ({"m": None}, {}, (F32, F32, 32), INVALID),
    ({"m_scale": None}, {}, (F32, F32, 8), INVALID), ({"master": A}, {}, (F32, F32, 32), INVALID),
    ({"m": A + 2}, {}, (F32, F32, 32), INVALID), ({"param": A + 1}, {}, (BF16, F32, 32), INVALID),
    ({}, {"beta1": 1.0}, (F32, F32, 32), INVALID), ({}, {"beta2": -0.1}, (F32, F32, 32), INVALID),
    ({}, {"eps": -1.0}, (F32, F32, 32), INVALID), ({}, {"lr": float("inf")}, (F32, F32, 32), INVALID),
    ({}, {"weight_decay": float("nan")}, (F32, F32, 32), INVALID), ({}, {"step": 0}, (F32, F32, 32), INVALID),
])
def test_adamw_arguments(ops, kw, hyper, types, status):
    t = ops.AdamwTensorC(**dict(TENSOR, **kw))
    h = ops.AdamwHyperC(**dict(HYPER, **hyper))
    assert ops._lib().sffn_adamw_step(ctypes.byref(t), 1, *types, ctypes.byref(h), None, None) == status


def test_adamw_lists(ops):
    f = ops._lib()
    h = ops.AdamwHyperC(**HYPER)
    assert f.sffn_adamw_step(None, 0, F32, F32, 32, ctypes.byref(h), None, None) == OK
    assert f.sffn_adamw_step(None, 1, F32, F32, 32, ctypes.byref(h), None, None) == INVALID
    assert f.sffn_adamw_step(None, -1, F32, F32, 32, ctypes.byref(h), None, None) == INVALID
    two = (ops.AdamwTensorC * 2)(ops.AdamwTensorC(**TENSOR), ops.AdamwTensorC(**dict(TENSOR, master=A)))
    assert f.sffn_adamw_step(two, 2, BF16, F32, 32, ctypes.byref(h), None, None) == INVALID
    assert f.sffn_adamw_step(two, 1, F32, F32, 32, None, None, None) == INVALID
    assert f.sffn_adamw_step(two, 1, F32, F32, 32, ctypes.byref(h), A + 1, None) == INVALID


def test_binding_needs_device_tensors(ops):
    import torch
    x, g = torch.zeros(2, 64), torch.ones(64)
    for call in (lambda: ops.rms_norm(x, g), lambda: ops.rms_norm_fp8(x, g),
                 lambda: ops.rms_norm_backward(x, x, g, torch.ones(2)), lambda: ops.mx4_quantize(x),
                 lambda: ops.Mx4Linear(torch.zeros((2, 32), dtype=torch.uint8), torch.zeros((2, 2), dtype=torch.uint8)),
                 lambda: ops.AdamW([x])):
        with pytest.raises(ValueError):
            call()


def _message():
    from activation_sparse_transformer_amd import sparse_ffn
    return sparse_ffn.last_error()


B = 1 << 28  # distance of the stand-in arrays below: more than any of them is long


@pytest.mark.parametrize("kw", [
    {"h": 1 * B + 128}, {"h": 2 * B - 2}, {"h": 4 * B}, {"h": 3 * B}, {"h": 5 * B}, {"y": 1 * B + 2}, {"y": 1 * B + 64 * 2 * 9 + 126},
    {"y": 2 * B + 2}, {"y": 3 * B - 2}, {"y": 5 * B}, {"stat": 1 * B}, {"stat": 2 * B + 4}, {"stat": 3 * B + 124}, {"stat": 4 * B},
    # in place only with the same stride, and a row's own type
    {"x_stride": 80, "h": 1 * B}, {"x_stride": 80, "y": 1 * B}, {"residual_stride": 65, "h": 2 * B},
    {"x_stride": 80, "y": 1 * B + 80 * 2 * 9},
])
def test_norm_overlap(ops, kw):
    """Outputs over inputs or one another, by a whole array, by its edge, or in a strided row."""
    a = dict(NORM, rows=10, x=1 * B, residual=2 * B, gain=3 * B, y=4 * B, h=None, stat=5 * B)
    a.update(kw)
    for fn in ("sffn_rms_norm", "sffn_rms_norm_fp8"):
        assert getattr(ops._lib(), fn)(*a.values(), None) == INVALID and "overlap" in _message(), fn


def test_norm_fp8_is_not_in_place(ops):
    a = dict(NORM, rows=10, x=1 * B, residual=2 * B, gain=3 * B, y=1 * B, h=None, stat=5 * B)
    assert ops._lib().sffn_rms_norm_fp8(*a.values(), None) == INVALID and "overlap" in _message()


@pytest.mark.parametrize("rows", [40, 5000])  # dgain summed beside the rows, and in a second launch
@pytest.mark.parametrize("kw", [
    {"dx": "dy"}, {"dx": "h"}, {"dx": "dy", "dres": "dy"}, {"dx": "h", "dgain": None}, {"dx": "gain"}, {"dx": "rstd"},
    {"dres_stride": 66, "dx": "dres"}, {"dgain": "gain"}, {"dgain": "dy"}, {"dgain": "dres"}, {"dgain": "dx"},
    {"dgain": "rstd"},
])
def test_norm_backward_overlap(ops, rows, kw):
    at = {k: (i + 1) * B for i, k in enumerate(("dy", "h", "gain", "rstd", "dres", "dx", "dgain", "ws"))}
    a = dict(GRAD, rows=rows, **at)
    a.update({k: at.get(v, v) for k, v in kw.items()})
    assert ops._lib().sffn_rms_norm_backward(*a.values(), None) == INVALID and "overlap" in _message()
    edge = dict(GRAD, rows=rows, **at)
    edge["dx"] = at["dy"] + (rows - 1) * 128 + 126  # the last element
    assert ops._lib().sffn_rms_norm_backward(*edge.values(), None) == INVALID and "overlap" in _message()


def test_norm_backward_workspace_overlap(ops):
    at = {k: (i + 1) * B for i, k in enumerate(("dy", "h", "gain", "rstd", "dres", "dx", "dgain", "ws"))}
    for k in ("dy", "h", "gain", "rstd", "dres", "dx", "dgain"):
        a = dict(GRAD, **dict(at, ws=at[k]))
        assert ops._lib().sffn_rms_norm_backward(*a.values(), None) == INVALID and "overlap" in _message(), k


def test_mx4_overlap(ops):
    f = ops._lib()
    a = dict(tiled=1 * B, N=48, K=64, x_dtype=BF16, x=2 * B, x_stride=64, x_scale=3 * B, T=3, bias=4 * B, relu=1,
             y_dtype=F32, y=5 * B)
    for y in (1 * B, 1 * B + 1088 * 3 - 4, 2 * B, 2 * B + 2 * 128 + 124, 2 * B - 4, 3 * B + 8, 4 * B, 4 * B + 47 * 4):
        assert f.sffn_mx4_linear(*dict(a, y=y).values(), None) == INVALID and "overlap" in _message(), y
    far = dict(a, x_stride=1000, y=2 * B + 2000 * 2)  # over the last row
    assert f.sffn_mx4_linear(*far.values(), None) == INVALID and "overlap" in _message()
    for codes, scales in ((1 * B, 2 * B), (1 * B + 16 * 32 * 4 - 1, 2 * B), (2 * B, 1 * B), (2 * B, 2 * B + 16), (2 * B, 2 * B)):
        assert f.sffn_mx4_quantize(F32, 1 * B, 32, 16, 32, codes, scales, None) == INVALID and "overlap" in _message()
    for tiled in (1 * B, 2 * B, 2 * B - 16, 1 * B + 16 * 15):
        assert f.sffn_mx4_tile(1 * B, 2 * B, 16, 32, tiled, None) == INVALID and "overlap" in _message()


@pytest.mark.parametrize("kw,bits", [
    ({"grad": "param"}, 32), ({"grad": "m"}, 32), ({"v": "m"}, 32), ({"m": "param"}, 32), ({"master": "param"}, 32),
    ({"master": "v"}, 32), ({"m_scale": "v_scale"}, 8), ({"m_scale": "m"}, 8), ({"v": "m"}, 8), ({"grad": "v_scale"}, 8),
])
def test_adamw_overlap(ops, kw, bits):
    at = {k: (i + 1) * B for i, k in enumerate(("param", "grad", "master", "m", "v", "m_scale", "v_scale"))}
    t = ops.AdamwTensorC(n=300, **dict(at, **{k: at[v] for k, v in kw.items()}))
    h = ops.AdamwHyperC(**HYPER)
    assert ops._lib().sffn_adamw_step(ctypes.byref(t), 1, BF16, F32, bits, ctypes.byref(h), None, None) == INVALID
    assert "overlap" in _message()


@pytest.mark.parametrize("name", ["k_adamw", "k_rms_norm", "k_rms_norm_grad", "k_mx4"])
def test_vector_accesses_are_declared_at_their_alignment(name):
    """Vector accesses to memory of an element's alignment are written as such (a type's lower
    alignment is lost in a template argument, and the compiler may then rely on the vector's)."""
    import subprocess
    from activation_sparse_transformer_amd import build
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-Werror=align-mismatch", "-fsyntax-only", "--cuda-device-only",
                        os.path.join(build.CSRC, name + ".hip")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
