"""Host-only checks of the later operators of include/ffn_ops.h (layer norm, gradient norm and
clipping, 4-bit tokens): bad arguments are refused before anything reaches the GPU.  Runs without
a GPU."""
import ctypes
import os
import re
import subprocess

import pytest

A = 0x1000  # stands for a device pointer; never followed
OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16, E4M3 = 0, 1, 2
B = 1 << 28  # distance of the stand-in arrays below: more than any of them is long


@pytest.fixture(scope="module")
def ops():
    import activation_sparse_transformer_amd as sffn
    from activation_sparse_transformer_amd import ffn_ops
    if not os.path.exists(sffn.LIB_PATH):
        pytest.fail("libsparse_ffn.so is not built (run __graft_entry__.build())")
    return ffn_ops


def _message():
    from activation_sparse_transformer_amd import sparse_ffn
    return sparse_ffn.last_error()


NORM = dict(dtype=BF16, gain_dtype=BF16, x=A, x_stride=64, residual=A, residual_stride=64, gain=A, bias=A,
            eps=1e-5, rows=0, d=64, y=A, mean=A, stat=A, h=A)


def _norm(ops, a, fp8):
    if fp8:
        return ops._lib().sffn_layer_norm_fp8(*[v for k, v in a.items() if k != "mean"], None)
    return ops._lib().sffn_layer_norm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), ({"dtype": 7}, INVALID), ({"dtype": E4M3}, INVALID), ({"gain_dtype": E4M3}, INVALID),
    ({"dtype": F32, "gain_dtype": BF16}, INVALID), ({"gain_dtype": F32}, OK), ({"bias": None}, OK),
    ({"d": 0}, INVALID), ({"d": -1}, INVALID), ({"d": 32769}, UNSUPPORTED), ({"rows": -1}, INVALID),
    ({"rows": (1 << 40) + 1}, INVALID), ({"eps": -1e-6}, INVALID), ({"eps": float("nan")}, INVALID),
    ({"residual": None}, INVALID), ({"rows": 2, "x": None}, INVALID), ({"rows": 2, "x_stride": 63}, INVALID),
    ({"rows": 2, "residual_stride": 0}, INVALID), ({"rows": 2, "gain": None}, INVALID),
    ({"rows": 2, "y": None}, INVALID), ({"rows": 2, "x": A + 1}, INVALID), ({"rows": 2, "h": A + 1}, INVALID),
    ({"rows": 2, "stat": A + 2}, INVALID), ({"rows": 2, "gain": A + 1}, INVALID), ({"rows": 2, "bias": A + 1}, INVALID),
])
def test_norm_arguments(ops, kw, status):
    for fp8 in (False, True):
        assert _norm(ops, dict(NORM, **kw), fp8) == status


def test_norm_statistics_arguments(ops):
    assert _norm(ops, dict(NORM, rows=2, stat=None), True) == INVALID
    assert _norm(ops, dict(NORM, rows=2, mean=A + 2), False) == INVALID


AT = {k: (i + 1) * B for i, k in enumerate(("x", "residual", "gain", "bias", "y", "mean", "stat", "h"))}


@pytest.mark.parametrize("out,over", [(o, i) for o in ("y", "mean", "stat", "h") for i in AT if i != o])
def test_norm_overlap(ops, out, over):
    """Outputs over inputs or one another, by their first and by their last bytes."""
    size = {"x": 1280, "residual": 1280, "gain": 128, "bias": 128, "y": 1280, "mean": 40, "stat": 40, "h": 1280}
    for fp8 in (False, True):
        if fp8 and "mean" in (out, over):
            continue
        n = dict(size, y=640) if fp8 else size
        for at in (AT[over] + n[over] - 4, AT[over] - n[out] + 4):
            assert _norm(ops, dict(NORM, rows=10, **dict(AT, **{out: at})), fp8) == INVALID
            assert "overlap" in _message()


def test_norm_in_place_needs_the_same_rows(ops):
    for kw in ({"x_stride": 80, "h": AT["x"]}, {"x_stride": 80, "y": AT["x"]}, {"residual_stride": 65, "h": AT["residual"]}):
        assert _norm(ops, dict(NORM, rows=10, **dict(AT, **kw)), False) == INVALID and "overlap" in _message()
    assert _norm(ops, dict(NORM, rows=10, **dict(AT, y=AT["x"])), True) == INVALID and "overlap" in _message()


GRAD = dict(dtype=BF16, gain_dtype=F32, dy=A, dy_stride=64, h=A, h_stride=64, gain=A, mean=A, rstd=A, dres=A,
            dres_stride=64, rows=20000, d=64, dx=A, dgain=A, dbias=A, ws=A, nb=1 << 30)


@pytest.mark.parametrize("kw,status", [
    ({"rows": 0, "dgain": None, "dbias": None}, OK), ({"dtype": 5}, INVALID), ({"rows": -2}, INVALID),
    ({"d": 40000}, UNSUPPORTED), ({"dy": None}, INVALID), ({"h": None}, INVALID), ({"h_stride": 32}, INVALID),
    ({"dres_stride": 32}, INVALID), ({"rstd": None}, INVALID), ({"mean": None}, INVALID), ({"mean": A + 2}, INVALID),
    ({"dx": None}, INVALID), ({"ws": None}, INVALID), ({"ws": A + 8}, INVALID), ({"nb": 16}, INVALID),
    ({"dx": A + 1}, INVALID), ({"dgain": A + 1}, INVALID), ({"dbias": A + 2}, INVALID), ({"rows": 0}, INVALID),
])
def test_norm_backward_arguments(ops, kw, status):
    assert ops._lib().sffn_layer_norm_backward(*dict(GRAD, **kw).values(), None) == status


def test_norm_workspace(ops):
    f, n = ops._lib(), ctypes.c_size_t()
    for d in (1, 64, 2048, 16384, 16385, 32768):
        for rows in (0, 1, 4, 1000, 1025, 100000, 1 << 30, 1 << 40):
            assert f.sffn_layer_norm_backward_workspace(rows, d, ctypes.byref(n)) == OK
            assert n.value % (d * 8) == 0 and n.value <= 512 * d * 8
            if rows <= 1024 and (rows * d <= 1 << 20 or d > 16384):
                assert n.value == 0  # few rows are summed in the same launch
            elif d <= 16384 or rows > 1024:
                assert n.value > 0
    assert f.sffn_layer_norm_backward_workspace(4, 2048, None) == INVALID


@pytest.mark.parametrize("rows,d", [(40, 64), (20000, 64), (3000, 20000)])
def test_norm_backward_overlap(ops, rows, d):
    ins, outs = ("dy", "h", "gain", "mean", "rstd", "dres"), ("dx", "dgain", "dbias")
    far = 1 << 34
    at = {k: (i + 1) * far for i, k in enumerate(ins + outs + ("ws",))}
    base = dict(GRAD, rows=rows, d=d, dy_stride=d, h_stride=d, dres_stride=d)
    for out in outs:
        for over in ins + outs:
            if out == over or (out, over) == ("dx", "dres"):
                continue
            a = dict(base, **dict(at, **{out: at[over]}))
            assert ops._lib().sffn_layer_norm_backward(*a.values(), None) == INVALID, (out, over)
            assert "overlap" in _message(), (out, over)
    a = dict(base, **dict(at, dx=at["dres"], dres_stride=d + 2))
    assert ops._lib().sffn_layer_norm_backward(*a.values(), None) == INVALID and "overlap" in _message()
    n = ctypes.c_size_t()
    ops._lib().sffn_layer_norm_backward_workspace(rows, d, ctypes.byref(n))
    if n.value:
        for over in ins + outs:
            a = dict(base, **dict(at, ws=at[over]))
            assert ops._lib().sffn_layer_norm_backward(*a.values(), None) == INVALID and "overlap" in _message(), over


GRADIENT = dict(grad=1 * B, out=2 * B, n=300, dtype=F32, zero=0)
CALL = dict(max_norm=1.0, norm=5 * B, factor=6 * B, ws=7 * B, nb=1 << 20)


def _grad_call(ops, name, tensors, kw):
    arr = (ops.GradC * max(1, len(tensors)))(*[ops.GradC(**dict(GRADIENT, **t)) for t in tensors])
    a = dict(CALL, **kw)
    return getattr(ops._lib(), name)(ctypes.byref(arr), len(tensors), *a.values(), None)


@pytest.mark.parametrize("kw,call,status", [
    ({"n": -1}, {}, INVALID), ({"n": (1 << 40) + 1}, {}, INVALID), ({"dtype": E4M3}, {}, INVALID),
    ({"grad": None}, {}, INVALID), ({"grad": A + 2}, {}, INVALID), ({"dtype": BF16, "grad": A + 1}, {}, INVALID),
    ({}, {"max_norm": -1.0}, INVALID), ({}, {"max_norm": float("nan")}, INVALID), ({}, {"norm": None}, INVALID),
    ({}, {"norm": A + 2}, INVALID), ({}, {"factor": A + 2}, INVALID), ({}, {"ws": None}, INVALID),
    ({}, {"ws": 7 * B + 8}, INVALID), ({}, {"nb": 7}, INVALID),
])
def test_grad_norm_arguments(ops, kw, call, status):
    for name in ("sffn_grad_norm", "sffn_grad_clip"):
        assert _grad_call(ops, name, [kw], call) == status, name


def test_grad_clip_arguments(ops):
    for kw, call in (({"out": None}, {}), ({"out": 2 * B + 2}, {}), ({}, {"factor": None})):
        assert _grad_call(ops, "sffn_grad_clip", [kw], call) == INVALID
    f, n = ops._lib(), ctypes.c_size_t()
    assert f.sffn_grad_norm(None, 1, 1.0, A, A, A, 8, None) == INVALID
    assert f.sffn_grad_norm(None, -1, 1.0, A, A, A, 8, None) == INVALID
    assert f.sffn_grad_norm_workspace(None, 0, ctypes.byref(n)) == OK and n.value == 0
    assert f.sffn_grad_norm_workspace(None, 0, None) == INVALID


def test_grad_norm_workspace(ops):
    """About 1024 parts, and one more for each tensor's end."""
    f, n = ops._lib(), ctypes.c_size_t()
    for sizes in ([1], [4096], [4097], [0, 5, 0], [1 << 22], [(1 << 22) + 1] * 3, [1 << 40] * 4, [77] * 500):
        arr = (ops.GradC * len(sizes))(*[ops.GradC(n=k) for k in sizes])
        assert f.sffn_grad_norm_workspace(ctypes.byref(arr), len(sizes), ctypes.byref(n)) == OK
        assert n.value % 8 == 0 and sum(k > 0 for k in sizes) <= n.value // 8 <= 1024 + len(sizes)
    many = (ops.GradC * 1100)(*[ops.GradC(n=1 << 40) for _ in range(1100)])
    assert f.sffn_grad_norm_workspace(ctypes.byref(many), 1100, ctypes.byref(n)) == UNSUPPORTED


@pytest.mark.parametrize("kw,call", [
    ({}, {"norm": 6 * B}), ({}, {"norm": 1 * B + 1196}), ({}, {"factor": 1 * B}), ({}, {"ws": 1 * B + 1184}),
    ({}, {"ws": 5 * B}), ({}, {"norm": 2 * B}), ({}, {"factor": 2 * B + 1196}), ({}, {"ws": 2 * B}),
    ({"out": 1 * B + 4}, {}), ({"out": 1 * B - 1196}, {}),
])
def test_grad_clip_overlap(ops, kw, call):
    assert _grad_call(ops, "sffn_grad_clip", [kw], call) == INVALID and "overlap" in _message()
    if not kw and 2 * B not in call.values() and 2 * B + 1196 not in call.values():
        assert _grad_call(ops, "sffn_grad_norm", [kw], call) == INVALID and "overlap" in _message()


@pytest.mark.parametrize("n", [2, 130, 400])
def test_grad_clip_overlap_between_tensors(ops, n):
    """Of all gradients of a call, wherever in the list: what is written may meet nothing else; what is
    only read may come twice."""
    apart = [dict(grad=B + 4096 * i, out=B + 4096 * i) for i in range(n)]
    last = dict(grad=9 * B, out=B + 4 * 299)  # over the first one's last element
    for tensors in (apart + [apart[0]], apart + [dict(grad=9 * B, out=apart[n - 1]["grad"] + 1196)],
                    [last] + apart, apart + [dict(grad=B - 1196, out=9 * B)]):
        assert _grad_call(ops, "sffn_grad_clip", tensors, {}) == INVALID and "overlap" in _message()
    assert _grad_call(ops, "sffn_grad_norm", apart + [dict(grad=5 * B - 1196, out=None)], {}) == INVALID
    assert "overlap" in _message()


MATMUL = dict(tiled=1 * B, N=48, K=64, tokens=2 * B, T=33, bias=3 * B, relu=1, y_dtype=F32, y=4 * B)
QUANTIZED = dict(tiled=1 * B, N=48, K=64, x_dtype=BF16, x=2 * B, x_stride=64, T=33, bias=3 * B, relu=1, y_dtype=F32, y=4 * B,
                 ws=5 * B, nb=1 << 20)


@pytest.mark.parametrize("kw,status", [
    ({"T": 0}, OK), ({"N": 0}, OK), ({"N": -1}, INVALID), ({"K": 0}, INVALID), ({"T": -1}, INVALID),
    ({"T": (1 << 20) + 1}, UNSUPPORTED), ({"N": 1 << 30, "K": 1 << 20}, UNSUPPORTED), ({"N": 1, "K": (1 << 28) + 1}, UNSUPPORTED),
    ({"T": 1 << 20, "K": 1 << 17}, UNSUPPORTED), ({"T": 1 << 20, "N": (1 << 17) + 1, "K": 1}, UNSUPPORTED),
    ({"N": (1 << 26) + 1, "K": 1}, UNSUPPORTED), ({"y_dtype": E4M3}, INVALID), ({"tiled": None}, INVALID),
    ({"tiled": A + 8}, INVALID), ({"y": None}, INVALID), ({"y": 4 * B + 1}, INVALID), ({"bias": A + 2}, INVALID),
])
def test_mx4_products_arguments(ops, kw, status):
    f = ops._lib()
    assert f.sffn_mx4_matmul(*dict(MATMUL, **kw).values(), None) == status
    assert f.sffn_mx4_quantized(*dict(QUANTIZED, **kw).values(), None) == status


def test_mx4_tokens_arguments(ops):
    f, n = ops._lib(), ctypes.c_size_t()
    for kw in ({"tokens": None}, {"tokens": 2 * B + 8}):
        assert f.sffn_mx4_matmul(*dict(MATMUL, **kw).values(), None) == INVALID
    for kw in ({"x_dtype": E4M3}, {"x_dtype": 9}, {"x": None}, {"x": 2 * B + 1}, {"x_stride": 63}, {"ws": None}, {"ws": A + 8}, {"nb": 100}):
        assert f.sffn_mx4_quantized(*dict(QUANTIZED, **kw).values(), None) == INVALID, kw
    assert f.sffn_mx4_tokens_bytes(33, 129, ctypes.byref(n)) == OK and n.value == 3 * 2 * 1088
    assert f.sffn_mx4_quantized_workspace(33, 129, ctypes.byref(n)) == OK and n.value == 3 * 2 * 1088
    for T in (0, 1, 16):
        assert f.sffn_mx4_quantized_workspace(T, 129, ctypes.byref(n)) == OK and n.value == 0
    for fn in (f.sffn_mx4_tokens_bytes, f.sffn_mx4_quantized_workspace):
        assert fn(33, 129, None) == INVALID and fn(-1, 129, ctypes.byref(n)) == INVALID and fn(3, 0, ctypes.byref(n)) == INVALID
        assert fn((1 << 20) + 1, 1, ctypes.byref(n)) == UNSUPPORTED and fn(1, (1 << 28) + 1, ctypes.byref(n)) == UNSUPPORTED
    tokens = dict(dtype=BF16, x=1 * B, x_stride=64, T=33, K=64, tokens=2 * B)
    for kw, status in (({"T": 0, "x": None, "tokens": None}, OK), ({"dtype": E4M3}, INVALID), ({"x": None}, INVALID), ({"x": B + 1}, INVALID),
                       ({"x_stride": 63}, INVALID), ({"tokens": None}, INVALID), ({"tokens": 2 * B + 8}, INVALID), ({"T": -1}, INVALID),
                       ({"K": 0}, INVALID), ({"T": (1 << 20) + 1}, UNSUPPORTED)):
        assert f.sffn_mx4_tokens(*dict(tokens, **kw).values(), None) == status, kw


def test_mx4_tokens_overlap(ops):
    f = ops._lib()
    size = {"tiled": 3 * 1088, "tokens": 3 * 1088, "bias": 192, "x": 33 * 128, "ws": 3 * 1088, "y": 33 * 48 * 4}
    for over in ("tiled", "tokens", "bias"):
        for at in (MATMUL[over] + size[over] - 4, MATMUL[over] - size["y"] + 4):
            assert f.sffn_mx4_matmul(*dict(MATMUL, y=at).values(), None) == INVALID and "overlap" in _message(), over
    for out, ins in (("y", ("tiled", "x", "bias", "ws")), ("ws", ("tiled", "x", "bias"))):
        for over in ins:
            for at in (QUANTIZED[over] + size[over] // 16 * 16 - 16, QUANTIZED[over] - size[out] + 16):
                assert f.sffn_mx4_quantized(*dict(QUANTIZED, **{out: at}).values(), None) == INVALID, (out, over)
                assert "overlap" in _message(), (out, over)
    for at in (B + 33 * 128 - 16, B - 3 * 1088 + 16):
        assert f.sffn_mx4_tokens(BF16, B, 64, 33, 64, at, None) == INVALID and "overlap" in _message()


def test_binding_needs_device_tensors(ops):
    import torch
    x, g = torch.zeros(2, 64), torch.ones(64)
    for call in (lambda: ops.layer_norm(x, g), lambda: ops.layer_norm_fp8(x, g),
                 lambda: ops.layer_norm_backward(x, x, g, torch.ones(2), torch.ones(2)),
                 lambda: ops.grad_norm([x]), lambda: ops.clip_grads([x], 1.0), lambda: ops.Mx4Tokens(x)):
        with pytest.raises(ValueError):
            call()


def test_a_factor_needs_a_norm_to_clip_to(ops):
    """A factor without max_norm is refused before anything else of the call, by both entry points: with no norm to
    clip to, a clipping call would scale by a factor that nobody asked for."""
    import torch
    x, one = torch.ones(64), torch.ones(1)
    for call in (lambda: ops.clip_grads([x], None, factor=one), lambda: ops.clip_grads([x], None, out=[x], factor=one),
                 lambda: ops.grad_norm([x], factor=one)):
        with pytest.raises(ValueError, match="max_norm"):
            call()


@pytest.mark.parametrize("name", ["k_layer_norm", "k_layer_norm_grad", "k_grad_norm", "k_mx4_tokens", "k_mx4_matmul"])
def test_vector_accesses_are_declared_at_their_alignment(name):
    """As for the earlier operators: a vector access to memory of an element's alignment is written as one."""
    from activation_sparse_transformer_amd import build
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-Werror=align-mismatch", "-fsyntax-only", "--cuda-device-only",
                        os.path.join(build.CSRC, name + ".hip")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]


def test_lds_of_the_tokens_is_declared_as_it_is_read(tmp_path):
    """The rounding of tokens reads its LDS in pieces of 16 bytes (codes) and 4 (scales): the arrays are declared of
    those, so that their alignment is no matter of where the compiler puts them."""
    from activation_sparse_transformer_amd import build
    out = tmp_path / "tokens.ll"
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-O0", "-S", "-emit-llvm", "--cuda-device-only",
                        os.path.join(build.CSRC, "k_mx4_tokens.hip"), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    lds = re.findall(r"\d(codes|scales) = internal addrspace\(3\) global \[\d+ x (.*?)\]", out.read_text())
    assert len(lds) == 4 and set(lds) == {("codes", "<4 x i32>"), ("scales", "i32")}
