"""GPU tests of products of 4-bit tokens with 4-bit weights, against 64 bits on the host.

With u = 2^-24, a result is a sum of at most ceil(K / 128) + 8 parts (the instruction's sums of 128
columns, and the waves'), each addition off by at most two roundings of the absolute values summed, and
the bias's addition by one: tol = 2 (ceil(K / 128) + 8) u sum|x w| + u (sum|x w| + |bias|); a bf16 result
is the rounding of such a value.  Where all scales are alike the sums are exact."""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.mx4_matmul_forms import FORMS
from tests.ops_helpers import rounded_from

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def _dt(torch, name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _weights(codes, scales, K):
    """Dense float64 values of codes [N, 16 G] and scales [N, G]."""
    N, G = scales.shape
    c = np.stack((codes & 15, codes >> 4), 2).reshape(N, G, 32)
    z = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (E2M1[c] * z[:, :, None]).reshape(N, -1)[:, :K]


def _round4(x):
    """Tokens x [T, K] in float64, rounded: the nearest of the e2m1 values by distance, the even code of
    two equally near ones, at the largest power of two whose multiples by 4 do not exceed the group's
    largest value (at least 2^-127)."""
    T, K = x.shape
    x = np.pad(x, ((0, 0), (0, -K % 32))).reshape(T, -1, 32)
    with np.errstate(invalid="ignore", divide="ignore"):
        top = np.abs(x).max(axis=2, keepdims=True)
        e = np.frexp(np.where(np.isfinite(top) & (top > 0), top, 1e-300))[1] - 3
        unit = 2.0 ** np.maximum(e, -127).astype(np.float64)
        a = np.abs(x) / unit
        order = [0, 2, 4, 6, 1, 3, 5, 7]
        d = np.abs(a[..., None] - E2M1[order])
        v = E2M1[order][d.argmin(axis=-1)] * np.sign(x) * unit
    v = np.where(np.isfinite(top), v, np.nan)
    return v.reshape(T, -1)[:, :K]


def _make(torch, T, N, K, x_type, seed=0, spread=6, pad=0):
    rng = np.random.default_rng(seed)
    G = -(-K // 32)
    codes = rng.integers(0, 256, (N, 16 * G)).astype(np.uint8)
    scales = rng.integers(120, 121 + spread, (N, G)).astype(np.uint8)
    x = rng.standard_normal((T, K + pad)).astype(np.float32)
    x *= 2.0 ** rng.integers(0, 1 + spread, (T, 1))
    x = torch.from_numpy(x).to(_dt(torch, x_type)).cuda()[:, :K]
    return codes, scales, x


def _to(torch, a):
    return torch.from_numpy(a).cuda()


def _check(torch, sffn, T, N, K, x_type="bf16", y_type="f32", bias=True, relu=False, seed=0, spread=6, pad=0,
           rounding=None):
    codes, scales, x = _make(torch, T, N, K, x_type, seed, spread, pad)
    b = np.random.default_rng(seed + 1).standard_normal(N).astype(np.float32) if bias else None
    lin = sffn.Mx4Linear(_to(torch, codes), _to(torch, scales), bias=_to(torch, b) if bias else None, relu=relu, in_features=K)
    y = lin.quantized(x if rounding is not False else sffn.Mx4Tokens(x), dtype=_dt(torch, y_type))
    assert y.shape == (T, N) and y.dtype == _dt(torch, y_type)
    w, xq = _weights(codes, scales, K), _round4(x.cpu().double().numpy())
    ref, size = xq @ w.T, np.abs(xq) @ np.abs(w).T
    tol = 2 * (-(-K // 128) + 8) * U * size + U * size
    if bias:
        ref, tol = ref + b, tol + U * np.abs(b)
    got = y.cpu().double().numpy()
    if relu:
        assert (got >= 0).all()
        ok = rounded_from(got, ref, tol, y_type == "bf16") | ((got == 0) & (ref <= tol))
    else:
        ok = rounded_from(got, ref, tol, y_type == "bf16")
    assert ok.all(), (int((~ok).sum()), np.argwhere(~ok)[:4].tolist())
    return lin, x, y


TOKENS = [1, 2, 15, 16, 17, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300, 513]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("N,K", [(1000, 513), (129, 2304), (4100, 128)])
def test_token_counts(T, N, K):
    torch, sffn = need_gpu()
    _check(torch, sffn, T, N, K, "bf16" if T % 2 else "f32", "f32" if T % 3 else "bf16", relu=T % 4 == 0, seed=T)


@pytest.mark.parametrize("rounding,T,N,K,form", FORMS)
@pytest.mark.parametrize("y_type", ["f32", "bf16"])
def test_every_form(rounding, T, N, K, form, y_type):
    """Each kernel form that the rule selects (test_mx4_matmul_form.py holds it to these sizes)."""
    torch, sffn = need_gpu()
    x_type = "f32" if (T + N) % 4 else "bf16"
    lin, x, y = _check(torch, sffn, T, N, K, x_type, y_type, relu=T % 4 == 1, seed=form, rounding=rounding, pad=form % 3)
    again = lin.quantized(sffn.Mx4Tokens(x) if rounding is not False else x, dtype=y.dtype)
    assert torch.equal(again, y)  # rounded by the kernel or before it


@pytest.mark.parametrize("x_type", ["bf16", "f32"])
@pytest.mark.parametrize("N", [300, 8201, 20000])
def test_rounding_in_the_kernel(x_type, N):
    """Both types of tokens in every form that rounds them, the last group of columns in part."""
    torch, sffn = need_gpu()
    for K in (5, 32, 37, 120, 130, 1007):
        _check(torch, sffn, 7, N, K, x_type, "f32", seed=K, pad=3)


@pytest.mark.parametrize("K", [1, 2, 31, 32, 33, 63, 65, 96, 127, 128, 129, 255, 257, 384, 500, 640, 769, 896, 1025, 4000])
@pytest.mark.parametrize("T", [3, 40, 150])
def test_column_counts(T, K):
    torch, sffn = need_gpu()
    _check(torch, sffn, T, 250, K, "f32", "f32", bias=False, seed=K)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 7, 8, 15, 16, 17, 31, 33, 63, 65, 127, 129, 255, 257, 1023])
@pytest.mark.parametrize("T", [1, 20, 130])
@pytest.mark.parametrize("y_type", ["f32", "bf16"])
def test_row_counts(T, N, y_type):
    torch, sffn = need_gpu()
    _check(torch, sffn, T, N, 200, "bf16", y_type, seed=N)


@pytest.mark.parametrize("T,N,K", [(2000, 4500, 300), (4096, 8192, 130), (1000, 20000, 96), (20000, 1000, 64)])
@pytest.mark.parametrize("y_type", ["f32", "bf16"])
def test_many_tiles(T, N, K, y_type):
    torch, sffn = need_gpu()
    _check(torch, sffn, T, N, K, "bf16", y_type, relu=True, pad=8)


@pytest.mark.parametrize("x_type", ["bf16", "f32"])
def test_rounding_of_tokens(x_type):
    """Through a matrix that copies columns (ones on the diagonal): values at, next to and between the
    middles of neighbouring codes, of every exponent that the type has, come out as the rounded values."""
    torch, sffn = need_gpu()
    K = 256
    rng = np.random.default_rng(3)
    codes = np.zeros((K, K // 2), np.uint8)
    codes[np.arange(K), np.arange(K) // 2] = np.where(np.arange(K) % 2 == 0, 2, 0x20)
    lin = sffn.Mx4Linear(_to(torch, codes), torch.full((K, K // 32), 127, dtype=torch.uint8, device="cuda"))
    mid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9])
    rows = []
    for e in list(range(-149, 125, 7)) + [-133, -132, -130, -129, -128, -127, -126, -125, -3, 0, 124]:
        v = rng.choice(mid, K) * 2.0 ** e * rng.choice([-1, 1], K)
        v = v.astype(np.float32)
        near = rng.integers(0, 3, K)
        v = np.where(near == 1, np.nextafter(v, np.float32(np.inf)), np.where(near == 2, np.nextafter(v, np.float32(-np.inf)), v))
        v.reshape(-1, 32)[::2, 5] = np.float32(min(4 * 2.0 ** e, 2.0 ** 126))  # some groups' largest value is a power of two
        rows.append(v)
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(_dt(torch, x_type))
    got = lin.quantized(x.cuda(), dtype=torch.float32).cpu().double().numpy()
    assert np.array_equal(got, _round4(x.double().numpy()))


def test_rounds_as_the_weights_are():
    """Tokens and weights of the same values are rounded alike: the products with a quantised copy of the
    tokens are those of the rounded values with themselves."""
    torch, sffn = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((40, 300), generator=g, device="cuda")
    codes, scales = sffn.mx4_quantize(x)
    w = _weights(codes.cpu().numpy(), scales.cpu().numpy(), 300)
    assert np.array_equal(w, _round4(x.cpu().double().numpy()))
    y = sffn.Mx4Linear.from_dense(x).quantized(x).cpu().double().numpy()
    size = np.abs(w) @ np.abs(w).T
    assert (np.abs(y - w @ w.T) <= 24 * U * size).all()


@pytest.mark.parametrize("T", [1, 16, 50, 200, 600])
def test_exact_sums(T):
    """Alike scales: every product and sum is a multiple of 1/4 below 2^22, so all forms give the exact
    value, and a token's results do not depend on the tokens beside it."""
    torch, sffn = need_gpu()
    rng = np.random.default_rng(T)
    N, K = 700, 1100
    codes = rng.integers(0, 256, (N, 16 * 35)).astype(np.uint8)
    lin = sffn.Mx4Linear(_to(torch, codes), torch.full((N, 35), 127, dtype=torch.uint8, device="cuda"), in_features=K)
    v = rng.choice(E2M1, (T, K))
    v[:, ::32] = 4.0  # the groups' scale is 1
    v[:, 1099] = 4.0
    x = torch.from_numpy(v).float().cuda()
    y = lin.quantized(x)
    ref = v @ _weights(codes, np.full((N, 35), 127, np.uint8), K).T
    assert np.array_equal(y.cpu().double().numpy(), ref)
    assert torch.equal(lin.quantized(x[T // 2:T // 2 + 1]), y[T // 2:T // 2 + 1])


@pytest.mark.parametrize("T", [5, 90, 300])
def test_scales_far_apart(T):
    """Weight scales over the whole range against tokens that bring the products back, and rows whose
    groups' scales lie far apart."""
    torch, sffn = need_gpu()
    N, K = 254, 256
    rng = np.random.default_rng(T)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = np.tile(np.arange(N, dtype=np.uint8)[:, None], (1, K // 32))
    lin = sffn.Mx4Linear(_to(torch, codes), _to(torch, scales))
    w = _weights(codes, scales, K)
    for e in (-100, 0, 100):
        x = (rng.standard_normal((T, K)) * 2.0 ** e).astype(np.float32)
        y = lin.quantized(_to(torch, x)).cpu().double().numpy()
        xq = _round4(x.astype(np.float64))
        ref, size = xq @ w.T, np.abs(xq) @ np.abs(w).T
        fits = (size > 2.0 ** -100) & (size < 2.0 ** 127)  # away from the ends of fp32
        assert fits.any() and (np.abs(y - ref) <= 21 * U * size)[fits].all()
    scales = rng.integers(100, 154, (N, K // 32)).astype(np.uint8)
    lin = sffn.Mx4Linear(_to(torch, codes), _to(torch, scales))
    w = _weights(codes, scales, K)
    x = (rng.standard_normal((T, K)) * 2.0 ** rng.integers(-25, 25, (T, K // 32)).repeat(32, 1)).astype(np.float32)
    y = lin.quantized(_to(torch, x)).cpu().double().numpy()
    xq = _round4(x.astype(np.float64))
    assert (np.abs(y - xq @ w.T) <= 21 * U * (np.abs(xq) @ np.abs(w).T)).all()


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("y_type", ["f32", "bf16"])
def test_not_finite(T, y_type):
    """An infinity or a NaN in a token makes that token's results NaN, a NaN scale its row's: no others.
    ReLU keeps NaN.  An infinite bias stays."""
    torch, sffn = need_gpu()
    N, K = 300, 200
    codes, scales, x = _make(torch, T, N, K, "f32")
    x = x.clone()
    x[1, 7], x[2, 199] = float("inf"), float("nan")
    scales[5, 3] = scales[299, 0] = 255
    bias = torch.zeros(N, device="cuda")
    bias[9] = float("inf")
    lin = sffn.Mx4Linear(_to(torch, codes), _to(torch, scales), bias=bias, relu=True, in_features=K)
    y = lin.quantized(x, dtype=_dt(torch, y_type)).float()
    rows = [t for t in range(T) if t not in (1, 2)]
    cols = [n for n in range(N) if n not in (5, 9, 299)]
    assert torch.isnan(y[[1, 2]]).all() and torch.isnan(y[:, [5, 299]]).all()
    assert torch.isinf(y[rows][:, 9]).all()
    assert torch.isfinite(y[rows][:, cols]).all()


@pytest.mark.parametrize("T", [2, 70, 300])
def test_tokens_made_once_strides_and_given_output(T):
    torch, sffn = need_gpu()
    lin, x, y = _check(torch, sffn, T, 777, 333, "bf16", "bf16", relu=True, pad=17)
    tokens = sffn.Mx4Tokens(x)
    assert tokens.shape == (T, 333) and tokens.dtype == torch.bfloat16 and tokens.device == x.device
    assert torch.equal(lin.quantized(tokens), y)
    flat = torch.full((T * 777 + 3,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = flat[1:T * 777 + 1].view(T, 777)
    assert lin.quantized(x.contiguous(), y=out) is out
    assert torch.equal(out, y) and flat[0] == 9 and (flat[-2:] == 9).all()  # what lies around it stays
    f = torch.full((T * 777 + 3,), 9.0, device="cuda")
    out = f[1:T * 777 + 1].view(T, 777)
    lin.quantized(tokens, y=out)
    assert torch.equal(out.bfloat16(), y) and f[0] == 9 and (f[-2:] == 9).all()
    base = torch.zeros(T * 333 + 1, dtype=torch.bfloat16, device="cuda")  # rows at odd addresses
    base[1:] = x.reshape(-1)
    assert torch.equal(lin.quantized(base[1:].view(T, 333)), y)


def test_no_tokens_and_no_rows():
    torch, sffn = need_gpu()
    lin = sffn.Mx4Linear.from_dense(torch.randn((64, 96), device="cuda"))
    assert lin.quantized(torch.empty((0, 96), device="cuda")).shape == (0, 64)
    none = sffn.Mx4Linear(torch.empty((0, 48), dtype=torch.uint8, device="cuda"), torch.empty((0, 3), dtype=torch.uint8, device="cuda"))
    assert none.quantized(torch.zeros((5, 96), device="cuda")).shape == (5, 0)


def test_the_most_tokens():
    torch, sffn = need_gpu()
    T = 1 << 20
    codes, scales, x = _make(torch, 64, 40, 70, "bf16")
    lin = sffn.Mx4Linear(_to(torch, codes), _to(torch, scales), in_features=70)
    first = lin.quantized(x)
    y = lin.quantized(x.repeat(T // 64, 1))
    assert y.shape == (T, 40) and (y.view(-1, 64, 40) == first).all()
    with pytest.raises(sffn.SffnError) as ei:
        lin.quantized(torch.zeros((T + 1, 70), dtype=torch.bfloat16, device="cuda"))
    assert ei.value.status == sffn.SFFN_ERR_UNSUPPORTED


@pytest.mark.parametrize("T", [3, 40, 200])
def test_long_rows(T):
    torch, sffn = need_gpu()
    _check(torch, sffn, T, 130, 70001, "bf16", "f32", spread=3)


def test_the_longest_rows():
    """2^28 columns, a row of blocks of more than 2^31 bytes: zeros but for few columns on both sides of its middle,
    of values that 4 bits hold, so that the sums are exact."""
    torch, sffn = need_gpu()
    N, K = 9, 1 << 28
    columns = [0, 5, 31, 127, 128, (1 << 27) - 1, 1 << 27, 252_645_136, 252_645_137, K - 33, K - 1]
    rng = np.random.default_rng(4)
    value = rng.integers(0, 16, (N, len(columns)))
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    for j, c in enumerate(columns):
        codes[:, c // 2] |= torch.from_numpy((value[:, j] << (4 * (c % 2))).astype(np.uint8)).cuda()
    lin = sffn.Mx4Linear(codes, torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda"))
    del codes
    assert lin.tiled.numel() > 1 << 31
    x = torch.zeros((17, K), dtype=torch.bfloat16, device="cuda")
    v = 2.0 ** rng.integers(0, 3, (17, len(columns))) * rng.choice([-1, 1], (17, len(columns)))
    for j, c in enumerate(columns):
        x[:, c] = torch.from_numpy(v[:, j]).cuda().to(torch.bfloat16)
    ref = torch.from_numpy(v @ E2M1[value].T).cuda().float()
    for t in (3, 17):  # rounded by the kernel, and before it
        assert torch.equal(lin.quantized(x[:t], dtype=torch.float32), ref[:t])
    assert torch.equal(lin.quantized(sffn.Mx4Tokens(x), dtype=torch.float32), ref)


def test_offsets_beyond_32_bits():
    """More than 2^31 results, and tokens more than 2^31 elements apart."""
    torch, sffn = need_gpu()
    T, N, K = 70000, 32768, 40
    codes, scales, x = _make(torch, T, N, K, "bf16")
    lin = sffn.Mx4Linear(_to(torch, codes), _to(torch, scales), in_features=K)
    y = lin.quantized(x)
    part = lin.quantized(x[-300:], dtype=torch.bfloat16)
    assert torch.equal(y[-300:], part) and torch.equal(y[:300], lin.quantized(x[:300]))
    del y
    stride = (1 << 31) + 24
    big = torch.zeros(stride + K, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((2, K), (stride, 1))
    far.copy_(x[:2])
    assert torch.equal(lin.quantized(far), lin.quantized(x[:2].contiguous()))


def test_streams_and_graph():
    """On another stream; recorded in a graph and replayed on new tokens with eager work between."""
    torch, sffn = need_gpu()
    for T in (1, 60, 300):
        lin, x, y = _check(torch, sffn, T, 600, 512, "bf16", "bf16", relu=True)
        x = x.contiguous()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y2 = lin.quantized(x, stream=side)
        tokens = sffn.Mx4Tokens(x, stream=side)
        y3 = lin.quantized(tokens, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, y2) and torch.equal(y, y3)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = lin.quantized(x)
        for k in range(3):
            x.copy_(torch.randn_like(x))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, lin.quantized(x))


def test_follows_a_replaced_bias():
    torch, sffn = need_gpu()
    lin, x, y = _check(torch, sffn, 20, 300, 128)
    new = torch.randn(300, device="cuda")
    lin.bias.data = new
    assert torch.allclose(lin.quantized(x, dtype=torch.float32) - new, lin.quantized(x, dtype=torch.float32) - lin.bias)
    lin.bias = None
    zero = lin.quantized(x, dtype=torch.float32)
    lin.bias = new
    assert torch.equal(lin.quantized(x, dtype=torch.float32), zero + new)


def test_works_on_replaced_tensors():
    """Products of 4-bit tokens take the bias and the weights as they stand, with another storage behind them too; a
    layout that does not fit is refused.  Each expected value is of other tensors than the layer's own."""
    torch, sffn = need_gpu()
    for T in (7, 20, 300):  # rounded by the kernel, before it, and in tiles
        codes, scales, x = _make(torch, T, 300, 128, "f32")
        bias = torch.zeros(300, device="cuda")
        lin = sffn.Mx4Linear(_to(torch, codes), _to(torch, scales), bias=bias)
        for tokens in (x, sffn.Mx4Tokens(x)):
            lin.bias = None
            y0 = lin.quantized(tokens)
            b = torch.randn(300, device="cuda")
            lin.bias = bias
            assert torch.equal(lin.quantized(tokens), y0)
            bias.data = b.clone()
            assert torch.equal(lin.quantized(tokens), y0 + b)  # (the bias's addition is one rounding in both)
            bias.data = torch.zeros(300, device="cuda")
            assert torch.equal(lin.quantized(tokens), y0)
            own = lin.tiled.clone()
            other = sffn.Mx4Linear(_to(torch, codes ^ 0x88), _to(torch, scales))  # every sign turned
            lin.tiled.data = other.tiled.clone()
            assert torch.equal(lin.quantized(tokens), -y0) and not torch.equal(y0, -y0)
            lin.tiled.data = own[:-1].clone()
            with pytest.raises(ValueError):
                lin.quantized(tokens)
            lin.tiled.data = own
            assert torch.equal(lin.quantized(tokens), y0)


def test_refusals():
    torch, sffn = need_gpu()
    lin = sffn.Mx4Linear.from_dense(torch.randn((64, 96), device="cuda"))
    x = torch.zeros((4, 96), device="cuda")
    q = sffn.Mx4Tokens(x)
    bad = [
        lambda: lin.quantized(x.half()),
        lambda: lin.quantized(x.cpu()),
        lambda: lin.quantized(x[:, :64]),
        lambda: lin.quantized(x[0]),
        lambda: lin.quantized(x.t()),
        lambda: lin.quantized(x, dtype=torch.float16),
        lambda: lin.quantized(x, y=torch.empty((4, 63), device="cuda")),
        lambda: lin.quantized(x, y=torch.empty((4, 64), device="cuda"), dtype=torch.bfloat16),
        lambda: lin.quantized(x, y=torch.empty((4, 64))),
        lambda: lin.quantized(sffn.Mx4Tokens(x[:, :64])),
        lambda: lin.quantized(x[0].expand(4, 96)),
        lambda: sffn.Mx4Tokens(x.cpu()),
        lambda: sffn.Mx4Tokens(x.double()),
        lambda: sffn.Mx4Tokens(x[0]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(sffn.SffnError) as ei:
        lin.quantized(q, y=q._data[:4 * 64 * 4].view(torch.float32).view(4, 64))
    assert ei.value.status == sffn.SFFN_ERR_INVALID_ARGUMENT
    for name in ("shape", "dtype", "device"):
        with pytest.raises(AttributeError):
            setattr(q, name, None)
