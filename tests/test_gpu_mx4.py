"""GPU tests of the 4-bit weights: quantisation, and products at serving batches, against the
format's definition and sums in 64 bits on the host.

Tolerance of a product: every e2m1 weight times its power of two and every token value is exact
in the kernel's operands, so only the additions round: at most K + 16 of them on a path, each at
most 2^-23 of the sum of absolute products (2^-24 to nearest; twice that allows truncation inside
the matrix cores), then the scale and bias (2^-23 of the result's terms); a bf16 output is the
rounding of such a value."""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.mx4_forms import FORMS
from tests.ops_helpers import rounded_from

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def _weights(rng, N, K, lo=118, hi=124):
    G = -(-K // 32)
    return (rng.integers(0, 256, (N, 16 * G)).astype(np.uint8),
            rng.integers(lo, hi, (N, G)).astype(np.uint8))


def _decode(codes, scales, K):
    N, G = scales.shape
    c = np.stack((codes & 15, codes >> 4), 2).reshape(N, 32 * G)
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    return (E2M1[c] * np.repeat(s, 32, axis=1))[:, :K]


def _tokens(torch, rng, T, K, kind, pad=0):
    x = torch.from_numpy(rng.standard_normal((T, K + pad)).astype(np.float32)).cuda()
    if kind == "fp8":
        sc = (x.abs().amax(1) / 448).contiguous()
        return (x / sc[:, None]).to(torch.float8_e4m3fn)[:, :K], sc
    return x.to(torch.bfloat16 if kind == "bf16" else torch.float32)[:, :K], None


def _check(torch, sffn, T, N, K, kind, y_dtype, bias, relu, seed=0, pad=0):
    rng = np.random.default_rng(seed + 131 * T + 17 * N + K)
    codes, scales = _weights(rng, N, K)
    x, sc = _tokens(torch, rng, T, K, kind, pad)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    lin = sffn.Mx4Linear(to(codes), to(scales), bias=None if b is None else to(b), relu=relu,
                         in_features=K)
    y = lin(x, x_scale=sc, dtype=y_dtype)
    W = _decode(codes, scales, K)
    x64 = x.float().cpu().double().numpy()
    s64 = 1.0 if sc is None else sc.cpu().double().numpy()[:, None]
    z = (x64 @ W.T) * s64
    size = (np.abs(x64) @ np.abs(W).T) * s64
    if b is not None:
        z, size = z + b, size + np.abs(b)
    if relu:
        z = np.maximum(z, 0)
    tol = (K + 20) * 2.0 ** -23 * size + 1e-30
    ok = rounded_from(y.float().cpu().double().numpy(), z, tol, y_dtype == torch.bfloat16)
    assert y.shape == (T, N) and np.all(ok), (T, N, K, kind, int((~ok).sum()))
    return lin, x, sc, y


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 48, 64, 65, 130])
def test_tokens(T, kind):
    torch, sffn = need_gpu()
    _check(torch, sffn, T, 80, 416, kind, torch.float32, True, False)


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 31), (15, 32), (16, 33), (17, 96), (33, 127), (100, 128),
                                 (31, 129), (64, 1000), (257, 2048), (2049, 160), (48, 8200)])
def test_sizes(N, K, kind):
    torch, sffn = need_gpu()
    for T, y_dtype, bias, relu in ((1, torch.float32, False, False), (5, torch.bfloat16, True, True),
                                   (40, torch.float32, True, True)):
        _check(torch, sffn, T, N, K, kind, y_dtype, bias, relu, pad=3)


def test_serving_shapes():
    """The up-projections of the 1.5B- and 2B-like layers."""
    torch, sffn = need_gpu()
    for T, N, K, kind in ((1, 8192, 2048, "bf16"), (7, 8192, 2048, "fp8"), (64, 9216, 2304, "fp8"),
                          (16, 6144, 1536, "f32")):
        lin, x, sc, y = _check(torch, sffn, T, N, K, kind, torch.float32, True, True)
        assert torch.equal(y, lin(x, x_scale=sc, dtype=torch.float32))
        # a token's result does not depend on how many others there are
        one = lin(x[:1], x_scale=None if sc is None else sc[:1], dtype=torch.float32)
        tol = (K + 20) * 2.0 ** -22 * float(y.abs().max() + x.float().abs().max() * K ** 0.5)
        assert float((one - y[:1]).abs().max()) <= tol


def test_scales_at_the_ends():
    """The smallest and largest powers of two, and 255, which is NaN."""
    torch, sffn = need_gpu()
    N, K = 16, 64
    rng = np.random.default_rng(0)
    codes, scales = _weights(rng, N, K)
    scales[:] = 127
    scales[0], scales[1], scales[2], scales[3, 1] = 0, 1, 240, 255
    W = _decode(codes, scales, K)
    x = torch.full((2, K), 0.25, device="cuda")
    x[1] = -2.0
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    for kind in (torch.float32, torch.bfloat16):
        y = sffn.Mx4Linear(to(codes), to(scales))(x.to(kind), dtype=torch.float32)
        z = x.cpu().double().numpy() @ W.T
        got = y.cpu().double().numpy()
        assert np.isnan(got[:, 3]).all()
        rest = [n for n in range(N) if n != 3]
        size = np.abs(x.cpu().double().numpy()) @ np.abs(W).T
        # the smallest weights are subnormal: they may count as zero
        tol = 200 * 2.0 ** -23 * size + np.array([K * 2 * 6 * 2.0 ** -126 if n < 2 else 0 for n in range(N)])
        assert np.all(np.abs(got - z)[:, rest] <= tol[:, rest])


def test_infinities_in_tokens():
    torch, sffn = need_gpu()
    rng = np.random.default_rng(1)
    codes, scales = _weights(rng, 32, 128)
    codes[0], codes[1] = 0x22, 0xAA  # all 1, all -1
    codes[2] = 0
    x = torch.from_numpy(rng.standard_normal((3, 128)).astype(np.float32)).cuda()
    x[1, 100] = float("inf")
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    lin = sffn.Mx4Linear(to(codes), to(scales))
    for kind in (torch.float32, torch.bfloat16):
        clean = lin(x[::2].to(kind).contiguous(), dtype=torch.float32)
        y = lin(x.to(kind), dtype=torch.float32)
        assert torch.equal(y[::2], clean)
        assert y[1, 0] == float("inf") and y[1, 1] == float("-inf") and torch.isnan(y[1, 2])
    big = torch.full((1, 128), 3.4e38, device="cuda")  # would round up to infinity in bf16
    big[0, 1:] = 0
    y = lin(big)
    w = _decode(codes, scales, 128)
    assert torch.isfinite(y).all()
    assert np.allclose(y.cpu().double().numpy()[0], 3.4e38 * w[:, 0], rtol=1e-6)


def test_layout_of_tokens():
    """Strided, unaligned and far-apart token rows give the bits of plain ones."""
    torch, sffn = need_gpu()
    rng = np.random.default_rng(2)
    codes, scales = _weights(rng, 40, 96)
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    lin = sffn.Mx4Linear(to(codes), to(scales))
    for kind in ("bf16", "f32", "fp8"):
        x, sc = _tokens(torch, rng, 3, 96, kind)
        y = lin(x, x_scale=sc, dtype=torch.float32)
        flat = torch.empty(3 * 96 + 1, dtype=x.dtype, device="cuda")
        flat[1:].view(torch.uint8).copy_(x.contiguous().view(-1).view(torch.uint8))
        assert torch.equal(lin(flat[1:].view(3, 96), x_scale=sc, dtype=torch.float32), y)
    x, _ = _tokens(torch, rng, 2, 96, "bf16")
    far = torch.zeros((1 << 31) + 200, dtype=torch.bfloat16, device="cuda").as_strided((2, 96), ((1 << 31) + 40, 1))
    far.copy_(x)
    assert torch.equal(lin(far), lin(x))


def test_weights_beyond_32_bits():
    """A layout of more than 2^31 bytes: its last rows give what they give alone."""
    torch, sffn = need_gpu()
    N, K, last = (1 << 22) + 9, 1024, 25
    rng = np.random.default_rng(5)
    codes, scales = _weights(rng, last, K)
    big = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    sc = torch.full((N, K // 32), 120, dtype=torch.uint8, device="cuda")
    big[-last:], sc[-last:] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    lin = sffn.Mx4Linear(big, sc)
    assert lin.tiled.numel() > 1 << 31
    del big, sc
    x = torch.from_numpy(rng.standard_normal((2, K)).astype(np.float32)).cuda().to(torch.bfloat16)
    y = lin(x, dtype=torch.float32)
    z = x.float().cpu().double().numpy() @ _decode(codes, scales, K).T
    size = np.abs(x.float().cpu().double().numpy()) @ np.abs(_decode(codes, scales, K)).T
    assert np.all(np.abs(y[:, -last:].cpu().double().numpy() - z) <= (K + 20) * 2.0 ** -23 * size + 1e-30)
    assert not y[:, :-last].any()


def test_empty_and_streams():
    torch, sffn = need_gpu()
    rng = np.random.default_rng(3)
    codes, scales = _weights(rng, 64, 256)
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    lin = sffn.Mx4Linear(to(codes), to(scales))
    assert lin(torch.empty((0, 256), device="cuda")).shape == (0, 64)
    x = torch.from_numpy(rng.standard_normal((4, 256)).astype(np.float32)).cuda()
    want = lin(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = lin(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)


def _quantize_reference(W):
    """Codes and scales by the definition, in 64 bits: nearest value, ties to the even code."""
    N, K = W.shape
    G = -(-K // 32)
    codes, scales = np.zeros((N, 32 * G), np.uint8), np.zeros((N, G), np.uint8)
    mags = E2M1[:8]
    for n in range(N):
        for g in range(G):
            w = W[n, g * 32:(g + 1) * 32]
            if not np.isfinite(w).all():
                scales[n, g] = 255
                continue
            big = np.abs(w).max()
            e = max(-127, int(np.floor(np.log2(big))) - 2) if big > 0 else -127
            scales[n, g] = e + 127
            a = np.abs(w) * 2.0 ** -e
            for k, v in enumerate(a):
                dist = np.abs(mags - min(v, 6.0))
                near = np.flatnonzero(dist == dist.min())
                c = next((i for i in near if i % 2 == 0), near[0])
                codes[n, g * 32 + k] = c | (8 if w[k] < 0 else 0)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


@pytest.mark.parametrize("K", [1, 32, 45, 96])
def test_quantize(K):
    torch, sffn = need_gpu()
    rng = np.random.default_rng(K)
    W = rng.standard_normal((24, K)).astype(np.float32)
    W[1] = 0
    W[2] *= 1e-30
    W[3] *= 2.0 ** 120
    W[4, 0] = np.nan
    W[5, K - 1] = np.inf
    W[6] *= 1e-41  # subnormal
    W[7] = np.float32(0.25) * rng.integers(-24, 25, K)  # many ties
    W[8] = 6.0
    W[9] = 2.0 ** -126
    for dt in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(W).to(dt).cuda()
        codes, scales = sffn.mx4_quantize(t)
        c, s = _quantize_reference(t.float().cpu().numpy().astype(np.float64))
        assert np.array_equal(scales.cpu().numpy(), s)
        assert np.array_equal(codes.cpu().numpy(), c)
        # strided rows, and the layer made from the dense weights
        wide = torch.zeros((24, K + 5), dtype=dt, device="cuda")
        wide[:, :K] = t
        c2, s2 = sffn.mx4_quantize(wide[:, :K])
        assert torch.equal(c2, codes) and torch.equal(s2, scales)
    ok = torch.from_numpy(np.delete(W, [4, 5], axis=0)).cuda()
    lin = sffn.Mx4Linear.from_dense(ok)
    x = torch.ones((1, K), device="cuda")
    assert lin.in_features == K and torch.isfinite(lin(x)).all()


def test_refusals():
    torch, sffn = need_gpu()
    codes = torch.zeros((8, 32), dtype=torch.uint8, device="cuda")
    scales = torch.full((8, 2), 127, dtype=torch.uint8, device="cuda")
    lin = sffn.Mx4Linear(codes, scales)
    x = torch.zeros((2, 64), device="cuda")
    bad = [
        lambda: sffn.Mx4Linear(codes[:, :16], scales),
        lambda: sffn.Mx4Linear(codes.cpu(), scales),
        lambda: sffn.Mx4Linear(codes, scales, bias=torch.zeros(7, device="cuda")),
        lambda: sffn.Mx4Linear(codes, scales, in_features=32),
        lambda: sffn.Mx4Linear(codes, scales, in_features=65),
        lambda: sffn.mx4_quantize(x.half()),
        lambda: lin(x[:, :32]),
        lambda: lin(x.half()),
        lambda: lin(x.to(torch.float8_e4m3fn)),
        lambda: lin(x, x_scale=torch.ones(3, device="cuda")),
        lambda: lin(x, dtype=torch.float16),
        lambda: lin(x, y=torch.zeros((2, 9), device="cuda")),
        lambda: lin(x, y=torch.zeros((2, 8), device="cuda"), dtype=torch.bfloat16),
        lambda: lin(x.t().contiguous().t()),
        lambda: lin(x.cpu()),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_replaced_tensors():
    """A call works on the bias and the weights as they stand, whether assigned or with another
    storage behind them; what does not fit is refused and changes nothing."""
    torch, sffn = need_gpu()
    rng = np.random.default_rng(6)
    codes, scales = _weights(rng, 40, 96)
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    bias = torch.zeros(40, device="cuda")
    lin = sffn.Mx4Linear(to(codes), to(scales), bias=bias)
    x = to(rng.standard_normal((3, 96)).astype(np.float32))
    y0 = lin(x)
    b = to(rng.standard_normal(40).astype(np.float32))
    bias.data = b.clone()
    assert torch.equal(lin(x), y0 + b)
    lin.bias = 2 * b
    assert torch.equal(lin(x), y0 + 2 * b) and torch.equal(lin.bias, 2 * b)
    for bad in (b[:39], b.double(), b.cpu(), torch.zeros(80, device="cuda")[::2]):
        with pytest.raises(ValueError):
            lin.bias = bad
    assert torch.equal(lin(x), y0 + 2 * b)
    lin.bias = None
    assert torch.equal(lin(x), y0)
    lin.relu = True
    assert torch.equal(lin(x), y0.clamp_min(0))
    lin.relu = False
    other = sffn.Mx4Linear(to(codes ^ 0x88), to(scales))  # every sign turned
    lin.tiled.data = other.tiled.clone()
    assert torch.equal(lin(x), other(x)) and not torch.equal(other(x), y0)
    lin.tiled.data = other.tiled[:-1].clone()
    with pytest.raises(ValueError):
        lin(x)
    for name in ("tiled", "in_features", "out_features", "device"):
        with pytest.raises(AttributeError):
            setattr(lin, name, getattr(lin, name))


def _decode_on_gpu(torch, codes, scales, K):
    """_decode, for weights that are large on the host."""
    c = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1).long()
    w = torch.from_numpy(E2M1).cuda()[c]
    return (w * torch.exp2(scales.double() - 127).repeat_interleave(32, 1))[:, :K]


@pytest.mark.parametrize("kind,T,N,K,form", FORMS)
def test_every_form(kind, T, N, K, form):
    """Every kernel form of the product, every result against 64 bits; bf16 results and the ReLU are
    those of the same sums."""
    torch, sffn = need_gpu()
    G = -(-K // 32)
    gen = torch.Generator(device="cuda").manual_seed(N + K + T)
    codes = torch.randint(0, 256, (N, 16 * G), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 124, (N, G), generator=gen, device="cuda", dtype=torch.uint8)
    x = torch.randn((T, K), generator=gen, device="cuda")
    sc = None
    if kind == "fp8":
        sc = x.abs().amax(1) / 448
        x = x / sc[:, None]
    x = x.to({"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[kind])
    bias = torch.randn(N, generator=gen, device="cuda")
    lin = sffn.Mx4Linear(codes, scales, bias=bias, in_features=K)
    y = lin(x, x_scale=sc, dtype=torch.float32)
    x64, s64 = x.float().double(), 1.0 if sc is None else sc.double()[:, None]
    step = max(1, (1 << 27) // K)
    for i in range(0, N, step):
        W = _decode_on_gpu(torch, codes[i:i + step], scales[i:i + step], K)
        b = bias[i:i + step].double()
        z = (x64 @ W.t()) * s64 + b
        size = (x64.abs() @ W.abs().t()) * s64 + b.abs()
        off = (y[:, i:i + step].double() - z).abs()
        assert bool((off <= (K + 20) * 2.0 ** -23 * size + 1e-30).all()), (i, float((off / size).max()))
        del W, z, size, off
    assert torch.equal(lin(x, x_scale=sc, dtype=torch.bfloat16), y.to(torch.bfloat16))
    lin.relu = True
    assert torch.equal(lin(x, x_scale=sc, dtype=torch.float32), y.clamp_min(0))


@pytest.mark.parametrize("T,N,K,kind", [(7, 8192, 2048, "fp8"), (64, 9216, 2304, "fp8"), (48, 8192, 2048, "bf16"),
                                        (16, 6144, 1536, "f32"), (33, 2048, 512, "f32")])
def test_one_token_alone_and_among_others(T, N, K, kind):
    """A token's result alone and in a batch: both within the bound of a product from the exact one,
    element by element, so within twice that of each other."""
    torch, sffn = need_gpu()
    rng = np.random.default_rng(T + N)
    codes, scales = _weights(rng, N, K)
    x, sc = _tokens(torch, rng, T, K, kind)
    lin = sffn.Mx4Linear(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    y = lin(x, x_scale=sc, dtype=torch.float32).cpu().double().numpy()
    size = np.abs(x.float().cpu().double().numpy()) @ np.abs(_decode(codes, scales, K)).T
    if sc is not None:
        size = size * sc.cpu().double().numpy()[:, None]
    for t in (0, T // 2, T - 1):
        one = lin(x[t:t + 1], x_scale=None if sc is None else sc[t:t + 1], dtype=torch.float32)
        off = np.abs(one.cpu().double().numpy()[0] - y[t])
        assert np.all(off <= 2 * ((K + 20) * 2.0 ** -23 * size[t] + 1e-30))


@pytest.mark.parametrize("T", [2, 20])
@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
def test_every_scale(T, kind):
    """Every code under every scale, times a token value that brings the product into fp32's range: the
    exact product, down to the smallest (subnormal) weights.  Weights of 2^128 and more (scales 253 and
    254) are beyond fp32's range, and their rows not finite."""
    torch, sffn = need_gpu()
    K, N = 32, 16 * 255
    codes = np.zeros((N, K // 2), np.uint8)
    codes[:, 0] = np.arange(N) % 16
    s = np.arange(N) // 16
    lin = sffn.Mx4Linear(torch.from_numpy(codes).cuda(), torch.from_numpy(s.astype(np.uint8)[:, None]).cuda())
    w = np.ldexp(E2M1[codes[:, 0]], s - 127)
    for power, rows in ((60, s <= 150), (-60, s >= 100)):
        x = torch.zeros((T, K), device="cuda")
        sc = None
        x[:, 0] = 2.0 ** power
        if kind == "fp8":  # the token's scale brings it
            x[:, 0] = 1.0
            sc = torch.full((T,), 2.0 ** power, device="cuda")
        x = x.to({"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[kind])
        y = lin(x, x_scale=sc, dtype=torch.float32).cpu().double().numpy()
        want = np.ldexp(w, power)
        if kind == "fp8":  # the sum before the token's scale is fp32 too
            rows = rows & (np.abs(w) >= 2.0 ** -126) | rows & (w == 0)
        fits = np.abs(w) < 2.0 ** 128
        assert np.array_equal(y[:, rows & fits], np.broadcast_to(want, y.shape)[:, rows & fits])
        assert not np.isfinite(y[:, ~fits]).any()
