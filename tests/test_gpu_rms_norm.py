"""GPU tests of the RMS norm (with the residual's sum, and with its output in 8 bits) and of its
gradient, against the formulas in 64 bits on the host.

Tolerances, with u = 2^-24 (one fp32 rounding):
  rstd    the sum of squares adds each term at most S = 8 * 8 + 6 + 16 times (a lane's vectors,
          the lanes, the waves): relative error at most (S + 8) u, with the divide and root
  y, q    that of rstd and three products; a bf16 y is the rounding of such a value; e4m3: 2^-4
          of the value or, below its normal range, 2^-10 of the scale
  dx      terms t and xh c with relative errors of a few u on each, c's sum as above on the
          absolute values; a bf16 dx is the rounding of such a value
  dgain   at most rows + 64 additions: (rows + 64) u of the sum of absolute values"""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.ops_helpers import rounded_from

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
S = 8 * 8 + 6 + 16
# lengths around the vectors (8), the lane groups (128, 256, 512), the waves' registers (4096,
# 16384) and the longest row
LENGTHS = [1, 7, 8, 9, 127, 128, 129, 256, 257, 512, 513, 1537, 2048, 2304, 4096, 4097, 6145, 16384,
           16385, 32768]


def _rows(torch, rows, d, dtype, seed, pad=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = scale * torch.randn((rows, d + pad), generator=g)
    return t.to(dtype).cuda()[:, :d]


def _f64(t):
    return t.detach().cpu().double().numpy()


def _dt(torch, name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _reference(x, res, gain, eps):
    h = x if res is None else x + res
    rstd = 1 / np.sqrt((h * h).mean(axis=1) + eps)
    return h, rstd, h * rstd[:, None] * gain


def _check_norm(torch, sffn, x, res, gain, dtype, eps=1e-6):
    h64, r64, y64 = _reference(_f64(x), None if res is None else _f64(res), _f64(gain), eps)
    y, h, rstd = sffn.rms_norm(x, gain, residual=res, eps=eps)
    rel = (S + 8) * U
    assert np.all(np.abs(_f64(rstd) - r64) <= rel * r64)
    bf16 = dtype == "bf16"
    assert np.all(rounded_from(_f64(y), y64, (rel + 5 * U) * np.abs(y64) + 1e-37, bf16))
    if res is None:
        assert h is x
    else:
        assert np.all(rounded_from(_f64(h), h64, 2 * U * np.abs(h64) + 1e-37, bf16))
    q, scale, h2 = sffn.rms_norm_fp8(x, gain, residual=res, eps=eps)
    s64 = np.maximum(np.abs(y64).max(axis=1) / 448, 2.0 ** -126)
    s = _f64(scale)
    assert np.all(np.abs(s - s64) <= (rel + 6 * U) * s64)
    v = _f64(q.float()) * s[:, None]
    assert np.all(np.abs(v - y64) <= (2.0 ** -4 + 2 * rel) * np.abs(y64) + 2.0 ** -10 * s[:, None])
    if res is not None:
        assert torch.equal(h2, h)
    return y, h, rstd, q, scale


@pytest.mark.parametrize("d", LENGTHS)
@pytest.mark.parametrize("dtype,gain_f32", [("bf16", False), ("bf16", True), ("f32", True)])
def test_norm_lengths(d, dtype, gain_f32):
    torch, sffn = need_gpu()
    dt = _dt(torch, dtype)
    gain = (1 + 0.1 * _rows(torch, 1, d, torch.float32, 9)[0]).to(torch.float32 if gain_f32 else dt)
    for rows, pad, with_res in ((1, 0, True), (5, 3, False), (3, 8, True)):
        x = _rows(torch, rows, d, dt, 1, pad)
        res = _rows(torch, rows, d, dt, 2, 0 if pad else 5, 2.0) if with_res else None
        _check_norm(torch, sffn, x, res, gain.contiguous(), dtype)


@pytest.mark.parametrize("rows,d", [(1023, 2048), (1024, 2048), (1025, 2304), (2000, 1537), (4099, 64),
                                    (1030, 4096), (1100, 72)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_many_rows(rows, d, dtype):
    torch, sffn = need_gpu()
    dt = _dt(torch, dtype)
    x, res = _rows(torch, rows, d, dt, 3), _rows(torch, rows, d, dt, 4, 0, 3.0)
    gain = (1 + 0.1 * _rows(torch, 1, d, dt, 5)[0]).contiguous()
    _check_norm(torch, sffn, x, res, gain, dtype)


def test_norm_special_rows():
    """Rows of zeros, of one value, tiny and large values, an infinity and a NaN: the other rows
    are untouched, and the special ones follow the formula."""
    torch, sffn = need_gpu()
    d = 300
    for dt in (torch.float32, torch.bfloat16):
        x = _rows(torch, 9, d, dt, 1)
        x[1] = 0
        x[2, 5] = float("inf")
        x[3, 299] = float("nan")
        x[4] *= 1e-30
        x[5] *= 1e15
        x[7] = 0
        x[7, 0] = 3
        gain = torch.ones(d, dtype=dt, device="cuda")
        y, h, rstd = sffn.rms_norm(x, gain, eps=1e-6)
        q, s, _ = sffn.rms_norm_fp8(x, gain, eps=1e-6)
        xf = x.float()
        ref = xf * (1 / torch.sqrt(xf.square().mean(1, keepdim=True) + 1e-6))
        good = [0, 1, 4, 5, 6, 7, 8]
        assert torch.isfinite(y[good].float()).all()
        assert torch.allclose(y[good].float(), ref[good], rtol=2.0 ** -8, atol=0)
        assert (y[1] == 0).all() and (q[1].float() == 0).all() and s[1] == 2.0 ** -126
        assert torch.isnan(y[2, 5]) and (y[2, :5] == 0).all() and rstd[2] == 0
        assert torch.isnan(y[3].float()).all() and torch.isnan(rstd[3])
        assert torch.isnan(s[2]) and torch.isnan(s[3])
        assert (q[7].float()[0] == 448) and (q[7].float()[1:] == 0).all()
        for r in good:
            assert torch.isfinite(q[r].float()).all() and torch.isfinite(s[r])
    # eps = 0 on a row of zeros: 0 * inf
    z = torch.zeros((2, 40), device="cuda")
    y, _, rstd = sffn.rms_norm(z, torch.ones(40, device="cuda"), eps=0.0)
    assert torch.isnan(y).all() and torch.isinf(rstd).all()


def test_norm_in_place_and_given_outputs():
    torch, sffn = need_gpu()
    x, res = _rows(torch, 70, 513, torch.bfloat16, 1), _rows(torch, 70, 513, torch.bfloat16, 2)
    gain = torch.ones(513, dtype=torch.bfloat16, device="cuda")
    y0, h0, r0 = sffn.rms_norm(x, gain, residual=res)
    stream = res.clone()
    y, rstd = torch.empty_like(x), torch.empty(70, device="cuda")
    a, b, c = sffn.rms_norm(x, gain, residual=stream, h=stream, y=y, rstd=rstd)
    assert a is y and b is stream and c is rstd
    assert torch.equal(y, y0) and torch.equal(stream, h0) and torch.equal(rstd, r0)
    own = x.clone()
    _, h, _ = sffn.rms_norm(own, gain, residual=res, h=own)
    assert h is own and torch.equal(own, h0)


def test_norm_more_rows_than_one_launch_takes():
    torch, sffn = need_gpu()
    rows = (1 << 21) + 37
    x = torch.randn((rows, 8), device="cuda").to(torch.bfloat16)
    gain = torch.ones(8, dtype=torch.bfloat16, device="cuda")
    y, h, rstd = sffn.rms_norm(x, gain, residual=x)
    for at in (slice(0, 64), slice((1 << 21) - 40, (1 << 21) + 37)):
        part = x[at].contiguous()
        y2, h2, r2 = sffn.rms_norm(part, gain, residual=part)
        assert torch.equal(y[at], y2) and torch.equal(h[at], h2) and torch.equal(rstd[at], r2)
    q, s, _ = sffn.rms_norm_fp8(x, gain)
    q2, s2, _ = sffn.rms_norm_fp8(x[-50:].contiguous(), gain)
    assert torch.equal(q[-50:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-50:], s2)


def test_norm_unaligned_and_repeatable():
    """Rows that start one element past an aligned address give the same bits."""
    torch, sffn = need_gpu()
    for dt in (torch.bfloat16, torch.float32):
        base = _rows(torch, 1, 4 * 777 + 1, dt, 3)[0]
        x = base[1:].view(4, 777)
        gain_base = _rows(torch, 1, 778, dt, 4)[0]
        gain = gain_base[1:]
        y, _, r = sffn.rms_norm(x, gain)
        y2, _, r2 = sffn.rms_norm(x.clone(), gain.clone())
        assert torch.equal(y, y2) and torch.equal(r, r2)
        q, s, _ = sffn.rms_norm_fp8(x, gain)
        q2, s2, _ = sffn.rms_norm_fp8(x.clone(), gain.clone())
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


def test_norm_offsets_beyond_32_bits():
    torch, sffn = need_gpu()
    stride = (1 << 31) + 24
    big = torch.zeros(stride + 264, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, 264), (stride, 1))
    rows = _rows(torch, 2, 264, torch.bfloat16, 1)
    x.copy_(rows)
    gain = torch.ones(264, dtype=torch.bfloat16, device="cuda")
    y, _, r = sffn.rms_norm(x, gain)
    y2, _, r2 = sffn.rms_norm(rows, gain)
    assert torch.equal(y, y2) and torch.equal(r, r2)
    dx, dg = sffn.rms_norm_backward(y, x, gain, r)
    dx2, dg2 = sffn.rms_norm_backward(y2, rows, gain, r2)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)


def test_norm_no_rows():
    torch, sffn = need_gpu()
    x = torch.empty((0, 64), device="cuda")
    gain = torch.ones(64, device="cuda")
    y, h, rstd = sffn.rms_norm(x, gain, residual=x)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    q, s, _ = sffn.rms_norm_fp8(x, gain)
    assert q.shape == (0, 64) and s.shape == (0,)
    dgain = torch.full((64,), 7.0, device="cuda")
    dx, dg = sffn.rms_norm_backward(x, x, gain, rstd, dgain=dgain)
    assert dx.shape == (0, 64) and dg is dgain and (dg == 0).all()


def test_norm_on_another_stream():
    torch, sffn = need_gpu()
    x = _rows(torch, 300, 2048, torch.bfloat16, 1)
    gain = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    y0, h0, r0 = sffn.rms_norm(x, gain, residual=x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, r = sffn.rms_norm(x, gain, residual=x, stream=side)
    dx, dg = sffn.rms_norm_backward(y, h, gain, r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    dx0, dg0 = sffn.rms_norm_backward(y0, h0, gain, r0)
    assert torch.equal(y, y0) and torch.equal(h, h0) and torch.equal(r, r0)
    assert torch.equal(dx, dx0) and torch.equal(dg, dg0)


# ------------------------------------------------------------------ gradient

def _grad_reference(dy, h, gain, rstd, dres):
    xh = h * rstd[:, None]
    t = dy * gain
    c = (t * xh).mean(axis=1, keepdims=True)
    dx = rstd[:, None] * (t - xh * c)
    size = np.abs(rstd[:, None]) * (np.abs(t) + np.abs(xh) * np.abs(t * xh).mean(axis=1, keepdims=True))
    if dres is not None:
        dx = dx + dres
        size = size + np.abs(dres)
    return dx, size, (dy * xh).sum(axis=0), np.abs(dy * xh).sum(axis=0)


def _check_grad(torch, sffn, rows, d, dtype, gain_f32=True, with_dres=True, pad=0):
    dt = _dt(torch, dtype)
    h, dy = _rows(torch, rows, d, dt, 1, pad, 2.0), _rows(torch, rows, d, dt, 2)
    dres = _rows(torch, rows, d, dt, 3, pad) if with_dres else None
    gain = (1 + 0.1 * _rows(torch, 1, d, torch.float32, 4)[0]).to(torch.float32 if gain_f32 else dt)
    gain = gain.contiguous()
    rstd = (1 / torch.sqrt(h.float().square().mean(1) + 1e-6)).contiguous()
    dx, dg = sffn.rms_norm_backward(dy, h, gain, rstd, dres=dres)
    dx64, size, dg64, dgsize = _grad_reference(_f64(dy), _f64(h), _f64(gain), _f64(rstd),
                                               None if dres is None else _f64(dres))
    assert dg.dtype == torch.float32 and dx.dtype == dt
    assert np.all(rounded_from(_f64(dx), dx64, (S + 11) * U * size + 1e-37, dtype == "bf16"))
    assert np.all(np.abs(_f64(dg) - dg64) <= (rows + 64) * U * dgsize + 1e-37)
    return dx, dg, (dy, h, gain, rstd, dres)


@pytest.mark.parametrize("d", LENGTHS)
@pytest.mark.parametrize("dtype,gain_f32", [("bf16", False), ("bf16", True), ("f32", True)])
def test_grad_lengths(d, dtype, gain_f32):
    torch, sffn = need_gpu()
    for rows, with_dres, pad in ((1, True, 0), (6, False, 3), (37, True, 8)):
        _check_grad(torch, sffn, rows, d, dtype, gain_f32, with_dres, pad)


@pytest.mark.parametrize("rows,d", [(1024, 2048), (5003, 2304), (1500, 1537), (20000, 64), (4100, 200),
                                    (3001, 2560), (1025, 2561), (300, 20000), (1024, 1024), (1024, 1025),
                                    (1000, 67)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grad_many_rows(rows, d, dtype):
    torch, sffn = need_gpu()
    dx, dg, (dy, h, gain, rstd, dres) = _check_grad(torch, sffn, rows, d, dtype, dtype == "f32")
    dx2, dg2 = sffn.rms_norm_backward(dy, h, gain, rstd, dres=dres)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)  # the order of the sums is fixed
    own = dres.clone()
    dx3, none = sffn.rms_norm_backward(dy, h, gain, rstd, dres=own, dx=own, with_dgain=False)
    assert none is None and dx3 is own and torch.equal(own, dx)


@pytest.mark.parametrize("d", [5, 64, 520])
def test_grad_against_differences(d):
    """The gradient is the derivative: central differences in 64 bits of
    L = sum(dy * y) + sum(dres * h) over x, the residual and the gain."""
    torch, sffn = need_gpu()
    rows, eps = 3, 1e-3
    rng = np.random.default_rng(d)
    x, res, dy, dres = (rng.standard_normal((rows, d)).astype(np.float32) for _ in range(4))
    gain = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)

    def loss(x_, g_):
        h, _, y = _reference(x_, res.astype(np.float64), g_, eps)
        return (dy * y).sum() + (dres * h).sum()

    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    y, h, rstd = sffn.rms_norm(to(x), to(gain), residual=to(res), eps=eps)
    dx, dg = sffn.rms_norm_backward(to(dy), h, to(gain), rstd, dres=to(dres))
    x64, g64, step = x.astype(np.float64), gain.astype(np.float64), 1e-5
    for i, j in [(0, 0), (1, d // 2), (2, d - 1)]:
        e = np.zeros_like(x64)
        e[i, j] = step
        num = (loss(x64 + e, g64) - loss(x64 - e, g64)) / (2 * step)
        # differences: 1e-10 of third derivatives of order 10 and 1e-16 / 1e-5 of a loss of order
        # 100; the kernel: some 100 roundings of terms of order 10
        assert abs(float(dx[i, j]) - num) <= 1e-4
        e = np.zeros_like(g64)
        e[j] = step
        num = (loss(x64, g64 + e) - loss(x64, g64 - e)) / (2 * step)
        assert abs(float(dg[j]) - num) <= 1e-4


def test_grad_special_rows():
    """A row whose gradient is not finite spoils its own dx and the columns of dgain it reaches,
    no other row."""
    torch, sffn = need_gpu()
    h, dy = _rows(torch, 8, 200, torch.float32, 1), _rows(torch, 8, 200, torch.float32, 2)
    gain = torch.ones(200, device="cuda")
    rstd = 1 / torch.sqrt(h.square().mean(1) + 1e-6)
    clean, dgc = sffn.rms_norm_backward(dy, h, gain, rstd)
    dy[3, 7] = float("nan")
    dx, dg = sffn.rms_norm_backward(dy, h, gain, rstd)
    rest = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(dx[rest], clean[rest]) and torch.isnan(dx[3]).all()
    cols = [c for c in range(200) if c != 7]
    assert torch.isnan(dg[7]) and torch.equal(dg[cols], dgc[cols])
    zero = torch.zeros_like(h)
    dz, dgz = sffn.rms_norm_backward(zero, zero, gain, torch.full((8,), 1e3, device="cuda"))
    assert (dz == 0).all() and (dgz == 0).all()


def test_norm_refusals():
    torch, sffn = need_gpu()
    x = torch.zeros((4, 64), device="cuda")
    gain = torch.ones(64, device="cuda")
    y, h, rstd = sffn.rms_norm(x, gain)
    bad = [
        lambda: sffn.rms_norm(x.half(), gain),
        lambda: sffn.rms_norm(x.cpu(), gain),
        lambda: sffn.rms_norm(x.t(), gain),
        lambda: sffn.rms_norm(x, gain[:32]),
        lambda: sffn.rms_norm(x, gain.bfloat16()),
        lambda: sffn.rms_norm(x, gain, residual=x[:2]),
        lambda: sffn.rms_norm(x, gain, residual=x.bfloat16()),
        lambda: sffn.rms_norm(x, gain, h=x),
        lambda: sffn.rms_norm(x, gain, y=x[:, :32]),
        lambda: sffn.rms_norm(x[0].expand(4, 64), gain),
        lambda: sffn.rms_norm_backward(x, x, gain, rstd[:2]),
        lambda: sffn.rms_norm_backward(x.bfloat16(), x, gain, rstd),
        lambda: sffn.rms_norm_backward(x, x, gain, rstd, dres=x[:1]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(sffn.SffnError) as ei:
        sffn.rms_norm(x, gain, eps=-1.0)
    assert ei.value.status == sffn.SFFN_ERR_INVALID_ARGUMENT
    wide = torch.zeros((1, 32769), device="cuda")
    with pytest.raises(sffn.SffnError) as ei:
        sffn.rms_norm(wide, torch.ones(32769, device="cuda"))
    assert ei.value.status == sffn.SFFN_ERR_UNSUPPORTED


# ------------------------------------------------------------------ 8-bit codes

def _midpoints():
    """The values half way between neighbours of e4m3 from 2^-6 to 448, as float32."""
    v = np.array([(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1])  # (the last one is NaN)
    return ((v[1:] + v[:-1]) / 2).astype(np.float32)


@pytest.mark.parametrize("size", [1.0, 2.0 ** -110, 2.0 ** -122, 2.0 ** 100])
def test_fp8_codes_are_of_the_quotient(size):
    """q = e4m3(y / scale) with the quotient in fp32, no reciprocal in its place: values of y within
    a few roundings of the middle between two codes take the code of the quotient.  The gain
    brings every column there without a change to the row's statistics."""
    torch, sffn = need_gpu()
    d = 32768
    rng = np.random.default_rng(11)
    x = (0.5 + rng.random((1, d))).astype(np.float32)
    x[0, 0] = 300
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    y0 = sffn.rms_norm(to(x), torch.ones(d, device="cuda"))[0].cpu().numpy()[0]
    top = np.float32(y0[0] * np.float32(size))
    s = max(top / np.float32(448), np.float32(2.0 ** -126))
    # in double; the sizes are powers of two, so only y0's own digits round here
    gain = (rng.choice(_midpoints(), d).astype(np.float64) * float(s) / y0).astype(np.float32)
    gain[0] = size
    y = sffn.rms_norm(to(x), to(gain))[0].cpu().numpy()
    q, scale, _ = sffn.rms_norm_fp8(to(x), to(gain))
    assert scale.cpu().numpy()[0] == s and np.abs(y).max() == y[0, 0]
    codes = lambda v: torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()  # noqa: E731
    want = codes(y / s)
    if size == 1.0:  # the inputs tell the two apart
        assert (codes(y * (np.float32(1) / s)) != want).any()
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want)


# ------------------------------------------------------------------ overlap

@pytest.mark.parametrize("d", [100, 513, 2304, 5000])
def test_norm_output_in_place_and_between_rows(d):
    """y in place of x or the residual gives the same bits, and so does an output that lies in the
    gap between strided rows; outputs over parts of inputs are refused."""
    torch, sffn = need_gpu()
    dt = torch.bfloat16
    x, res = _rows(torch, 21, d, dt, 1), _rows(torch, 21, d, dt, 2)
    gain = (1 + 0.1 * _rows(torch, 1, d, dt, 5)[0]).contiguous()
    y0, h0, r0 = sffn.rms_norm(x, gain, residual=res)
    a, b = x.clone(), res.clone()
    y, h, r = sffn.rms_norm(a, gain, residual=b, y=a, h=b)
    assert y is a and h is b and torch.equal(a, y0) and torch.equal(b, h0) and torch.equal(r, r0)
    a, b = x.clone(), res.clone()
    sffn.rms_norm(a, gain, residual=b, y=b, h=a)
    assert torch.equal(b, y0) and torch.equal(a, h0)
    wide = torch.zeros((2, 30 * d), dtype=dt, device="cuda")
    wide[:, :d] = x[:2]
    gap = wide[0, d + 1:3 * d + 1].view(2, d)
    y, _, _ = sffn.rms_norm(wide[:, :d], gain, residual=res[:2].contiguous(), y=gap)
    assert torch.equal(gap, y0[:2]) and torch.equal(wide[:, :d], x[:2])
    flat = torch.zeros(4 * d + 2, dtype=dt, device="cuda")
    two = flat[:2 * d].view(2, d)
    for bad in (lambda: sffn.rms_norm(two, gain, y=flat[2:2 * d + 2].view(2, d)),
                lambda: sffn.rms_norm(wide[:, :d], gain, y=wide[0, :2 * d].view(2, d)),
                lambda: sffn.rms_norm(two, gain, residual=two.clone(), y=flat[2 * d:4 * d].view(2, d),
                                      h=flat[2 * d:4 * d].view(2, d)),
                lambda: sffn.rms_norm_backward(x, h0, gain, r0, dx=x),
                lambda: sffn.rms_norm_backward(x, h0, gain, r0, dres=x, dx=x),
                lambda: sffn.rms_norm_backward(x, h0, gain, r0, dx=h0)):
        with pytest.raises(sffn.SffnError) as ei:
            bad()
        assert ei.value.status == sffn.SFFN_ERR_INVALID_ARGUMENT
