"""GPU tests of the layer norm (with the residual's sum, and with its output in 8 bits) and of its
gradient, against the formulas in 64 bits on the host.

Tolerances, with u = 2^-24 (one fp32 rounding), D = h - mean(h) and S = 8 * 8 + 6 + 16, the most
additions that a term of a row's sum goes through (a lane's vectors, the lanes, the waves):
  D       the sum with a residual is off by u |h|, and so its mean by u mean|h|; a deviation is
          rounded, their own mean (off by (S + 2) u mean|D|) is taken from it, and that is rounded
  mean    as D's last two, and its own rounding
  rstd    the variance is off by (S + 6) u of itself and, with a residual, by 2 u mean(|D| (|h| +
          mean|h|)); half of that, relative to var + eps, and the divide and root
  y, q    those of D and rstd, three products and a sum; a bf16 y is the rounding of such a value;
          e4m3: 2^-4 of the value or, below its normal range, 2^-10 of the scale
  dx      t, mean(t) and xh mean(t xh) with relative errors of a few u on each and (S + 6) u on the
          means' absolute terms; a bf16 dx is the rounding of such a value
  dgain, dbias  at most rows + 64 additions of terms off by 4 u: (rows + 68) u of the absolute sum"""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.layer_norm_shapes import SIZES
from tests.ops_helpers import rounded_from

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
S = 8 * 8 + 6 + 16
# lengths around the vectors (8), the lane groups (128, 256, 512), the waves' registers (4096,
# 16384) and the longest row
LENGTHS = [1, 2, 7, 8, 9, 127, 128, 129, 256, 257, 512, 513, 1537, 2048, 2304, 4096, 4097, 6145, 16384,
           16385, 32768]


def _rows(torch, rows, d, dtype, seed, pad=0, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    t = scale * torch.randn((rows, d + pad), generator=g)
    t += shift * torch.randn((rows, 1), generator=g)
    return t.to(dtype).cuda()[:, :d]


def _f64(t):
    return t.detach().cpu().double().numpy()


def _dt(torch, name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _reference(x, res, gain, bias, eps):
    h = x if res is None else x + res
    mean = h.mean(axis=1, keepdims=True)
    D = h - mean
    rstd = 1 / np.sqrt((D * D).mean(axis=1, keepdims=True) + eps)
    return h, mean, D, rstd, D * rstd * gain + bias


def _check_norm(torch, sffn, x, res, gain, bias, dtype, eps=1e-5):
    b64 = 0.0 if bias is None else _f64(bias)
    g64 = _f64(gain)
    h64, m64, D, r64, y64 = _reference(_f64(x), None if res is None else _f64(res), g64, b64, eps)
    y, h, mean, rstd = sffn.layer_norm(x, gain, bias=bias, residual=res, eps=eps)
    size, spread = np.abs(h64).mean(axis=1, keepdims=True), np.abs(D).mean(axis=1, keepdims=True)
    from_res = U * (np.abs(h64) + size) if res is not None else 0 * h64
    tiny = 1e-37
    tol_d = from_res + U * (2 * np.abs(D) + (S + 3) * spread)
    tol_m = (U * size if res is not None else 0) + U * ((S + 3) * spread + np.abs(m64)) + tiny
    var = (D * D).mean(axis=1, keepdims=True)
    rel_r = ((S + 6) * U * var + 2 * (np.abs(D) * from_res).mean(axis=1, keepdims=True)) / (2 * (var + eps)) + 4 * U
    tol_y = np.abs(g64) * r64 * (tol_d + np.abs(D) * (rel_r + 4 * U)) * (1 + 1e-4) + U * np.abs(y64) + tiny
    assert np.all(np.abs(_f64(mean)[:, None] - m64) <= tol_m)
    assert np.all(np.abs(_f64(rstd)[:, None] - r64) <= rel_r * (1 + 1e-4) * r64)
    bf16 = dtype == "bf16"
    assert np.all(rounded_from(_f64(y), y64, tol_y, bf16))
    if res is None:
        assert h is x
    else:
        assert np.all(rounded_from(_f64(h), h64, 2 * U * np.abs(h64) + tiny, bf16))
    q, scale, h2 = sffn.layer_norm_fp8(x, gain, bias=bias, residual=res, eps=eps)
    s64 = np.maximum(np.abs(y64).max(axis=1) / 448, 2.0 ** -126)
    s = _f64(scale)
    assert np.all(np.abs(s - s64) <= tol_y.max(axis=1) / 448 + 3 * U * s64)
    v = _f64(q.float()) * s[:, None]
    assert np.all(np.abs(v - y64) <= (2.0 ** -4 + 4 * U) * (np.abs(y64) + tol_y) + 2.0 ** -10 * s[:, None] + tol_y)
    if res is not None:
        assert torch.equal(h2, h)
    return y, h, mean, rstd, q, scale


def _params(torch, d, dt, gain_f32=False):
    t = torch.float32 if gain_f32 else dt
    gain = (1 + 0.1 * _rows(torch, 1, d, torch.float32, 9)[0]).to(t).contiguous()
    return gain, (0.3 * _rows(torch, 1, d, torch.float32, 8)[0]).to(t).contiguous()


@pytest.mark.parametrize("d", LENGTHS)
@pytest.mark.parametrize("dtype,gain_f32", [("bf16", False), ("bf16", True), ("f32", True)])
def test_norm_lengths(d, dtype, gain_f32):
    torch, sffn = need_gpu()
    dt = _dt(torch, dtype)
    gain, bias = _params(torch, d, dt, gain_f32)
    for rows, pad, with_res, with_bias in ((1, 0, True, True), (5, 3, False, True), (3, 8, True, False)):
        x = _rows(torch, rows, d, dt, 1, pad, shift=1.0)
        res = _rows(torch, rows, d, dt, 2, 0 if pad else 5, 2.0) if with_res else None
        _check_norm(torch, sffn, x, res, gain, bias if with_bias else None, dtype)


@pytest.mark.parametrize("rows,d", [(1023, 2048), (1025, 2304), (2000, 1537), (4099, 64), (1030, 4096), (1100, 72)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_many_rows(rows, d, dtype):
    torch, sffn = need_gpu()
    dt = _dt(torch, dtype)
    x, res = _rows(torch, rows, d, dt, 3), _rows(torch, rows, d, dt, 4, 0, 3.0)
    gain, bias = _params(torch, d, dt)
    _check_norm(torch, sffn, x, res, gain, bias, dtype)


@pytest.mark.parametrize("shift", [30.0, 1e3, 1e5])
@pytest.mark.parametrize("d", [100, 2304, 9000, 20000])
def test_norm_of_rows_far_from_zero(shift, d):
    """A mean many times the deviations costs no digits of them: without a residual the bounds above
    know only the deviations."""
    torch, sffn = need_gpu()
    x = _rows(torch, 6, d, torch.float32, 5, shift=shift)
    gain, bias = _params(torch, d, torch.float32)
    _check_norm(torch, sffn, x, None, gain, bias, "f32")


@pytest.mark.parametrize("d", [40, 300, 2304, 20000])
def test_fp8_codes_are_of_the_quotient(d):
    """q = e4m3(y / scale), the quotient in fp32 of the y that the same call gives in fp32."""
    torch, sffn = need_gpu()
    x = _rows(torch, 50, d, torch.float32, 3, shift=2.0)
    x[7] *= 1e-35
    x[8] = 0
    gain, bias = _params(torch, d, torch.float32)
    for b in (bias, None, 1e-37 * bias):
        y = sffn.layer_norm(x, gain, bias=b)[0].cpu()
        q, scale, _ = sffn.layer_norm_fp8(x, gain, bias=b)
        s = (y.abs().amax(1) / 448).clamp_min(2.0 ** -126)
        assert torch.equal(scale.cpu(), s)
        assert torch.equal(q.cpu().view(torch.uint8) & 127, (y / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8) & 127)


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
        x[7] = 3
        gain, bias = _params(torch, d, dt)
        y, h, mean, rstd = sffn.layer_norm(x, gain, bias=bias)
        q, s, _ = sffn.layer_norm_fp8(x, gain, bias=bias)
        good = [0, 1, 4, 5, 6, 7, 8]
        ref = _reference(_f64(x[good]), None, _f64(gain), _f64(bias), 1e-5)[4]
        assert torch.isfinite(y[good].float()).all()
        assert np.allclose(_f64(y)[good], ref, rtol=2.0 ** -8 + 1e-4, atol=1e-5)
        for r in (1, 7):  # no deviations: the bias
            assert torch.equal(y[r], bias) and rstd[r] == rstd[1]
        assert mean[1] == 0 and mean[7] == 3
        assert torch.isnan(y[2].float()).all() and torch.isnan(rstd[2])
        assert torch.isnan(y[3].float()).all() and torch.isnan(rstd[3])
        assert torch.isnan(s[2]) and torch.isnan(s[3])
        for r in good:
            assert torch.isfinite(q[r].float()).all() and torch.isfinite(s[r])
        zero, sz, _ = sffn.layer_norm_fp8(x[1:2], gain)
        assert (zero.float() == 0).all() and sz[0] == 2.0 ** -126
    # eps = 0 on a row of zeros: 0 * inf
    z = torch.zeros((2, 40), device="cuda")
    y, _, _, rstd = sffn.layer_norm(z, torch.ones(40, device="cuda"), eps=0.0)
    assert torch.isnan(y).all() and torch.isinf(rstd).all()


@pytest.mark.parametrize("d", [100, 513, 2304, 5000])
def test_norm_in_place_and_given_outputs(d):
    torch, sffn = need_gpu()
    dt = torch.bfloat16
    x, res = _rows(torch, 70, d, dt, 1), _rows(torch, 70, d, dt, 2)
    gain, bias = _params(torch, d, dt)
    y0, h0, m0, r0 = sffn.layer_norm(x, gain, bias=bias, residual=res)
    stream = res.clone()
    y, mean, rstd = torch.empty_like(x), torch.empty(70, device="cuda"), torch.empty(70, device="cuda")
    a, b, c, e = sffn.layer_norm(x, gain, bias=bias, residual=stream, h=stream, y=y, mean=mean, rstd=rstd)
    assert a is y and b is stream and c is mean and e is rstd
    assert torch.equal(y, y0) and torch.equal(stream, h0) and torch.equal(mean, m0) and torch.equal(rstd, r0)
    a, b = x.clone(), res.clone()
    sffn.layer_norm(a, gain, bias=bias, residual=b, y=b, h=a)
    assert torch.equal(b, y0) and torch.equal(a, h0)
    q0, s0, _ = sffn.layer_norm_fp8(x, gain, bias=bias, residual=res)
    own, q, s = x.clone(), torch.empty((70, d), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(70, device="cuda")
    sffn.layer_norm_fp8(own, gain, bias=bias, residual=res, h=own, q=q, scale=s)
    assert torch.equal(own, h0) and torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)
    flat = torch.zeros(4 * d + 2, dtype=dt, device="cuda")
    two = flat[:2 * d].view(2, d)
    for bad in (lambda: sffn.layer_norm(two, gain, y=flat[2:2 * d + 2].view(2, d)),
                lambda: sffn.layer_norm(x, gain, bias=bias, mean=mean, rstd=mean),
                lambda: sffn.layer_norm(flat[:d].view(1, d), gain, bias=flat[d:2 * d], y=flat[d:2 * d].view(1, d)),
                lambda: sffn.layer_norm_backward(x, h0, gain, m0, r0, dx=x),
                lambda: sffn.layer_norm_backward(x, h0, gain, m0, r0, dx=h0)):
        with pytest.raises(sffn.SffnError) as ei:
            bad()
        assert ei.value.status == sffn.SFFN_ERR_INVALID_ARGUMENT


def test_norm_more_rows_than_one_launch_takes():
    torch, sffn = need_gpu()
    rows = (1 << 21) + 37
    x = torch.randn((rows, 8), device="cuda").to(torch.bfloat16)
    gain, bias = _params(torch, 8, torch.bfloat16)
    y, h, mean, rstd = sffn.layer_norm(x, gain, bias=bias, residual=x)
    for at in (slice(0, 64), slice((1 << 21) - 40, (1 << 21) + 37)):
        part = x[at].contiguous()
        other = sffn.layer_norm(part, gain, bias=bias, residual=part)
        assert all(torch.equal(a[at], b) for a, b in zip((y, h, mean, rstd), other))
    q, s, _ = sffn.layer_norm_fp8(x, gain)
    q2, s2, _ = sffn.layer_norm_fp8(x[-50:].contiguous(), gain)
    assert torch.equal(q[-50:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-50:], s2)


def test_norm_unaligned_and_repeatable():
    """Rows that start one element past an aligned address give the same bits."""
    torch, sffn = need_gpu()
    for dt in (torch.bfloat16, torch.float32):
        x = _rows(torch, 1, 4 * 777 + 1, dt, 3)[0][1:].view(4, 777)
        gain, bias = (_rows(torch, 1, 778, dt, k)[0][1:] for k in (4, 5))
        one = sffn.layer_norm(x, gain, bias=bias)
        two = sffn.layer_norm(x.clone(), gain.clone(), bias=bias.clone())
        assert all(torch.equal(a, b) for a, b in zip(one, two))
        q, s, _ = sffn.layer_norm_fp8(x, gain, bias=bias)
        q2, s2, _ = sffn.layer_norm_fp8(x.clone(), gain.clone(), bias=bias.clone())
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


def test_norm_offsets_beyond_32_bits():
    torch, sffn = need_gpu()
    stride = (1 << 31) + 24
    big = torch.zeros(stride + 264, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, 264), (stride, 1))
    rows = _rows(torch, 2, 264, torch.bfloat16, 1)
    x.copy_(rows)
    gain, bias = _params(torch, 264, torch.bfloat16)
    y, _, m, r = sffn.layer_norm(x, gain, bias=bias)
    y2, _, m2, r2 = sffn.layer_norm(rows, gain, bias=bias)
    assert torch.equal(y, y2) and torch.equal(m, m2) and torch.equal(r, r2)
    one = sffn.layer_norm_backward(y, x, gain, m, r)
    two = sffn.layer_norm_backward(y2, rows, gain, m2, r2)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_norm_no_rows():
    torch, sffn = need_gpu()
    x = torch.empty((0, 64), device="cuda")
    gain = torch.ones(64, device="cuda")
    y, h, mean, rstd = sffn.layer_norm(x, gain, residual=x)
    assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    q, s, _ = sffn.layer_norm_fp8(x, gain)
    assert q.shape == (0, 64) and s.shape == (0,)
    dgain, dbias = torch.full((64,), 7.0, device="cuda"), torch.full((64,), 7.0, device="cuda")
    dx, dg, db = sffn.layer_norm_backward(x, x, gain, mean, rstd, dgain=dgain, dbias=dbias)
    assert dx.shape == (0, 64) and dg is dgain and db is dbias and (dg == 0).all() and (db == 0).all()


def test_norm_on_another_stream():
    torch, sffn = need_gpu()
    x = _rows(torch, 1300, 2048, torch.bfloat16, 1)
    gain, bias = _params(torch, 2048, torch.bfloat16)
    first = sffn.layer_norm(x, gain, bias=bias, residual=x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = sffn.layer_norm(x, gain, bias=bias, residual=x, stream=side)
    y, h, m, r = again
    grads = sffn.layer_norm_backward(y, h, gain, m, r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    y, h, m, r = first
    grads0 = sffn.layer_norm_backward(y, h, gain, m, r)
    assert all(torch.equal(a, b) for a, b in zip(first + grads0, again + grads))


# ------------------------------------------------------------------ gradient

def _grad_reference(dy, h, gain, mean, rstd, dres):
    rstd = rstd[:, None]
    xh = (h - mean[:, None]) * rstd
    t = dy * gain
    mean_of = lambda a: a.mean(axis=1, keepdims=True)  # noqa: E731
    dx = rstd * (t - mean_of(t) - xh * mean_of(t * xh))
    size = np.abs(rstd) * (np.abs(t) + mean_of(np.abs(t)) + np.abs(xh) * mean_of(np.abs(t * xh)))
    if dres is not None:
        dx = dx + dres
        size = size + np.abs(dres)
    return dx, size, (dy * xh).sum(axis=0), np.abs(dy * xh).sum(axis=0), dy.sum(axis=0), np.abs(dy).sum(axis=0)


def _check_grad(torch, sffn, rows, d, dtype, gain_f32=True, with_dres=True, pad=0):
    dt = _dt(torch, dtype)
    h, dy = _rows(torch, rows, d, dt, 1, pad, 2.0, 1.0), _rows(torch, rows, d, dt, 2)
    dres = _rows(torch, rows, d, dt, 3, pad) if with_dres else None
    gain, _ = _params(torch, d, dt, gain_f32)
    h64 = h.double()
    mean = h64.mean(1).float()
    rstd = (1 / torch.sqrt(h64.var(1, unbiased=False) + 1e-5)).float()
    dx, dg, db = sffn.layer_norm_backward(dy, h, gain, mean, rstd, dres=dres)
    dx64, size, dg64, dgsize, db64, dbsize = _grad_reference(
        *(_f64(t) for t in (dy, h, gain, mean, rstd)), None if dres is None else _f64(dres))
    assert dg.dtype == db.dtype == torch.float32 and dx.dtype == dt
    assert np.all(rounded_from(_f64(dx), dx64, (S + 12) * U * size + 1e-37, dtype == "bf16"))
    assert np.all(np.abs(_f64(dg) - dg64) <= (rows + 68) * U * dgsize + 1e-37)
    assert np.all(np.abs(_f64(db) - db64) <= (rows + 68) * U * dbsize + 1e-37)
    return dx, dg, db, (dy, h, gain, mean, rstd, dres)


@pytest.mark.parametrize("d", LENGTHS)
@pytest.mark.parametrize("dtype,gain_f32", [("bf16", False), ("bf16", True), ("f32", True)])
def test_grad_lengths(d, dtype, gain_f32):
    torch, sffn = need_gpu()
    for rows, with_dres, pad in ((1, True, 0), (6, False, 3), (37, True, 8)):
        _check_grad(torch, sffn, rows, d, dtype, gain_f32, with_dres, pad)


# few and many rows, both sides of the rules by which registers or other workgroups sum the columns
@pytest.mark.parametrize("rows,d", [(1024, 2048), (5003, 2304), (1500, 1537), (20000, 64), (4100, 200), (3001, 2560),
                                    (1025, 2561), (300, 20000), (1024, 1024), (1024, 1025), (1000, 67), (70, 16384),
                                    (1100, 16385), (2500, 17000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grad_many_rows(rows, d, dtype):
    torch, sffn = need_gpu()
    dx, dg, db, (dy, h, gain, mean, rstd, dres) = _check_grad(torch, sffn, rows, d, dtype, dtype == "f32")
    dx2, dg2, db2 = sffn.layer_norm_backward(dy, h, gain, mean, rstd, dres=dres)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2) and torch.equal(db, db2)  # the order of the sums is fixed
    own = dres.clone()
    dx3, none, none2 = sffn.layer_norm_backward(dy, h, gain, mean, rstd, dres=own, dx=own, with_dgain=False, with_dbias=False)
    assert none is None and none2 is None and dx3 is own and torch.equal(own, dx)
    _, one, none = sffn.layer_norm_backward(dy, h, gain, mean, rstd, dres=dres, with_dbias=False)
    assert none is None and torch.equal(one, dg)
    _, none, one = sffn.layer_norm_backward(dy, h, gain, mean, rstd, dres=dres, with_dgain=False)
    assert none is None and torch.equal(one, db)


@pytest.mark.parametrize("many,few,d", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grad_every_form(many, few, d, dtype):
    """Every way in which the kernel shares rows and sums columns, each result against 64 bits."""
    torch, sffn = need_gpu()
    _check_grad(torch, sffn, many, d, dtype, dtype == "f32" or d % 2 == 0)
    _check_grad(torch, sffn, few, d, dtype, True, False, 5)


@pytest.mark.parametrize("d", [5, 64, 520])
def test_grad_against_differences(d):
    """The gradient is the derivative: central differences in 64 bits of
    L = sum(dy * y) + sum(dres * h) over x, the residual, the gain and the bias."""
    torch, sffn = need_gpu()
    rows, eps = 3, 1e-3
    rng = np.random.default_rng(d)
    x, res, dy, dres = (rng.standard_normal((rows, d)).astype(np.float32) for _ in range(4))
    gain, bias = ((k + 0.1 * rng.standard_normal(d)).astype(np.float32) for k in (1, 0))

    def loss(x_, g_, b_):
        h, _, _, _, y = _reference(x_, res.astype(np.float64), g_, b_, eps)
        return (dy * y).sum() + (dres * h).sum()

    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    y, h, mean, rstd = sffn.layer_norm(to(x), to(gain), bias=to(bias), residual=to(res), eps=eps)
    dx, dg, db = sffn.layer_norm_backward(to(dy), h, to(gain), mean, rstd, dres=to(dres))
    x64, g64, b64, step = x.astype(np.float64), gain.astype(np.float64), bias.astype(np.float64), 1e-5
    for i, j in [(0, 0), (1, d // 2), (2, d - 1)]:
        e = np.zeros_like(x64)
        e[i, j] = step
        num = (loss(x64 + e, g64, b64) - loss(x64 - e, g64, b64)) / (2 * step)
        # differences: 1e-10 of third derivatives of order 10 and 1e-16 / 1e-5 of a loss of order
        # 100; the kernel: some 100 roundings of terms of order 10
        assert abs(float(dx[i, j]) - num) <= 1e-4
        e = np.zeros_like(g64)
        e[j] = step
        num = (loss(x64, g64 + e, b64) - loss(x64, g64 - e, b64)) / (2 * step)
        assert abs(float(dg[j]) - num) <= 1e-4
        num = (loss(x64, g64, b64 + e) - loss(x64, g64, b64 - e)) / (2 * step)
        assert abs(float(db[j]) - num) <= 1e-4


@pytest.mark.parametrize("rows,d", [(8, 200), (1500, 1000)])
def test_grad_special_rows(rows, d):
    """A row whose gradient is not finite spoils its own dx and the columns it reaches, no other
    row; one whose statistics are not spoils every column of dgain and none of dbias."""
    torch, sffn = need_gpu()
    h, dy = _rows(torch, rows, d, torch.float32, 1), _rows(torch, rows, d, torch.float32, 2)
    gain = torch.ones(d, device="cuda")
    mean, rstd = h.mean(1), 1 / torch.sqrt(h.var(1, unbiased=False) + 1e-5)
    clean, dgc, dbc = sffn.layer_norm_backward(dy, h, gain, mean, rstd)
    rest = [r for r in range(rows) if r != 3]
    bad = dy.clone()
    bad[3, 7] = float("nan")
    dx, dg, db = sffn.layer_norm_backward(bad, h, gain, mean, rstd)
    assert torch.equal(dx[rest], clean[rest]) and torch.isnan(dx[3]).all()
    cols = [c for c in range(d) if c != 7]
    assert torch.isnan(dg[7]) and torch.equal(dg[cols], dgc[cols])
    assert torch.isnan(db[7]) and torch.equal(db[cols], dbc[cols])
    rstd[3] = float("inf")
    dx, dg, db = sffn.layer_norm_backward(dy, h, gain, mean, rstd)
    assert torch.equal(dx[rest], clean[rest]) and torch.isnan(dx[3]).all()
    assert not torch.isfinite(dg).any() and torch.equal(db, dbc)
    # far from zero and flat: the deviations of the elements that are there are small
    h[3], mean[3], rstd[3] = 1e38, 1e38, 300.0
    dx, dg, db = sffn.layer_norm_backward(dy, h, gain, mean, rstd)
    assert torch.isfinite(dx).all() and torch.isfinite(dg).all() and torch.equal(db, dbc)


def test_norm_refusals():
    torch, sffn = need_gpu()
    x = torch.zeros((4, 64), device="cuda")
    gain, bias = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    y, h, mean, rstd = sffn.layer_norm(x, gain, bias=bias)
    bad = [
        lambda: sffn.layer_norm(x.half(), gain),
        lambda: sffn.layer_norm(x.cpu(), gain),
        lambda: sffn.layer_norm(x.t(), gain),
        lambda: sffn.layer_norm(x, gain[:32]),
        lambda: sffn.layer_norm(x, gain.bfloat16()),
        lambda: sffn.layer_norm(x, gain, bias=bias.bfloat16()),
        lambda: sffn.layer_norm(x, gain, bias=bias[:32]),
        lambda: sffn.layer_norm(x, gain, bias=bias.cpu()),
        lambda: sffn.layer_norm(x, gain, residual=x[:2]),
        lambda: sffn.layer_norm(x, gain, residual=x.bfloat16()),
        lambda: sffn.layer_norm(x, gain, h=x),
        lambda: sffn.layer_norm(x, gain, y=x[:, :32]),
        lambda: sffn.layer_norm(x, gain, mean=mean[:3]),
        lambda: sffn.layer_norm(x[0].expand(4, 64), gain),
        lambda: sffn.layer_norm_fp8(x, gain, q=x),
        lambda: sffn.layer_norm_backward(x, x, gain, mean, rstd[:2]),
        lambda: sffn.layer_norm_backward(x, x, gain, mean.double(), rstd),
        lambda: sffn.layer_norm_backward(x.bfloat16(), x, gain, mean, rstd),
        lambda: sffn.layer_norm_backward(x, x, gain, mean, rstd, dres=x[:1]),
        lambda: sffn.layer_norm_backward(x, x, gain, mean, rstd, dbias=bias[:3]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(sffn.SffnError) as ei:
        sffn.layer_norm(x, gain, eps=-1.0)
    assert ei.value.status == sffn.SFFN_ERR_INVALID_ARGUMENT
    wide = torch.zeros((1, 32769), device="cuda")
    with pytest.raises(sffn.SffnError) as ei:
        sffn.layer_norm(wide, torch.ones(32769, device="cuda"))
    assert ei.value.status == sffn.SFFN_ERR_UNSUPPORTED


def test_norm_and_gradient_in_a_graph():
    """Forward and backward recorded in a HIP graph while their eager results live: replays on new
    inputs, with eager work between, give the eager calls' bits."""
    torch, sffn = need_gpu()
    for rows, d in ((40, 300), (2000, 513)):
        x, res, dy = (_rows(torch, rows, d, torch.bfloat16, k) for k in (1, 2, 3))
        gain, bias = _params(torch, d, torch.bfloat16)

        def calls():
            y, h, mean, rstd = sffn.layer_norm(x, gain, bias=bias, residual=res)
            q, s, _ = sffn.layer_norm_fp8(x, gain, bias=bias, residual=res)
            return [y, h, mean, rstd, q.view(torch.uint8), s, *sffn.layer_norm_backward(dy, h, gain, mean, rstd, dres=dy)]
        eager = calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = calls()
        for k in range(3):
            x.copy_(_rows(torch, rows, d, torch.bfloat16, 10 + k))
            dy.copy_(_rows(torch, rows, d, torch.bfloat16, 20 + k))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, calls()))
        del eager
