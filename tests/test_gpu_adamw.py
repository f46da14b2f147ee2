"""GPU tests of the AdamW step over many tensors, states in 32 and in 8 bits, against the
formulas in 64 bits on the host.

Tolerances, with u = 2^-24: m and v are two products and a sum (and the gradient's scaling):
5 u of their terms' absolute values.  The step divides m by a root and a sum: what m's error makes
of it, plus 16 u of itself; the parameter rounds twice (3 u), and a bf16 one is the rounding of
such a value.  8-bit values: half a step of e4m3, 2^-4 of the value, or below the normal range 2^-10 of the
scale (2^-9 for the root, which never becomes zero); scales: 8 u more than the largest value's error."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import need_gpu
from tests.ops_helpers import rounded_from

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SIZES = [1, 7, 8, 255, 256, 257, 0, 2047, 2048, 2049, 40003]
HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _cut(torch, flat, sizes, shift):
    """Views of one flat tensor: from `shift` on, so that few start at an aligned address."""
    out, at = [], shift
    for n in sizes:
        out.append(flat[at:at + n])
        at += n
    return out


def _make(torch, sizes, param, grad, master, seed, shift=1):
    g = torch.Generator().manual_seed(seed)
    n = sum(sizes) + shift
    draw = lambda s: (s * torch.randn(n, generator=g)).cuda()  # noqa: E731
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    w = draw(0.1)
    gr = draw(1e-2) * torch.exp(2 * draw(1.0))
    cut = lambda t: _cut(torch, t, sizes, shift)  # noqa: E731
    return cut(w.to(dt[param])), cut(gr.to(dt[grad])), cut(w) if master else None


def _blocks(n):
    return -(-n // 256)


def _spread(s, n):
    return np.repeat(s, 256)[:n]


def _moments(opt, i):
    """m and v of tensor i as they stand, in 64 bits."""
    if opt.state_bits == 32:
        return _f64(opt.state[0][i]), _f64(opt.state[1][i])
    n = opt.params[i].numel()
    m = _f64(opt.state[0][i]) * _spread(_f64(opt.state[1][i]), n)
    r = _f64(opt.state[2][i]) * _spread(_f64(opt.state[3][i]), n)
    return m, r * r


def _step_and_check(torch, opt, grads, scale, hyper):
    b1, b2 = hyper["betas"]
    t = opt.steps + 1
    before = []
    for i, p in enumerate(opt.params):
        w = _f64(opt.master[i] if opt.master is not None else p)
        before.append((w, *_moments(opt, i)))
    opt.step(grads, grad_scale=scale)
    assert opt.steps == t
    f = 1.0 if scale is None else float(scale)
    for i, p in enumerate(opt.params):
        n = p.numel()
        if n == 0:
            continue
        w, m, v = before[i]
        g = _f64(grads[i]) * f
        ma, va = b1 * np.abs(m) + (1 - b1) * np.abs(g), b2 * v + (1 - b2) * g * g
        m, v = b1 * m + (1 - b1) * g, va
        den = np.sqrt(v / (1 - b2 ** t)) + hyper["eps"]
        step = hyper["lr"] / (1 - b1 ** t)
        upd = step * m / den
        new = w - hyper["lr"] * hyper["weight_decay"] * w - upd
        tol = 3 * U * np.abs(w) + step * 5 * U * ma / den + 16 * U * np.abs(upd) + 1e-37
        if opt.master is not None:
            assert np.all(np.abs(_f64(opt.master[i]) - new) <= tol), i
            assert torch.equal(p, opt.master[i].to(p.dtype))
        else:
            assert np.all(rounded_from(_f64(p), new, tol, p.dtype == torch.bfloat16)), i
        if opt.state_bits == 32:
            assert np.all(np.abs(_f64(opt.state[0][i]) - m) <= 5 * U * ma + 1e-37), i
            assert np.all(np.abs(_f64(opt.state[1][i]) - v) <= 5 * U * va + 1e-37), i
            continue
        pad = lambda a: np.pad(a, (0, -n % 256)).reshape(-1, 256)  # noqa: E731
        r = np.sqrt(v)
        for k, (x, xa, low) in enumerate(((m, ma, 2.0 ** -10), (r, r, 2.0 ** -9))):
            s = _f64(opt.state[2 * k + 1][i])
            want = np.maximum(np.abs(pad(x)).max(axis=1) / 448, 2.0 ** -126)
            slack = 8 * U * pad(xa).max(axis=1) / 448
            assert np.all(np.abs(s - want) <= slack + 1e-44), (i, k)
            got = _f64(opt.state[2 * k][i]) * _spread(s, n)
            assert np.all(np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + low * _spread(s, n) + 10 * U * xa), (i, k)
            if k == 1:
                assert np.all((got > 0) == (r > 0))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,master", [("f32", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_steps(bits, param, master, grad):
    torch, sffn = need_gpu()
    params, grads, w = _make(torch, SIZES, param, grad, master, 1)
    opt = sffn.AdamW(params, master=w, state_bits=bits, **HYPER)
    for k in range(3):
        scale = torch.tensor([0.37], device="cuda") if k == 1 else None
        _, grads, _ = _make(torch, SIZES, param, grad, False, 10 + k, shift=3)
        _step_and_check(torch, opt, grads, scale, HYPER)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More tensors than one launch takes, empty ones among them; neighbours in one flat tensor
    stay untouched."""
    torch, sffn = need_gpu()
    sizes = [(37 * i) % 613 for i in range(131)]
    params, grads, _ = _make(torch, sizes, "f32", "f32", False, 2)
    opt = sffn.AdamW(params, state_bits=bits, **HYPER)
    _step_and_check(torch, opt, grads, None, HYPER)
    flat = torch.full((1000,), 5.0, device="cuda")
    opt = sffn.AdamW([flat[101:808]], state_bits=bits, **HYPER)
    opt.step([torch.ones(707, device="cuda")])
    assert (flat[:101] == 5).all() and (flat[808:] == 5).all() and (flat[101:808] != 5).all()


def test_large_tensor_and_continued_state():
    """A tensor of some millions, its states given with the steps done."""
    torch, sffn = need_gpu()
    n = 3 * (1 << 20) + 5
    for bits in (32, 8):
        params, grads, w = _make(torch, [n], "bf16", "f32", True, 3, shift=0)
        opt = sffn.AdamW(params, master=w, state_bits=bits, **HYPER)
        opt.step(grads)
        again = sffn.AdamW(params, master=w, state=opt.state, step=opt.steps, **HYPER)
        assert again.state_bits == bits
        _step_and_check(torch, again, [g * 0.5 for g in grads], None, HYPER)


def test_offsets_beyond_32_bits():
    """A tensor of more than 2^31 elements: its last blocks take the step of a small tensor."""
    torch, sffn = need_gpu()
    n, tail = (1 << 31) + 256 + 77, 256 + 77  # the tail starts at a block
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-tail:] = torch.randn(tail, device="cuda").to(torch.bfloat16)
    g[-tail:] = torch.randn(tail, device="cuda").to(torch.bfloat16)
    small, sg = p[-tail:].clone(), g[-tail:].clone()
    opt = sffn.AdamW([p], state_bits=8, **HYPER)
    ref = sffn.AdamW([small], state_bits=8, **HYPER)
    for _ in range(2):
        opt.step([g])
        ref.step([sg])
    assert torch.equal(p[-tail:], small) and not p[:-tail].any()
    for k, count in zip(range(4), (tail, 2, tail, 2)):
        assert torch.equal(opt.state[k][0][-count:].float(), ref.state[k][0].float())


def test_matrix_parameters_and_late_steps():
    torch, sffn = need_gpu()
    hyper = dict(lr=3e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0)
    p = torch.randn(33, 65, device="cuda")
    g = torch.randn(33, 65, device="cuda")
    opt = sffn.AdamW([p], state=[[torch.zeros_like(p)], [torch.full_like(p, 1e-3)]], step=9999, **hyper)
    w0, m0, v0 = _f64(p), np.zeros((33, 65)), np.full((33, 65), np.float64(np.float32(1e-3)))
    opt.step([g])
    m = 0.1 * _f64(g)
    v = 0.999 * v0 + 0.001 * _f64(g) ** 2
    new = w0 - 3e-4 * m / (1 - 0.9 ** 10000) / (np.sqrt(v / (1 - 0.999 ** 10000)) + 1e-8)
    assert np.all(np.abs(_f64(p) - new) <= 3 * U * np.abs(w0) + 24 * U * np.abs(new - w0))


def test_zero_and_non_finite_gradients():
    torch, sffn = need_gpu()
    for bits in (32, 8):
        p = torch.ones(1024, device="cuda")
        opt = sffn.AdamW([p], state_bits=bits, **HYPER)
        opt.step([torch.zeros(1024, device="cuda")])
        want = np.float64(1) - 1e-2 * 0.1
        assert np.all(np.abs(_f64(p) - want) <= 3 * U)
        g = torch.full((1024,), 1e-3, device="cuda")
        g[300] = float("nan")
        opt.step([g])
        bad = torch.isnan(p)
        assert bad[300] and int(bad.sum()) == 1  # the step itself is per element
        opt.step([torch.full((1024,), 1e-3, device="cuda")])
        # an 8-bit block shares its scale with the NaN from then on
        rows = torch.isnan(p).view(4, 256).any(1)
        assert rows.tolist() == [False, True, False, False]
        assert int(torch.isnan(p).sum()) == (1 if bits == 32 else 256)


def test_root_never_becomes_zero():
    """Within one 8-bit block, gradients 2^30 apart: the small ones keep a positive root, so
    their steps stay bounded."""
    torch, sffn = need_gpu()
    g = torch.full((256,), 2.0 ** -20, device="cuda")
    g[0] = 2.0 ** 10
    p = torch.zeros(256, device="cuda")
    opt = sffn.AdamW([p], state_bits=8, lr=1e-3, betas=(0.9, 0.95), eps=0.0, weight_decay=0.0)
    for _ in range(4):
        opt.step([g])
    assert torch.isfinite(p).all()
    assert (opt.state[2][0].float() > 0).all()
    assert float(p.abs().max()) <= 4 * 1e-3 * 1.01


def test_other_stream_and_repeat():
    torch, sffn = need_gpu()
    res = []
    for side in (None, torch.cuda.Stream()):
        params, grads, w = _make(torch, SIZES, "bf16", "f32", True, 5)
        opt = sffn.AdamW(params, master=w, state_bits=8, **HYPER)
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
        opt.step(grads, stream=side)
        if side is not None:
            torch.cuda.current_stream().wait_stream(side)
        res.append([t.float().clone() for k in opt.state for t in k] + [t.clone() for t in w])
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_refusals():
    torch, sffn = need_gpu()
    p = torch.zeros(300, device="cuda")
    b = p.bfloat16()
    opt = sffn.AdamW([p])
    bad = [
        lambda: sffn.AdamW([]),
        lambda: sffn.AdamW([p.half()]),
        lambda: sffn.AdamW([p.cpu()]),
        lambda: sffn.AdamW([p, b]),
        lambda: sffn.AdamW([p, p]),
        lambda: sffn.AdamW([p], master=[p]),
        lambda: sffn.AdamW([b], master=[p[:10]]),
        lambda: sffn.AdamW([p], state_bits=16),
        lambda: sffn.AdamW([p], state=[[p]]),
        lambda: sffn.AdamW([p], state=[[p], [p[:5]]]),
        lambda: sffn.AdamW([p[::2]]),
        lambda: opt.step([]),
        lambda: opt.step([p[:5]]),
        lambda: opt.step([p.half()]),
        lambda: opt.step([p], grad_scale=torch.ones(2, device="cuda")),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for kw in (dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(lr=math.nan), dict(weight_decay=-0.1)):
        with pytest.raises(sffn.SffnError) as ei:
            sffn.AdamW([p], **kw).step([p.clone()])
        assert ei.value.status == sffn.SFFN_ERR_INVALID_ARGUMENT


def test_8bit_codes_are_of_the_quotient():
    """The codes are e4m3(m / scale) and e4m3(r / scale) with the quotients in fp32, no reciprocal in
    their place: first steps whose moments lie within a few roundings of the middle between two
    codes.  From zero states both forms of the state compute the same m and v."""
    torch, sffn = need_gpu()
    n = 1 << 16
    rng = np.random.default_rng(12)
    v = np.array([(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1])
    mid = rng.choice((v[1:] + v[:-1]) / 2, n) * rng.choice([-1.0, 1.0], n)
    top = np.repeat((1 + rng.random(n // 256)).astype(np.float32), 256)  # scales of many digits
    g = (mid * (top.astype(np.float64) / 448)).astype(np.float32)
    g = (g.view(np.int32) + rng.integers(-3, 4, n).astype(np.int32)).view(np.float32)
    g[::256] = top[::256]
    opts = []
    for bits in (32, 8):
        opts.append(sffn.AdamW([torch.zeros(n, device="cuda")], state_bits=bits, **HYPER))
        opts[-1].step([torch.from_numpy(g).cuda()])
    m = opts[0].state[0][0].cpu().numpy()
    r = np.sqrt(opts[0].state[1][0].cpu().numpy())
    codes = lambda a: torch.from_numpy(a).to(torch.float8_e4m3fn).view(torch.uint8).numpy()  # noqa: E731
    for k, x in enumerate((m, r)):
        s = opts[1].state[2 * k + 1][0].cpu().numpy()
        assert np.array_equal(s, np.abs(x).reshape(-1, 256).max(1) / np.float32(448))
        s = np.repeat(s, 256)
        want = codes(x / s)
        assert (codes(x * (np.float32(1) / s)) != want).any()  # the inputs tell the two apart
        assert np.array_equal(opts[1].state[2 * k][0].view(torch.uint8).cpu().numpy(), want), k


@pytest.mark.parametrize("bits", [32, 8])
def test_replaced_tensors(bits):
    """A step works on the tensors as they stand: on a storage that replaced another's, and on
    parameters, masters and states that were assigned; nothing can be replaced past the checks."""
    torch, sffn = need_gpu()
    sizes = [300, 5000]
    params, grads, w = _make(torch, sizes, "bf16", "f32", True, 7)
    opt = sffn.AdamW(params, master=w, state_bits=bits, **HYPER)
    _step_and_check(torch, opt, grads, None, HYPER)
    # new storages behind the same tensors; the old memory is left alone
    old = [t.detach() for t in (params[1], w[0], opt.state[0][1])]
    before = [t.clone() for t in old]
    for t in (params[1], w[0], opt.state[0][1]):
        t.data = t.clone()
    _step_and_check(torch, opt, grads, None, HYPER)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(old, before))
    # assigned lists
    opt.state = [[t.clone() for t in k] for k in opt.state]
    opt.master = [t.clone() for t in opt.master]
    opt.params = [t.clone() for t in opt.params]
    kept = [t.clone() for t in params + w]
    _step_and_check(torch, opt, grads, None, HYPER)
    assert all(torch.equal(a, b) for a, b in zip(params + w, kept))
    # a single entry cannot be replaced, and what does not fit is refused and changes nothing
    with pytest.raises(TypeError):
        opt.state[0][0] = opt.state[0][0].clone()
    for name, value in (("state", [[t[:5] for t in k] for k in opt.state]), ("state", opt.state[:1]),
                        ("master", [t.double() for t in opt.master]), ("params", opt.params[:1]), ("params", [])):
        with pytest.raises(ValueError):
            setattr(opt, name, value)
    for name in ("state_bits", "device", "dtype"):
        with pytest.raises(AttributeError):
            setattr(opt, name, getattr(opt, name))
    _step_and_check(torch, opt, grads, None, HYPER)
    p = opt.params[0]
    p.data = p.float()
    with pytest.raises(ValueError):
        opt.step(grads)


def test_overlapping_tensors_are_refused():
    """Every tensor that a step writes has memory of its own; neighbours in one buffer are fine."""
    torch, sffn = need_gpu()
    flat = torch.zeros(6000, device="cuda")
    p, q, z = flat[:300], flat[300:600], [flat[1000 + 300 * i:1300 + 300 * i] for i in range(8)]
    low = torch.zeros(900, device="cuda").bfloat16()
    ok = sffn.AdamW([p, q], state=[z[:2], z[2:4]])
    bad = [
        lambda: sffn.AdamW([p, p]),
        lambda: sffn.AdamW([p, flat[299:599]]),
        lambda: sffn.AdamW([p], state=[[z[0]], [z[0]]]),
        lambda: sffn.AdamW([p, q], state=[[z[0], z[1]], [z[2], z[0]]]),
        lambda: sffn.AdamW([p], state=[[p], [z[0]]]),
        lambda: sffn.AdamW([p], state=[[z[0]], [flat[200:500]]]),
        lambda: sffn.AdamW([low[:300], low[300:600]], master=[z[0], z[0]]),
        lambda: sffn.AdamW([low[:300]], master=[z[0]], state=[[z[1]], [z[0]]]),
        lambda: sffn.AdamW([low[:300]], master=[low.view(torch.float32)[:300]]),
        lambda: setattr(ok, "state", [z[:2], z[1:3]]),
        lambda: setattr(ok, "params", [p, p]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    e = flat[:0]
    sffn.AdamW([e, p, e], state=[[e, z[0], e], [e, z[1], e]]).step([e, q, e])
    ok.step([torch.ones_like(p), torch.ones_like(q)])
