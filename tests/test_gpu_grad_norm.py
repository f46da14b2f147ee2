"""GPU tests of the gradient norm and of clipping, against 64 bits on the host.

The norm's squares are exact and their sum is in 64 bits (n 2^-53 of it at most), so the norm is off by
its one rounding to fp32, 2^-24, and 1e-9 covers the rest; the factor is the rounded quotient by that
norm, and a clipped gradient the rounded product by that factor, bit for bit."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _make(torch, sizes, types, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(scale * torch.randn(n, generator=g, device="cuda")).to(types[i % len(types)])
            for i, n in enumerate(sizes)]


def _norm64(torch, grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


def _check(torch, sffn, grads, max_norm):
    ref = _norm64(torch, grads)
    norm, factor = sffn.grad_norm(grads, max_norm=max_norm)
    assert norm.shape == factor.shape == (1,) and norm.dtype == factor.dtype == torch.float32
    n = float(norm)
    assert abs(n - ref) <= (U + 1e-9) * ref
    want = 1.0 if n <= max_norm else np.float32(max_norm / n)
    assert float(factor) == want
    only, none = sffn.grad_norm(grads)
    assert none is None and torch.equal(only, norm)
    expect = [(t.float() * factor).to(t.dtype) for t in grads]
    out = [torch.full_like(t, 7.0) for t in grads]
    n2, f2 = sffn.clip_grads(grads, max_norm, out=out)
    assert torch.equal(n2, norm) and torch.equal(f2, factor)
    assert all(torch.equal(a, b) for a, b in zip(out, expect))
    own = [t.clone() for t in grads]
    sffn.clip_grads(own, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(own, expect))
    return norm, factor


@pytest.mark.parametrize("sizes", [[1], [7], [8], [9], [2047], [4096], [4097], [8193], [300007], [5_000_011],
                                   [1, 0, 5, 8191, 8192, 1000], [0, 3]])
@pytest.mark.parametrize("types", ["f32", "bf16", "both"])
def test_sizes(sizes, types):
    torch, sffn = need_gpu()
    t = {"f32": [torch.float32], "bf16": [torch.bfloat16], "both": [torch.bfloat16, torch.float32]}[types]
    grads = _make(torch, sizes, t)
    ref = _norm64(torch, grads)
    for max_norm in (ref / 3, 2 * ref, 0.0):
        _check(torch, sffn, grads, max_norm)


@pytest.mark.parametrize("count", [63, 64, 65, 95, 96, 97, 127, 128, 129, 300])
def test_many_tensors(count):
    """More tensors than one launch's table holds, of the norm and of the scaling."""
    torch, sffn = need_gpu()
    rng = np.random.default_rng(count)
    grads = _make(torch, rng.integers(0, 9000, count).tolist(), [torch.float32, torch.float32, torch.bfloat16], count)
    _check(torch, sffn, grads, _norm64(torch, grads) / 2)


@pytest.mark.parametrize("n", [(1 << 22) - 1, (1 << 22) + 1, 12_345_679])
def test_large_chunks(n):
    """Around the size from which a workgroup's part grows with the total."""
    torch, sffn = need_gpu()
    _check(torch, sffn, _make(torch, [n, 100, n // 3], [torch.float32, torch.bfloat16], 3), 1.0)


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 1e30])
def test_no_square_overflows_or_vanishes(scale):
    torch, sffn = need_gpu()
    grads = _make(torch, [1000, 513], [torch.float32, torch.bfloat16], 5, scale)
    _check(torch, sffn, grads, 10 * scale)


def test_one_against_many():
    """A large element does not hide small ones from the sum: 2^24 + 1 equal squares."""
    torch, sffn = need_gpu()
    n = (1 << 24) + 1
    g = torch.ones(n, device="cuda")
    g[0] = 4096.0
    norm, _ = sffn.grad_norm([g])
    assert float(norm) == np.float32(math.sqrt((1 << 24) + (1 << 24)))


def test_special_values():
    torch, sffn = need_gpu()
    for dt in (torch.float32, torch.bfloat16):
        g = torch.zeros(5000, dtype=dt, device="cuda")
        norm, factor = sffn.clip_grads([g], 1.0)
        assert float(norm) == 0 and float(factor) == 1 and (g == 0).all()
        g[4999] = float("inf")
        norm, factor = sffn.grad_norm([g, g], max_norm=1.0)
        assert math.isinf(float(norm)) and float(factor) == 0
        norm, factor = sffn.grad_norm([g], max_norm=float("inf"))
        assert math.isinf(float(norm)) and float(factor) == 1
        g[3] = float("nan")
        norm, factor = sffn.grad_norm([g], max_norm=1.0)
        assert math.isnan(float(norm)) and math.isnan(float(factor))
        g[3] = 1
        sffn.clip_grads([g], 1.0)  # 0 * infinity, and the others 0
        assert torch.isnan(g[4999]) and (g[:4999] == 0).all()
    big = torch.full((4,), 3e38, device="cuda")
    norm, factor = sffn.grad_norm([big], max_norm=1.0)  # beyond fp32
    assert math.isinf(float(norm)) and float(factor) == 0


def test_unaligned_and_repeatable():
    torch, sffn = need_gpu()
    for dt in (torch.float32, torch.bfloat16):
        base = _make(torch, [100_004], [dt], 9)[0]
        view = base[1:100_002]
        a = sffn.grad_norm([view], max_norm=1.0)
        b = sffn.grad_norm([view.clone()], max_norm=1.0)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        first, last = base[0].clone(), base[100_002:].clone()
        expect = (view.float() * a[1]).to(dt)
        sffn.clip_grads([view], 1.0)
        assert torch.equal(view, expect) and base[0] == first and torch.equal(base[100_002:], last)


def test_offsets_beyond_32_bits():
    torch, sffn = need_gpu()
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[0], g[n - 1], g[1 << 31] = 3, 4, 12
    norm, factor = sffn.clip_grads([g], 6.5)
    assert float(norm) == 13 and float(factor) == 0.5
    assert g[0] == 1.5 and g[n - 1] == 2 and g[1 << 31] == 6 and int((g != 0).sum()) == 3


def test_given_outputs_streams_and_adamw():
    """On another stream, into given tensors; the factor feeds AdamW without a wait for the host."""
    torch, sffn = need_gpu()
    grads = _make(torch, [3000, 70], [torch.float32], 2)
    norm, factor = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    a, b = sffn.grad_norm(grads, max_norm=1.0, norm=norm, factor=factor)
    assert a is norm and b is factor
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, d = sffn.grad_norm(grads, max_norm=1.0, stream=side)
    own = [t.clone() for t in grads]
    side.wait_stream(torch.cuda.current_stream())
    sffn.clip_grads(own, 1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c, norm) and torch.equal(d, factor)
    p, q = ([torch.ones_like(t) for t in grads] for _ in range(2))
    sffn.AdamW(p, lr=1e-2).step(grads, grad_scale=factor)
    sffn.AdamW(q, lr=1e-2).step(own)
    assert all(torch.equal(x, y) for x, y in zip(p, q))


def test_in_a_graph():
    """Recorded while eager results live; replays on new gradients, with eager work between."""
    torch, sffn = need_gpu()
    grads = _make(torch, [3000, 70, 20000], [torch.float32, torch.bfloat16], 2)
    own = [t.clone() for t in grads]
    out = [torch.empty_like(t) for t in grads]

    def calls():
        return (*sffn.grad_norm(grads, max_norm=2.0), *sffn.clip_grads(grads, 2.0, out=out), *sffn.clip_grads(own, 3.0))
    eager = calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        recorded = calls()
    for k in range(3):
        for t, o, new in zip(grads, own, _make(torch, [3000, 70, 20000], [torch.float32, torch.bfloat16], 30 + k)):
            t.copy_(new)
            o.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        n, f = sffn.grad_norm(grads, max_norm=2.0)
        n3, f3 = sffn.grad_norm(grads, max_norm=3.0)
        assert all(torch.equal(a, b) for a, b in zip(recorded, (n, f, n, f, n3, f3)))
        for t, o, w in zip(grads, out, own):
            assert torch.equal(o, (t.float() * f).to(t.dtype)) and torch.equal(w, (t.float() * f3).to(t.dtype))
    del eager


def test_refusals():
    torch, sffn = need_gpu()
    g = torch.zeros(64, device="cuda")
    one = torch.empty(1, device="cuda")
    flat = torch.zeros(100, device="cuda")
    bad = [
        lambda: sffn.grad_norm([]),
        lambda: sffn.grad_norm([g.cpu()]),
        lambda: sffn.grad_norm([g, g.cpu()]),
        lambda: sffn.grad_norm([g.half()]),
        lambda: sffn.grad_norm([g.view(8, 8).t()]),
        lambda: sffn.grad_norm([g], norm=one.double()),
        lambda: sffn.grad_norm([g], factor=one),
        lambda: sffn.grad_norm([g], max_norm=1.0, factor=one[:0]),
        lambda: sffn.clip_grads([g], 1.0, out=[g, g]),
        lambda: sffn.clip_grads([g], 1.0, out=[g.bfloat16()]),
        lambda: sffn.clip_grads([g], 1.0, out=[g[:32]]),
        lambda: sffn.clip_grads([g, g.clone()], 1.0, out=[one, one]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: sffn.grad_norm([g], max_norm=-1.0), lambda: sffn.grad_norm([g], max_norm=float("nan")),
              lambda: sffn.grad_norm([g], norm=g[:1]), lambda: sffn.grad_norm([g], max_norm=1.0, norm=one, factor=one),
              lambda: sffn.clip_grads([g], 1.0, factor=g[3:4]), lambda: sffn.clip_grads([g], None),
              lambda: sffn.clip_grads([g, g], 1.0), lambda: sffn.clip_grads([flat[:64], flat[32:96]], 1.0),
              lambda: sffn.clip_grads([flat[:64]], 1.0, out=[flat[1:65]]),
              lambda: sffn.clip_grads([flat[:40], flat[40:80]], 1.0, out=[flat[40:80], flat[:40]]),
              lambda: sffn.clip_grads([flat[i:i + 1] for i in range(100)] * 2, 1.0),
              lambda: sffn.clip_grads([g] * 150, 1.0, out=[torch.empty_like(g) for _ in range(149)] + [g])):
        with pytest.raises(sffn.SffnError) as ei:
            f()
        assert ei.value.status == sffn.SFFN_ERR_INVALID_ARGUMENT
    assert float(sffn.grad_norm([g, g])[0]) == 0  # read only: a tensor may come twice
    a, b = torch.empty_like(g), torch.empty_like(g)
    sffn.clip_grads([g, g], 1.0, out=[a, b])
    assert (a == 0).all() and (b == 0).all()


def test_clipping_to_no_norm_changes_nothing():
    """None, which grad_norm takes for no clipping, is refused by a call that clips, also with a factor kept for a
    graph: the gradients and the given tensors stay as they are."""
    torch, sffn = need_gpu()
    grads = _make(torch, [300, 70], [torch.float32, torch.bfloat16], 4)
    kept, out = [t.clone() for t in grads], [torch.full_like(t, 7.0) for t in grads]
    factor, norm = torch.full((1,), 0.5, device="cuda"), torch.full((1,), 3.0, device="cuda")
    for kw in ({}, {"out": out}, {"norm": norm}):
        with pytest.raises(ValueError):
            sffn.clip_grads(grads, None, factor=factor, **kw)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept)) and all((t == 7).all() for t in out)
    assert float(factor) == 0.5 and float(norm) == 3
