"""GPU test of the operators used together: the example's residual blocks, their gradient
against automatic differentiation in 64 bits, training with 8-bit optimizer states, serving in
4 and 8 bits, and a replayed HIP graph of the serving calls."""
import pytest

from tests.gpu_helpers import decode_dense, need_gpu

pytestmark = pytest.mark.gpu


def _plain(torch, model, x):
    """The model in float64 on the host, from the same bf16 values, as autograd leaves.  The ReLU's
    mask is the one the forward stored, on which the layer's backward is defined."""
    leaves = [t.detach().cpu().double().requires_grad_() for t in model.tensors()]
    xl = x.detach().cpu().double().requires_grad_()
    norm = lambda h, g: h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * g  # noqa: E731
    h = xl
    for i in range(len(model.blocks)):
        gain, W_up, b_up, W_down = leaves[4 * i:4 * i + 4]
        b = model.blocks[i]
        mask = torch.from_numpy(decode_dense(b.cfg, b.saved[3].to_host(), x.shape[0]) > 0)
        h = h + ((norm(h, gain) @ W_up.t() + b_up) * mask) @ W_down
    return norm(h, leaves[-1]), xl, leaves


def test_gradient_of_the_blocks():
    """Every gradient of two blocks and the last norm.  Each stage of the bf16 path rounds its
    tensors once (relative 2^-8 at most, 2^-9.4 in the mean square), with about ten stages one
    after another: 2e-2 in the norm."""
    torch, sffn = need_gpu()
    from examples.ffn_block import Model
    model = Model(tokens=96, d_model=256, d_ff=512)
    for t in model.tensors():
        if t.dim() == 1 and t.numel() == 256:
            t.add_(0.1 * torch.randn(256, device="cuda").to(t.dtype))
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((96, 256), generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn((96, 256), generator=gen, device="cuda").to(torch.bfloat16)
    y = model.forward(x)
    dx, grads = model.backward(dy)
    ref, xl, leaves = _plain(torch, model, x)
    ref.backward(dy.cpu().double())

    def off(a, b):
        return float((a.cpu().double() - b).norm() / b.norm())
    assert off(y, ref.detach()) <= 2e-2
    assert off(dx, xl.grad) <= 2e-2
    for g, leaf in zip(grads, leaves):
        assert g.shape == leaf.shape and off(g, leaf.grad) <= 2e-2


def test_training_and_serving():
    """The loss falls to under half, and the served outputs are near: a 4-bit weight is off by 10%
    in the mean square, so an FFN's hidden values are too, and the stream's parts stay below
    that."""
    torch, sffn = need_gpu()
    from examples.ffn_block import main
    r = main(steps=40, tokens=256, d_model=256, d_ff=1024, log=lambda s: print(s, flush=True))
    assert r["losses"][-1] < 0.5 * r["losses"][0]
    assert all(v < 0.15 for v in r["served"].values())


def test_serving_in_a_graph():
    """The norm, the 4-bit product and AdamW recorded in a HIP graph: three replays on new inputs,
    with eager work between, give the eager calls' bits."""
    torch, sffn = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(4)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    W, gain, x, res = draw(512, 256), draw(256), draw(3, 256), draw(3, 256)
    up = sffn.Mx4Linear.from_dense(W, relu=True)
    q = torch.empty((3, 256), dtype=torch.float8_e4m3fn, device="cuda")
    scale, h = torch.empty(3, device="cuda"), torch.empty_like(x)
    y = torch.empty((3, 512), device="cuda")
    p, g = torch.zeros(700, device="cuda"), torch.ones(700, device="cuda")
    opt = sffn.AdamW([p], lr=1e-2, weight_decay=0.0)

    def calls():
        sffn.rms_norm_fp8(x, gain, residual=res, q=q, scale=scale, h=h)
        up(q, x_scale=scale, y=y)
        opt.step([g])
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in range(3):
        x.copy_(draw(3, 256))
        res.copy_(draw(3, 256))
        g.fill_(0.5 + k)
        before = [t.clone() for t in (p, opt.state[0][0], opt.state[1][0])]
        graph.replay()
        torch.cuda.synchronize()
        q2, s2, h2 = sffn.rms_norm_fp8(x, gain, residual=res)
        y2 = up(q2, x_scale=s2, dtype=torch.float32)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scale, s2)
        assert torch.equal(h, h2) and torch.equal(y, y2)
        # the recorded step is the second one, with its bias corrections
        ref = sffn.AdamW([before[0]], state=[[before[1]], [before[2]]], step=1, lr=1e-2, weight_decay=0.0)
        ref.step([g])
        assert torch.equal(p, before[0]) and torch.equal(opt.state[1][0], before[2])
        torch.cuda.synchronize()


def _busy(torch):
    """Some tenths of a second of work on the current stream, and an event behind it."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device="cuda")
    b = torch.empty_like(a)
    for _ in range(300):
        torch.mm(a, a, out=b)
    return b


@pytest.mark.parametrize("with_stream", [False, True])
@pytest.mark.parametrize("what", ["weights", "bias", "8-bit states", "replaced states"])
def test_held_memory_outlives_its_owner(what, with_stream):
    """What a layer or an optimizer holds is not given to another tensor of its stream while a
    call on a different stream has yet to run, also with stream=None: the owner goes (or takes
    other tensors) while the call waits behind other work."""
    torch, sffn = need_gpu()
    n = 3 << 20
    x = torch.randn((2, 1024), device="cuda")
    W = torch.randn((4096, 1024), device="cuda")
    side, home = torch.cuda.Stream(), torch.cuda.Stream()
    busy = _busy(torch)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(home):  # the allocations' stream
        if what == "weights":
            own = sffn.Mx4Linear.from_dense(W)
            hold = [own.tiled]
        elif what == "bias":
            own = sffn.Mx4Linear.from_dense(W.repeat(1024, 1)[:n // 4, :32], bias=torch.zeros(n // 4, device="cuda"))
            x = x[:, :32].contiguous()
            hold = [own.bias]
        else:
            own = sffn.AdamW([torch.ones(n, device="cuda")], state_bits=8)
            g = torch.ones(n, device="cuda")
            hold = [own.state[0][0], own.state[2][0]]
    torch.cuda.synchronize()
    ptrs = [t.data_ptr() for t in hold]
    sizes = [t.numel() * t.element_size() for t in hold]
    with torch.cuda.stream(side):
        busy = _busy(torch)
        done = torch.cuda.Event()
        done.record()
    call = (lambda **k: own.step([g], **k)) if "states" in what else (lambda **k: own(x, **k))
    if with_stream:
        call(stream=side)
    else:
        with torch.cuda.stream(side):
            call()
    with torch.cuda.stream(home):
        if what == "replaced states":
            own.state = [[t.clone() for t in k] for k in own.state]
            del hold
        else:
            del own, hold, call
        new = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(3)]
    assert not done.query()  # the call has not run yet
    assert not set(ptrs) & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    assert float(busy[0, 0]) == 8192.0
