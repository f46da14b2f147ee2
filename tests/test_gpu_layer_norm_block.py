"""GPU test of the later operators used together: the example's blocks with layer norms (their gradient
against automatic differentiation in 64 bits), the gradient norm that feeds AdamW, prompts served with
tokens and weights in 4 bits, and all of them in replayed HIP graphs."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import decode_dense, need_gpu

pytestmark = pytest.mark.gpu


def _model(torch, tokens, d_model, d_ff):
    from examples.ffn_block import Model
    model = Model(tokens=tokens, d_model=d_model, d_ff=d_ff, layer_norm=True)
    for n in [b.norm for b in model.blocks] + [model.norm]:
        for t in n.tensors():
            t.add_(0.1 * torch.randn(d_model, device="cuda").to(t.dtype))
    return model


def _plain(torch, model, x):
    """The model in float64 on the host, from the same bf16 values, as autograd leaves.  The ReLU's
    mask is the one the forward stored, on which the layer's backward is defined."""
    leaves = [t.detach().cpu().double().requires_grad_() for t in model.tensors()]
    xl = x.detach().cpu().double().requires_grad_()

    def norm(h, gain, bias):
        c = h - h.mean(1, keepdim=True)
        return c * torch.rsqrt(c.square().mean(1, keepdim=True) + 1e-5) * gain + bias
    h = xl
    for i, b in enumerate(model.blocks):
        gain, bias, W_up, b_up, W_down = leaves[5 * i:5 * i + 5]
        mask = torch.from_numpy(decode_dense(b.cfg, b.saved[3].to_host(), x.shape[0]) > 0)
        h = h + ((norm(h, gain, bias) @ W_up.t() + b_up) * mask) @ W_down
    return norm(h, *leaves[-2:]), xl, leaves


def test_gradient_of_the_blocks():
    """Every gradient of two blocks and the last norm, and their norm.  Each stage of the bf16 path
    rounds its tensors once (relative 2^-8 at most, 2^-9.4 in the mean square), with about ten stages
    one after another: 2e-2 in the norm."""
    torch, sffn = need_gpu()
    model = _model(torch, 96, 256, 512)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.randn((96, 256), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
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
    total = math.sqrt(sum(float(leaf.grad.square().sum()) for leaf in leaves))
    norm, factor = sffn.grad_norm(grads, max_norm=total / 2)
    assert abs(float(norm) - total) <= 2e-2 * total and abs(float(factor) - 0.5) <= 2e-2


@pytest.mark.parametrize("layer_norm", [False, True])
def test_the_example_runs(layer_norm):
    torch, sffn = need_gpu()
    from examples.ffn_block import main
    lines = []
    r = main(steps=3, tokens=100, d_model=256, d_ff=512, layer_norm=layer_norm, log=lines.append)
    assert np.isfinite(r["losses"]).all() and np.isfinite(list(r["served"].values())).all()
    assert any("prompt of 100" in s for s in lines)


def test_a_served_prompt():
    """A prompt through two blocks: what each call gives alone, and the hidden values those of the rounded
    tokens and weights."""
    torch, sffn = need_gpu()
    model = _model(torch, 200, 256, 512)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((200, 256), generator=gen, device="cuda").to(torch.bfloat16)
    y = model.serve()(x)
    f, h = x, None
    for b in model.blocks:
        n, h, _, _ = sffn.layer_norm(f, b.norm.gain, bias=b.norm.bias, residual=h)
        bias = b.b_up.float()
        hidden = sffn.Mx4Linear.from_dense(b.W_up, bias=bias, relu=True).quantized(n, dtype=torch.float32)
        w, q = (_values(torch, *sffn.mx4_quantize(t)) for t in (b.W_up, n))
        ref, size = q @ w.T, np.abs(q) @ np.abs(w).T
        ref = np.maximum(ref + bias.cpu().double().numpy(), 0)
        # 2 blocks of columns, the bias: at most 5 roundings of the absolute values
        assert (np.abs(hidden.cpu().double().numpy() - ref) <= 5 * 2.0 ** -24 * (size + np.abs(ref))).all()
        f = b.ffn.down(sffn.twell_pack(b.cfg, hidden))
    out = sffn.layer_norm(f, model.norm.gain, bias=model.norm.bias, residual=h)[0]
    assert torch.equal(y, out)


def _values(torch, codes, scales):
    e2m1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
    c, z = codes.cpu().numpy(), 2.0 ** (scales.cpu().numpy().astype(np.float64) - 127)
    c = np.stack((c & 15, c >> 4), 2).reshape(z.shape[0], z.shape[1], 32)
    return (e2m1[c] * z[:, :, None]).reshape(z.shape[0], -1)


@pytest.mark.parametrize("layer_norm", [False, True])
def test_serving_between_forward_and_backward(layer_norm):
    """What is served while a training step is under way leaves that step's gradients as they are, prompts of the
    step's own number of tokens among it."""
    torch, _ = need_gpu()
    from examples.ffn_block import Model
    model = Model(tokens=96, d_model=256, d_ff=512, layer_norm=layer_norm)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, dy, other = (torch.randn((96, 256), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    model.forward(x)
    dx, grads = model.backward(dy)
    run = model.serve()
    for t in (5, 64, 96):
        model.forward(x)
        run(other[:t])
        dx2, grads2 = model.backward(dy)
        assert torch.equal(dx, dx2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_prompts_of_blocks_with_rms_norms():
    """Blocks with RMS norms serve any number of tokens in 8 bits unless 4 are asked for, and 4 concern prompts alone."""
    torch, sffn = need_gpu()
    from examples.ffn_block import Model
    model = Model(tokens=200, d_model=256, d_ff=512)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((200, 256), generator=gen, device="cuda").to(torch.bfloat16)
    ups = [sffn.Mx4Linear.from_dense(b.W_up, bias=b.b_up.float(), relu=True) for b in model.blocks]

    def eight(x):
        f, h = x, None
        for b, up in zip(model.blocks, ups):
            q, scale, h = sffn.rms_norm_fp8(f, b.norm.gain, residual=h)
            f = b.ffn.down(sffn.twell_pack(b.cfg, up(q, x_scale=scale, dtype=torch.float32)))
        return sffn.rms_norm(f, model.norm.gain, residual=h)[0]

    def four(x):
        f, h = x, None
        for b, up in zip(model.blocks, ups):
            n, h, _ = sffn.rms_norm(f, b.norm.gain, residual=h)
            f = b.ffn.down(sffn.twell_pack(b.cfg, up.quantized(n, dtype=torch.float32)))
        return sffn.rms_norm(f, model.norm.gain, residual=h)[0]
    run = model.serve()
    for t in (1, 64, 65, 200):
        assert torch.equal(run(x[:t]), eight(x[:t]))
    for t in (1, 64, 65, 200):
        assert torch.equal(model.serve(prompt_bits=4)(x[:t]), (eight if t <= 64 else four)(x[:t]))
    with pytest.raises(ValueError):
        model.serve(prompt_bits=5)


def test_a_training_step_in_a_graph():
    """Norm, its gradient, the gradients' norm and AdamW recorded while eager results live; replays on new
    inputs with eager work between give the eager step's bits."""
    torch, sffn = need_gpu()
    rows, d = 1500, 300
    x, dy = (torch.randn((rows, d), device="cuda") for _ in range(2))
    gain, bias = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")

    def step(opt):
        y, h, mean, rstd = sffn.layer_norm(x, opt.params[0], bias=opt.params[1], residual=x)
        dx, dgain, dbias = sffn.layer_norm_backward(dy, h, opt.params[0], mean, rstd, dres=dy)
        norm, factor = sffn.grad_norm([dgain, dbias], max_norm=1.0)
        opt.step([dgain, dbias], grad_scale=factor)
        return y, dx, dgain, dbias, norm, factor

    def optimizer(params):
        return sffn.AdamW(params, lr=1e-2, weight_decay=0.0)
    eager = step(optimizer([gain.clone(), bias.clone()]))
    opt = optimizer([gain.clone(), bias.clone()])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        recorded = step(opt)
    for k in range(3):
        x.copy_(torch.randn((rows, d), device="cuda") + k)
        dy.copy_(torch.randn((rows, d), device="cuda"))
        for t, v in zip(opt.params, (gain, bias)):
            t.copy_(v)
        for s in opt.state:
            for t in s:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        other = optimizer([gain.clone(), bias.clone()])
        expect = step(other)
        assert all(torch.equal(a, b) for a, b in zip(recorded, expect))
        assert all(torch.equal(a, b) for a, b in zip(opt.params, other.params))
    del eager


def test_two_graphs_and_eager_calls_share_nothing():
    """Two graphs recorded one after the other and eager calls, replayed in any order: every call has its own
    workspace."""
    torch, sffn = need_gpu()
    W = torch.randn((600, 256), device="cuda")
    lin = sffn.Mx4Linear.from_dense(W)
    xs = [torch.randn((n, 256), device="cuda") for n in (90, 300)]
    rows = [torch.randn((2000, 256), device="cuda") for _ in range(2)]
    gain, bias = torch.ones(256, device="cuda"), torch.zeros(256, device="cuda")

    def calls(i):
        y, h, mean, rstd = sffn.layer_norm(rows[i], gain, bias=bias)
        return [lin.quantized(xs[i]), *sffn.layer_norm_backward(y, h, gain, mean, rstd),
                *sffn.grad_norm([rows[i], xs[i]], max_norm=1.0)]
    expect = [calls(0), calls(1)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(calls(i))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for i in order:
            graphs[i].replay()
        again = calls(order[0])
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], expect[i]))
        assert all(torch.equal(a, b) for a, b in zip(again, expect[order[0]]))
        for o in outs:
            for t in o:
                t.zero_()
        for i in (0, 1):
            graphs[i].replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], expect[i]))


def _busy(torch):
    """Some tenths of a second of work on the current stream."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device="cuda")
    b = torch.empty_like(a)
    for _ in range(300):
        torch.mm(a, a, out=b)
    return b


@pytest.mark.parametrize("what", ["weights", "tokens", "tokens of a given stream"])
def test_memory_outlives_a_call_that_waits(what):
    """What a product on another stream has yet to read is not given to another tensor: the weights that the
    layer holds and the tokens, on whatever stream the call runs."""
    torch, sffn = need_gpu()
    x = torch.randn((70, 1024), device="cuda")
    W = torch.randn((4096, 1024), device="cuda")
    side, home = torch.cuda.Stream(), torch.cuda.Stream()
    busy = _busy(torch)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(home):
        own = sffn.Mx4Linear.from_dense(W)
        tokens = sffn.Mx4Tokens(x)
        hold = own.tiled if what == "weights" else tokens._data
    torch.cuda.synchronize()
    expect = own.quantized(tokens)
    ptr, size = hold.data_ptr(), hold.numel()
    with torch.cuda.stream(side):
        busy = _busy(torch)
        done = torch.cuda.Event()
        done.record()
    if what == "tokens of a given stream":
        y = own.quantized(tokens, stream=side)
    else:
        with torch.cuda.stream(side):
            y = own.quantized(tokens)
    with torch.cuda.stream(home):
        if what == "weights":
            del own
        else:
            del tokens
        del hold
        new = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not done.query()  # the call has not run yet
    assert ptr not in {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    assert torch.equal(y, expect) and float(busy[0, 0]) == 8192.0
