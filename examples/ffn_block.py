"""Two pre-norm residual FFN blocks trained and then served with the library's operators.

Training, bf16 with fp32 masters: RMS norm (or layer norm) with the residual's sum, the sparse FFN
forward and backward, the norm's gradient, and one AdamW step over all tensors with states in 8 bits
and the gradients clipped to a norm on the device.  Serving: the norm with its output in 8 bits, the
up-projection in 4 bits, the TwELL pack and the sparse down-projection; prompts also with the tokens in
4 bits.

    python examples/ffn_block.py [--steps 40] [--tokens 512] [--d-model 512] [--d-ff 2048] [--layer-norm]
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import activation_sparse_transformer_amd as sffn  # noqa: E402


class Norm:
    """The norm of h = x + residual: RMS with a gain, or layer norm with a gain and a bias."""

    def __init__(self, d_model, layer):
        self.gain = torch.ones(d_model, device="cuda", dtype=torch.bfloat16)
        self.bias = torch.zeros_like(self.gain) if layer else None

    def tensors(self):
        return [self.gain] if self.bias is None else [self.gain, self.bias]

    def forward(self, x, residual=None):
        """(y, h, statistics): the latter two are what backward takes."""
        if self.bias is None:
            y, h, *stats = sffn.rms_norm(x, self.gain, residual=residual)
        else:
            y, h, *stats = sffn.layer_norm(x, self.gain, bias=self.bias, residual=residual)
        return y, h, stats

    def backward(self, dy, h, stats, dres=None):
        """The gradient of x (and the residual), and of tensors()."""
        grad = sffn.rms_norm_backward if self.bias is None else sffn.layer_norm_backward
        dx, *grads = grad(dy, h, self.gain, *stats, dres=dres)
        return dx, grads

    def fp8(self, x, residual=None):
        """(q, scale, h), for serving"""
        if self.bias is None:
            return sffn.rms_norm_fp8(x, self.gain, residual=residual)
        return sffn.layer_norm_fp8(x, self.gain, bias=self.bias, residual=residual)


class Block:
    """h = x + residual; f = FFN(norm(h)).  The next block (or the last norm) adds f to h."""

    def __init__(self, tokens, d_model, d_ff, gen, layer_norm=False):
        def draw(*shape, scale=1.0):
            return (scale * torch.randn(shape, generator=gen, device="cuda")).to(torch.bfloat16)
        self.cfg = sffn.Config(d_model=d_model, d_ff=d_ff, tile=128, ell_width=64, max_tokens=tokens,
                               backup_capacity=tokens * (d_ff // 128), dtype="bf16")
        self.norm = Norm(d_model, layer_norm)
        self.W_up = draw(d_ff, d_model, scale=d_model ** -0.5)
        self.b_up = draw(d_ff, scale=0.1) - 1.0
        self.W_down = draw(d_ff, d_model, scale=d_ff ** -0.5)
        self.ffn = sffn.SparseFFN(self.cfg, self.W_up, self.b_up, self.W_down)

    def tensors(self):
        return self.norm.tensors() + [self.W_up, self.b_up, self.W_down]

    def forward(self, x, residual=None):
        n, h, stats = self.norm.forward(x, residual)
        f, act = self.ffn.forward(n)
        self.saved = (n, h, stats, act)
        return f, h

    def backward(self, df, dh):
        """Gradients of x (and the residual) and of tensors(), from those of f and h."""
        n, h, stats, act = self.saved
        dn, dW_up, dW_down, db, _, _ = self.ffn.backward(n, df, act)
        dx, dnorm = self.norm.backward(dn, h, stats, dres=dh)
        return dx, dnorm + [dW_up, db, dW_down]


class Model:
    def __init__(self, tokens, d_model, d_ff, n_blocks=2, seed=0, layer_norm=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.blocks = [Block(tokens, d_model, d_ff, gen, layer_norm) for _ in range(n_blocks)]
        self.norm = Norm(d_model, layer_norm)

    def tensors(self):
        return [t for b in self.blocks for t in b.tensors()] + self.norm.tensors()

    def forward(self, x):
        f, h = self.blocks[0].forward(x)
        for b in self.blocks[1:]:
            f, h = b.forward(f, residual=h)
        y, *self.saved = self.norm.forward(f, h)
        return y

    def backward(self, dy):
        """(dx, gradients in the order of tensors())."""
        d, grads = self.norm.backward(dy, *self.saved)
        for b in reversed(self.blocks):  # d: the gradient of both f and h
            d, g = b.backward(d, d)
            grads = g + grads
        return d, grads

    def serve(self, prompt_bits=None):
        """The forward for serving, up-projections in 4 bits laid out once.  Up to 64 tokens are multiplied
        in 8 bits, those of longer prompts in 8 or 4: by default 8 after RMS norms, 4 after layer norms."""
        bits = prompt_bits or (8 if self.norm.bias is None else 4)
        if bits not in (4, 8):
            raise ValueError("prompt_bits must be 4 or 8")
        ups = [sffn.Mx4Linear.from_dense(b.W_up, bias=b.b_up.float(), relu=True) for b in self.blocks]

        def run(x):
            f, h = x, None
            for b, up in zip(self.blocks, ups):
                if bits == 8 or x.shape[0] <= 64:
                    q, scale, h = b.norm.fp8(f, h)
                    hidden = up(q, x_scale=scale, dtype=torch.float32)
                else:
                    n, h, _ = b.norm.forward(f, h)
                    hidden = up.quantized(n, dtype=torch.float32)
                f = b.ffn.down(sffn.twell_pack(b.cfg, hidden))
            return self.norm.forward(f, h)[0]
        return run


def main(steps=40, tokens=512, d_model=512, d_ff=2048, lr=2e-3, max_norm=1.0, layer_norm=False, log=print):
    model = Model(tokens, d_model, d_ff, layer_norm=layer_norm)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, d_model), generator=gen, device="cuda").to(torch.bfloat16)
    mix = torch.randn((d_model, d_model), generator=gen, device="cuda") * d_model ** -0.5
    target = x.float() + torch.relu(x.float() @ mix)
    target = target * torch.rsqrt(target.square().mean(1, keepdim=True))
    params = model.tensors()
    opt = sffn.AdamW(params, master=[p.float() for p in params], state_bits=8, lr=lr,
                     betas=(0.9, 0.95), weight_decay=0.01)
    losses = []
    for step in range(steps):
        err = model.forward(x).float() - target
        losses.append(err.square().mean())
        _, grads = model.backward((2.0 / err.numel() * err).to(torch.bfloat16))
        _, factor = sffn.grad_norm(grads, max_norm=max_norm)
        opt.step(grads, grad_scale=factor)
    losses = torch.stack(losses).tolist()
    log(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    run = model.serve(prompt_bits=4)
    y = model.forward(x).float()
    far = {}
    for t in (1, 5, 64):
        far[t] = float((run(x[:t]).float() - y[:t]).norm() / y[:t].norm())
        log(f"served {t} tokens: {far[t]:.3f} from the bf16 forward")
    if tokens > 64:
        prompt = float((run(x).float() - y).norm() / y.norm())
        log(f"served a prompt of {tokens}, tokens in 4 bits: {prompt:.3f} from the bf16 forward")
    return {"losses": losses, "served": far}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    for name, value in (("steps", 40), ("tokens", 512), ("d-model", 512), ("d-ff", 2048)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--layer-norm", action="store_true")
    main(**vars(ap.parse_args()))
