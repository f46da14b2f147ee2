"""Two pre-norm residual FFN blocks trained and then served with the library's operators.

Training, bf16 with fp32 masters: RMS norm with the residual's sum, the sparse FFN forward and
backward, the norm's gradient, and one AdamW step over all tensors with states in 8 bits and the
gradients clipped to a norm on the device.  Serving: the norm with its output in 8 bits, the
up-projection in 4 bits, the TwELL pack and the sparse down-projection.

    python examples/ffn_block.py [--steps 40] [--tokens 512] [--d-model 512] [--d-ff 2048]
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import activation_sparse_transformer_amd as sffn  # noqa: E402


class Block:
    """h = x + residual; f = FFN(rms_norm(h)).  The next block (or the last norm) adds f to h."""

    def __init__(self, tokens, d_model, d_ff, gen):
        def draw(*shape, scale=1.0):
            return (scale * torch.randn(shape, generator=gen, device="cuda")).to(torch.bfloat16)
        self.cfg = sffn.Config(d_model=d_model, d_ff=d_ff, tile=128, ell_width=64, max_tokens=tokens,
                               backup_capacity=tokens * (d_ff // 128), dtype="bf16")
        self.gain = torch.ones(d_model, device="cuda", dtype=torch.bfloat16)
        self.W_up = draw(d_ff, d_model, scale=d_model ** -0.5)
        self.b_up = draw(d_ff, scale=0.1) - 1.0
        self.W_down = draw(d_ff, d_model, scale=d_ff ** -0.5)
        self.ffn = sffn.SparseFFN(self.cfg, self.W_up, self.b_up, self.W_down)

    def tensors(self):
        return [self.gain, self.W_up, self.b_up, self.W_down]

    def forward(self, x, residual=None):
        n, h, rstd = sffn.rms_norm(x, self.gain, residual=residual)
        f, act = self.ffn.forward(n)
        self.saved = (n, h, rstd, act)
        return f, h

    def backward(self, df, dh):
        """Gradients of x (and the residual) and of tensors(), from those of f and h."""
        n, h, rstd, act = self.saved
        dn, dW_up, dW_down, db, _, _ = self.ffn.backward(n, df, act)
        dx, dgain = sffn.rms_norm_backward(dn, h, self.gain, rstd, dres=dh)
        return dx, [dgain, dW_up, db, dW_down]


class Model:
    def __init__(self, tokens, d_model, d_ff, n_blocks=2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.blocks = [Block(tokens, d_model, d_ff, gen) for _ in range(n_blocks)]
        self.gain = torch.ones(d_model, device="cuda", dtype=torch.bfloat16)

    def tensors(self):
        return [t for b in self.blocks for t in b.tensors()] + [self.gain]

    def forward(self, x):
        f, h = self.blocks[0].forward(x)
        for b in self.blocks[1:]:
            f, h = b.forward(f, residual=h)
        y, self.h, self.rstd = sffn.rms_norm(f, self.gain, residual=h)
        return y

    def backward(self, dy):
        """(dx, gradients in the order of tensors())."""
        d, dgain = sffn.rms_norm_backward(dy, self.h, self.gain, self.rstd)
        grads = [dgain]
        for b in reversed(self.blocks):  # d: the gradient of both f and h
            d, g = b.backward(d, d)
            grads = g + grads
        return d, grads

    def serve(self):
        """The forward for few tokens: 8-bit norms, 4-bit up-projections laid out once."""
        ups = [sffn.Mx4Linear.from_dense(b.W_up, bias=b.b_up.float(), relu=True) for b in self.blocks]

        def run(x):
            f, h = x, None
            for b, up in zip(self.blocks, ups):
                q, scale, h = sffn.rms_norm_fp8(f, b.gain, residual=h)
                act = sffn.twell_pack(b.cfg, up(q, x_scale=scale, dtype=torch.float32))
                f = b.ffn.down(act)
            return sffn.rms_norm(f, self.gain, residual=h)[0]
        return run


def main(steps=40, tokens=512, d_model=512, d_ff=2048, lr=2e-3, max_norm=1.0, log=print):
    model = Model(tokens, d_model, d_ff)
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
        norm = torch.stack([g.norm() for g in grads]).norm()
        opt.step(grads, grad_scale=(max_norm / norm).clamp(max=1.0).reshape(1))
    losses = torch.stack(losses).tolist()
    log(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    run = model.serve()
    y = model.forward(x).float()
    far = {}
    for t in (1, 5, 64):
        far[t] = float((run(x[:t]).float() - y[:t]).norm() / y[:t].norm())
        log(f"served {t} tokens: {far[t]:.3f} from the bf16 forward")
    return {"losses": losses, "served": far}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    for name, value in (("steps", 40), ("tokens", 512), ("d-model", 512), ("d-ff", 2048)):
        ap.add_argument("--" + name, type=int, default=value)
    main(**vars(ap.parse_args()))
