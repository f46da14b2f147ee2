"""Cases and plain forms of further operators around the sparse FFN layer: the layer norm with the
residual's sum (also with an 8-bit output for serving) and its gradient, the norm of all gradients
and clipping by it, and products whose tokens are rounded to 4 bits as the weights are, from one
token to long prompts.

`run` computes one pass in plain torch operations, or through the library where `own` is set;
`exact` computes the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
FP8_MAX = 448.0  # largest e4m3 value
SCALE_MIN = 2.0 ** -126
GROUP = 32       # values that share a scale in the 4-bit format
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
NORM_EPS = 1e-5
MAX_NORM = 16384 * 2304            # elements of the largest norm
MAX_GRADS = 2 * (2 * 2304 * 9216 + 9216 + 2 * 2304)
MAX_PROMPT = 16384 * 9216          # outputs of the largest product
MAX_PRODUCT = MAX_PROMPT * 2304
MAX_WEIGHTS = 65536 * 4096


def listed():
    return [
        # one token being decoded: the norm whose 8-bit output the 4-bit product reads
        dict(name="layer norm: one token, 8 bits", op="norm", rows=1, d=2048, dtype="bf16", residual=True, bias=True, out="fp8", pad=0),
        # a training batch of the 1.5B-like layer
        dict(name="layer norm: 1.5B-like batch", op="norm", rows=8192, d=2048, dtype="bf16", residual=True, bias=True, out="same", pad=0),
        # a long prompt of the 2B-like layer, served in 8 bits
        dict(name="layer norm: 2B-like batch, 8 bits", op="norm", rows=16384, d=2304, dtype="bf16", residual=True, bias=True, out="fp8", pad=0),
        # a small f32 run with odd sizes: rows that start at no vector's boundary
        dict(name="layer norm gradient: odd, f32", op="norm_grad", rows=333, d=1537, dtype="f32", dres=True),
        # the training batch of the 2B-like layer
        dict(name="layer norm gradient: 2B-like batch", op="norm_grad", rows=16384, d=2304, dtype="bf16", dres=True),
        # many small odd tensors, as the gains and biases of a deep model are: norm and factor for AdamW
        dict(name="gradient norm: small odd tensors", op="grads", D=0, F=0, layers=0, tensors=48, total=300007, split=7, grad="f32", clip=False, above=True, gain=1.0),
        # two 2B-like layers with the f32 gradients that the layer's backward gives
        dict(name="gradient norm: 2B-like, f32", op="grads", D=2304, F=9216, layers=2, tensors=10, total=0, split=0, grad="f32", clip=False, above=True, gain=1.0),
        # one 1.5B-like layer's bf16 gradients, clipped, in the units of a scaled loss
        dict(name="clipping: 1.5B-like, bf16", op="grads", D=2048, F=8192, layers=1, tensors=5, total=0, split=0, grad="bf16", clip=True, above=True, gain=65536.0),
        # one token through the up-projection of the 1.5B-like layer; f32 out for the TwELL pack
        dict(name="4-bit tokens: one", op="mx4", T=1, N=8192, K=2048, x="bf16", y="f32", bias=True, relu=True, pad=0),
        # a short f32 prompt, odd numbers of tokens and rows
        dict(name="4-bit tokens: odd, f32", op="mx4", T=333, N=9999, K=1504, x="f32", y="f32", bias=True, relu=False, pad=0),
        # a prompt through the up-projection of the 1.5B-like layer; f32 out for the TwELL pack
        dict(name="4-bit tokens: 1.5B-like prompt", op="mx4", T=2048, N=8192, K=2048, x="bf16", y="f32", bias=True, relu=True, pad=0),
        # the largest batch of prompts, 2B-like
        dict(name="4-bit tokens: 2B-like prompts", op="mx4", T=16384, N=9216, K=2304, x="bf16", y="bf16", bias=True, relu=True, pad=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Spread over the logarithm of lo..hi: a power of two, a multiple of 80 or an odd number."""
    n = _log(rng, lo, hi)
    kind = rng.randrange(3)
    if kind == 0:
        n = 1 << (n.bit_length() - 1)
    elif kind == 1 and n >= 80:
        n = n // 80 * 80
    else:
        n = n - 1 | 1
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "grads", "mx4"))
    if op in ("norm", "norm_grad"):
        d = _size(rng, 64, 16384)
        rows = _size(rng, 1, max(1, min(16384, MAX_NORM // (2 * d))))
        c = dict(op=op, rows=rows, d=d, dtype=rng.choice(("bf16", "bf16", "f32")))
        if op == "norm":
            c.update(residual=rng.random() < 0.75, bias=rng.random() < 0.75, out=rng.choice(("same", "fp8")), pad=rng.choice((0, 0, 8, 17)))
        else:
            c.update(dres=rng.random() < 0.75)
        return c
    if op == "grads":
        return dict(op=op, D=0, F=0, layers=0, tensors=_log(rng, 1, 200), total=_log(rng, 1000, MAX_GRADS // 2), split=rng.randrange(1 << 20),
                    grad=rng.choice(("f32", "bf16")), clip=rng.random() < 0.5, above=rng.random() < 0.75, gain=rng.choice((1.0, 1.0, 65536.0)))
    K = _size(rng, 64, 8192)
    N = _size(rng, 64, min(65536, MAX_WEIGHTS // K))
    T = _size(rng, 1, min(16384, MAX_PRODUCT // (2 * N * K), MAX_PROMPT // (2 * N)))
    return dict(op=op, T=T, N=N, K=K, x=rng.choice(("bf16", "bf16", "f32")), y=rng.choice(("bf16", "f32")),
                bias=rng.random() < 0.5, relu=rng.random() < 0.5, pad=rng.choice((0, 0, 8, 17)))


def _sizes(case):
    """Element counts of the gradients."""
    if case["layers"]:
        D, F = case["D"], case["F"]
        return [D * F, F, D * F, D, D] * case["layers"]  # W_up, b_up, W_down, the norm's gain and bias
    r = random.Random(case["split"])
    w = [math.exp(r.uniform(0, 6)) for _ in range(case["tensors"])]
    return [max(1, int(case["total"] * v / sum(w))) for v in w]


def work(case):
    op = case["op"]
    if op == "norm":
        n, e = case["rows"] * case["d"], BYTES[case["dtype"]]
        o, stats = (1, 1) if case["out"] == "fp8" else (e, 2)
        return {"bytes": n * (e + (2 * e if case["residual"] else 0) + o) + 4 * stats * case["rows"] + e * case["d"] * (2 if case["bias"] else 1), "flops": 9 * n}
    if op == "norm_grad":
        n, e = case["rows"] * case["d"], BYTES[case["dtype"]]
        return {"bytes": n * e * (4 if case["dres"] else 3) + 8 * case["rows"] + (e + 8) * case["d"], "flops": 14 * n}
    if op == "grads":
        n = sum(_sizes(case))
        return {"bytes": n * BYTES[case["grad"]] * (2 if case["clip"] else 1), "flops": n * (3 if case["clip"] else 2)}
    T, N, K = case["T"], case["N"], case["K"]
    G = -(-K // GROUP)
    return {"bytes": N * G * 17 + T * K * BYTES[case["x"]] + T * N * BYTES[case["y"]] + (4 * N if case["bias"] else 0), "flops": 2 * T * N * K}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _stream_rows(rows, d, g, dtype, pad=0):
    """Rows of a residual stream: some tokens and some channels are many times the others, and
    every row has a mean of its own."""
    t = torch.randn((rows, d + pad), generator=g, device="cuda")
    t *= 1 + 15 * (torch.rand((rows, 1), generator=g, device="cuda") < 0.01)
    t *= 1 + 7 * (torch.rand((1, d + pad), generator=g, device="cuda") < 0.01)
    t += 0.5 * torch.randn((rows, 1), generator=g, device="cuda")
    return t.to(dtype)[:, :d]


def _to_codes(w):
    """Codes [n, 16 G] (low half first) and scales [n, G] of f32 rows w [n, K]."""
    w = torch.nn.functional.pad(w, (0, -w.shape[1] % GROUP))
    n, G = w.shape[0], w.shape[1] // GROUP
    w = w.view(n, G, GROUP)
    e = torch.frexp(w.abs().amax(2).clamp_min(1e-30))[1] - 3
    a = torch.ldexp(w, -e[:, :, None])
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    c = (torch.bucketize(a.abs(), edges, out_int32=True).to(torch.uint8) | ((a < 0).to(torch.uint8) << 3)).view(n, G * 16, 2)
    return c[:, :, 0] | (c[:, :, 1] << 4), (e + 127).to(torch.uint8)


def _weights(case, g):
    """4-bit weights of a normal matrix, made in parts so that the f32 matrix stays small."""
    N, K = case["N"], case["K"]
    G = -(-K // GROUP)
    codes = torch.empty((N, G * 16), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N, G), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // K)
    for i in range(0, N, step):
        n = min(step, N - i)
        codes[i:i + n], scales[i:i + n] = _to_codes(_normal((n, K), g) / math.sqrt(K))
    return codes, scales


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(op=op, case=case)
    if own:
        import activation_sparse_transformer_amd as sffn
        s["lib"] = sffn
    if op == "norm":
        dt = DTYPES[case["dtype"]]
        s["x"] = _stream_rows(case["rows"], case["d"], g, dt, case["pad"])
        s["residual"] = 2 * _stream_rows(case["rows"], case["d"], g, dt) if case["residual"] else None
        s["gain"] = 1 + 0.1 * _normal(case["d"], g, dt)
        s["bias"] = 0.1 * _normal(case["d"], g, dt) if case["bias"] else None
    elif op == "norm_grad":
        dt = DTYPES[case["dtype"]]
        s["h"] = 2 * _stream_rows(case["rows"], case["d"], g, dt)
        s["dy"] = _normal((case["rows"], case["d"]), g, dt)
        s["dres"] = _normal((case["rows"], case["d"]), g, dt) if case["dres"] else None
        s["gain"] = 1 + 0.1 * _normal(case["d"], g, dt)
        h = s["h"].double()
        s["mean"] = h.mean(1).float()
        s["rstd"] = torch.rsqrt(h.var(1, unbiased=False) + NORM_EPS).float()
    elif op == "grads":
        sizes = _sizes(case)
        n = sum(sizes)
        flat = 1e-3 * case["gain"] * _normal(n, g)
        flat *= torch.exp(_normal(-(-n // 256), g)).repeat_interleave(256)[:n]  # parts of a model learn at different rates
        flat = flat.to(DTYPES[case["grad"]])
        s["grads"] = list(torch.split(flat, sizes))
        size = 1.65e-3 * case["gain"] * math.sqrt(n)  # the norm, nearly
        s["max_norm"] = size / 3 if case["above"] else size * 10
        if case["clip"]:
            s["flat"] = torch.empty_like(flat)
            s["out"] = list(torch.split(s["flat"], sizes))
    else:
        s["codes"], s["scales"] = _weights(case, g)
        x = _normal((case["T"], case["K"] + case["pad"]), g)
        x *= 1 + 7 * (torch.rand((1, case["K"] + case["pad"]), generator=g, device="cuda") < 0.01)
        s["x"] = x.to(DTYPES[case["x"]])[:, :case["K"]]
        s["bias"] = 0.3 * _normal(case["N"], g) if case["bias"] else None
        s["y"] = DTYPES[case["y"]]
        s["lut"] = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
        if own:  # the weights laid out once, as a serving program keeps them
            s["handle"] = s["lib"].Mx4Linear(s["codes"], s["scales"], bias=s["bias"], relu=case["relu"], in_features=case["K"])
    return s


# ------------------------------------------------------------------ one pass

def _norm(s):
    case = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    mean = h.mean(1)
    c = h - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(1) + NORM_EPS)
    y = c * rstd[:, None] * s["gain"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out = [] if s["residual"] is None else [h.to(s["x"].dtype)]
    if case["out"] == "same":
        return [y.to(s["x"].dtype), mean, rstd] + out
    scale = (y.abs().amax(1) / FP8_MAX).clamp_min(SCALE_MIN)
    return [(y / scale[:, None]).to(torch.float8_e4m3fn), scale] + out


def _norm_own(s):
    args = dict(bias=s["bias"], residual=s["residual"], eps=NORM_EPS)
    if s["case"]["out"] == "same":
        y, h, mean, rstd = s["lib"].layer_norm(s["x"], s["gain"], **args)
        return [y, mean, rstd] if s["residual"] is None else [y, mean, rstd, h]
    q, scale, h = s["lib"].layer_norm_fp8(s["x"], s["gain"], **args)
    return [q, scale] if s["residual"] is None else [q, scale, h]


def _norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["h"].float() - s["mean"][:, None]) * rstd
    t = dy * s["gain"].float()
    dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return [dx.to(s["h"].dtype), (dy * xh).sum(0), dy.sum(0)]


def _norm_grad_own(s):
    return list(s["lib"].layer_norm_backward(s["dy"], s["h"], s["gain"], s["mean"], s["rstd"], dres=s["dres"]))


def _grads(s):
    total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum()
    norm = total.sqrt().float().reshape(1)
    factor = torch.where(norm <= s["max_norm"], torch.ones_like(norm), s["max_norm"] / norm)
    if not s["case"]["clip"]:
        return [norm, factor]
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * factor)
    return [norm, factor, s["flat"]]


def _grads_own(s):
    if not s["case"]["clip"]:
        return list(s["lib"].grad_norm(s["grads"], max_norm=s["max_norm"]))
    return list(s["lib"].clip_grads(s["grads"], s["max_norm"], out=s["out"])) + [s["flat"]]


def _round4(x):
    """The e2m1 values, ties to even codes, of x [T, K] by groups of 32 that share a power of two."""
    T, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % GROUP)).view(T, -1, GROUP)
    e = (torch.frexp(x.abs().amax(2))[1] - 3).clamp_min(-127)[:, :, None]
    a = torch.ldexp(x.abs(), -e)
    v = 0.5 * (a > 0.25).float() + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + (a > 2.5).float() + (a >= 3.5) + 2 * (a > 5).float()
    return torch.ldexp(torch.copysign(v, x), e).view(T, -1)[:, :K]


def _mx4(s):
    case = s["case"]
    c = s["codes"]
    c = torch.stack((c & 15, c >> 4), 2).view(-1).int()
    w = s["lut"].index_select(0, c).view(case["N"], -1, GROUP)
    w = (w * torch.exp2(s["scales"].float() - 127)[:, :, None]).view(case["N"], -1)[:, :case["K"]]
    y = _round4(s["x"].float()) @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return (y.clamp_min(0) if case["relu"] else y).to(s["y"])


def _mx4_own(s):
    return s["handle"].quantized(s["x"], dtype=s["y"])


PLAIN = {"norm": _norm, "norm_grad": _norm_grad, "grads": _grads, "mx4": _mx4}
OWN = {"norm": _norm_own, "norm_grad": _norm_grad_own, "grads": _grads_own, "mx4": _mx4_own}


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "grads": _exact_grads, "mx4": _exact_mx4}[case["op"]](s, case)


def _exact_norm(s, case):
    h = s["x"].double()
    if case["residual"]:
        h = h + s["residual"].double()
    mean = h.sum(1) / case["d"]
    var = ((h - mean.unsqueeze(1)) ** 2).sum(1) / case["d"]
    inv = 1 / (var + NORM_EPS).sqrt()
    y = s["gain"].double() * (h - mean.unsqueeze(1)) * inv.unsqueeze(1)
    if case["bias"]:
        y = y + s["bias"].double()
    tail = [h] if case["residual"] else []
    if case["out"] == "same":
        return [y, mean, inv] + tail
    a = y.abs().max(1).values / FP8_MAX
    return [y / a.unsqueeze(1), a] + tail


def _exact_norm_grad(s, case):
    h, dy, gain, mean, inv = (s[k].double() for k in ("h", "dy", "gain", "mean", "rstd"))
    # y_i = gain_i (h_i - m) inv: through h_i itself, through m, and through inv = (var + eps)^(-1/2),
    # d inv / dh_j = -inv^3 (h_j - m) / d
    c, inv = h - mean.unsqueeze(1), inv.unsqueeze(1)
    t = dy * gain
    dx = inv * t - inv * t.sum(1, keepdim=True) / case["d"] - inv ** 3 * c * (t * c).sum(1, keepdim=True) / case["d"]
    if case["dres"]:
        dx = dx + s["dres"].double()
    return [dx, (dy * c * inv).sum(0), dy.sum(0)]


def _exact_grads(s, case):
    g = torch.cat([t.reshape(-1) for t in s["grads"]]).double()
    norm = torch.dot(g, g).sqrt().reshape(1)
    factor = (s["max_norm"] / norm).clamp(max=1.0)
    return [norm, factor, g * factor] if case["clip"] else [norm, factor]


def _e2m1(c):
    """Values of 4-bit codes: exponent in bits 1 and 2, one fraction bit, sign in bit 3."""
    e, f = ((c // 2) % 4).double(), (c % 2).double()
    return torch.where(e > 0, (1 + f / 2) * 2 ** (e - 1), f / 2) * (1 - 2 * (c // 8).double())


def _exact_mx4(s, case):
    T, N, K = case["T"], case["N"], case["K"]
    out = torch.empty((T, N), dtype=torch.float64, device="cuda")
    # the nearest of the fifteen values by distance, of two equally near ones the even code's
    x = torch.nn.functional.pad(s["x"].double(), (0, -K % GROUP)).view(T, -1, GROUP)
    top = x.abs().max(2, keepdim=True).values
    unit = 2.0 ** (torch.floor(torch.log2(top.clamp_min(2.0 ** -140))) - 2).clamp_min(-127)
    a = (x / unit).abs()
    best, value = torch.full_like(a, math.inf), torch.zeros_like(a)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):
        v = float(_e2m1(torch.tensor(c)))
        near = (a - v).abs()
        value = torch.where(near < best, torch.full_like(a, v), value)
        best = torch.minimum(best, near)
    x = (value * torch.sign(x) * unit).view(T, -1)[:, :K]
    step = max(1, (1 << 26) // K)
    for i in range(0, N, step):
        b = s["codes"][i:i + step]
        c = torch.empty((b.shape[0], b.shape[1] * 2), dtype=torch.uint8, device=b.device)
        c[:, 0::2], c[:, 1::2] = b % 16, b // 16
        z = 2.0 ** (s["scales"][i:i + step].double() - 127)
        w = (_e2m1(c) * z.repeat_interleave(GROUP, 1))[:, :K]
        out[:, i:i + step] = x @ w.t()
    if case["bias"]:
        out += s["bias"].double()
    return out.relu_() if case["relu"] else out
