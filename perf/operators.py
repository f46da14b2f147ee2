"""Cases and plain forms of the operators around the sparse FFN layer: the RMS norm with the
residual's sum (also with an 8-bit output for serving), its gradient, products with 4-bit
weights at serving batches, and the AdamW step over the layer's tensors.

`run` computes one pass in plain torch operations, or through the library where `own` is set;
`exact` computes the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "fp8": 1}
FP8_MAX = 448.0       # largest e4m3 value
FP8_TINY = 2.0 ** -9  # smallest positive e4m3 value
SCALE_MIN = 2.0 ** -126
GROUP = 32            # weights that share a scale in the 4-bit format
BLOCK = 256           # values that share a scale in an 8-bit optimizer state
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LR, B1, B2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1
NORM_EPS = 1e-6
MAX_NORM = 16384 * 2304     # elements of the largest norm
MAX_WEIGHTS = 65536 * 8192  # weights of the largest product
MAX_PARAMS = 2 * (2 * 2304 * 9216 + 9216 + 2304)


def listed():
    return [
        # one token being decoded: the norm whose 8-bit output the 4-bit product reads
        dict(name="norm: one token, 8 bits", op="norm", rows=1, d=2048, dtype="bf16", residual=True, out="fp8", pad=0),
        # a training batch of the 1.5B-like layer
        dict(name="norm: 1.5B-like batch", op="norm", rows=8192, d=2048, dtype="bf16", residual=True, out="same", pad=0),
        # a long prefill of the 2B-like layer, served in 8 bits
        dict(name="norm: 2B-like batch, 8 bits", op="norm", rows=16384, d=2304, dtype="bf16", residual=True, out="fp8", pad=0),
        # a small f32 run with odd sizes: rows that start at no vector's boundary
        dict(name="norm gradient: odd, f32", op="norm_grad", rows=333, d=1537, dtype="f32", dres=True),
        # the training batch of the 2B-like layer
        dict(name="norm gradient: 2B-like batch", op="norm_grad", rows=16384, d=2304, dtype="bf16", dres=True),
        # one token through the up-projection of the 1.5B-like layer; f32 out for the TwELL pack
        dict(name="4-bit: one token", op="mx4", T=1, N=8192, K=2048, x="bf16", y="f32", bias=True, relu=True),
        # a few f32 tokens, odd numbers of rows and groups
        dict(name="4-bit: odd, f32", op="mx4", T=5, N=9999, K=1504, x="f32", y="f32", bias=True, relu=False),
        # the largest serving batch, on the 8-bit rows that the norm writes
        dict(name="4-bit: 64 tokens, 8 bits", op="mx4", T=64, N=9216, K=2304, x="fp8", y="f32", bias=True, relu=True),
        # a wide projection at a small batch: 285 MB of weights
        dict(name="4-bit: wide", op="mx4", T=4, N=65536, K=8192, x="bf16", y="bf16", bias=False, relu=False),
        # many small odd tensors, as the gains and biases of a deep model are
        dict(name="adamw: small odd tensors", op="adamw", D=0, F=0, layers=0, tensors=48, total=300007, split=7, bits=32, param="f32", master=False, grad="f32", scaled=False),
        # one 1.5B-like layer with states in 8 bits; gradients in f32 as the layer's backward gives them
        dict(name="adamw: 1.5B-like, 8 bits", op="adamw", D=2048, F=8192, layers=1, tensors=4, total=0, split=0, bits=8, param="bf16", master=True, grad="f32", scaled=True),
        # two 2B-like layers with states in 32 bits and an f32 master
        dict(name="adamw: 2B-like, 32 bits", op="adamw", D=2304, F=9216, layers=2, tensors=8, total=0, split=0, bits=32, param="bf16", master=True, grad="f32", scaled=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, step=1):
    """Spread over the logarithm of lo..hi: a power of two, a multiple of 80 or an odd number, times step."""
    n = _log(rng, lo, hi)
    kind = rng.randrange(3)
    if kind == 0:
        n = 1 << (n.bit_length() - 1)
    elif kind == 1 and n >= 80:
        n = n // 80 * 80
    else:
        n = n - 1 | 1
    return max(lo, n) * step


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "mx4", "adamw"))
    if op in ("norm", "norm_grad"):
        d = _size(rng, 64, 16384)
        rows = _size(rng, 1, max(1, min(16384, MAX_NORM // (2 * d))))
        c = dict(op=op, rows=rows, d=d, dtype=rng.choice(("bf16", "bf16", "f32")))
        if op == "norm":
            c.update(residual=rng.random() < 0.75, out=rng.choice(("same", "fp8")), pad=rng.choice((0, 0, 8, 17)))
        else:
            c.update(dres=rng.random() < 0.75)
        return c
    if op == "mx4":
        K = _size(rng, 2, 256, GROUP)
        N = _size(rng, 64, min(65536, MAX_WEIGHTS // K))
        return dict(op=op, T=_log(rng, 1, 64), N=N, K=K, x=rng.choice(("bf16", "bf16", "f32", "fp8")),
                    y=rng.choice(("bf16", "f32")), bias=rng.random() < 0.5, relu=rng.random() < 0.5)
    param = rng.choice(("bf16", "bf16", "f32"))
    return dict(op=op, D=0, F=0, layers=0, tensors=_log(rng, 1, 64), total=_log(rng, 1000, MAX_PARAMS // 2), split=rng.randrange(1 << 20),
                bits=rng.choice((8, 32)), param=param, master=param == "bf16" and rng.random() < 0.7,
                grad=rng.choice(("f32", "f32", "bf16")), scaled=rng.random() < 0.5)


def _sizes(case):
    """Element counts of the tensors of an optimizer step."""
    if case["layers"]:
        D, F = case["D"], case["F"]
        return [D * F, F, D * F, D] * case["layers"]  # W_up, b_up, W_down, the norm's gain
    r = random.Random(case["split"])
    w = [math.exp(r.uniform(0, 6)) for _ in range(case["tensors"])]
    return [max(1, int(case["total"] * v / sum(w))) for v in w]


def work(case):
    op = case["op"]
    if op == "norm":
        n, e = case["rows"] * case["d"], BYTES[case["dtype"]]
        o = 1 if case["out"] == "fp8" else e
        return {"bytes": n * (e + (2 * e if case["residual"] else 0) + o) + 4 * case["rows"] + e * case["d"], "flops": 6 * n}
    if op == "norm_grad":
        n, e = case["rows"] * case["d"], BYTES[case["dtype"]]
        return {"bytes": n * e * (4 if case["dres"] else 3) + 4 * case["rows"] + (e + 4) * case["d"], "flops": 10 * n}
    if op == "mx4":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": N * K / 2 + N * (K // GROUP) + T * K * BYTES[case["x"]] + T * N * BYTES[case["y"]] + (4 * N if case["bias"] else 0), "flops": 2 * T * N * K}
    n = sum(_sizes(case))
    p = BYTES[case["param"]]
    each = BYTES[case["grad"]] + (p + 8 if case["master"] else 2 * p) + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
    return {"bytes": n * each, "flops": 15 * n}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _stream_rows(rows, d, g, dtype, pad=0):
    """Rows of a residual stream: some tokens and some channels are many times the others."""
    t = torch.randn((rows, d + pad), generator=g, device="cuda")
    t *= 1 + 15 * (torch.rand((rows, 1), generator=g, device="cuda") < 0.01)
    t *= 1 + 7 * (torch.rand((1, d + pad), generator=g, device="cuda") < 0.01)
    return t.to(dtype)[:, :d]


def _to_codes(w):
    """Codes [n, K/2] (low half first) and scales [n, K/32] of f32 rows w [n, K]."""
    n, K = w.shape
    w = w.view(n, K // GROUP, GROUP)
    e = torch.floor(torch.log2(w.abs().amax(2).clamp_min(1e-30))) - 2
    a = w / torch.exp2(e)[:, :, None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    c = (torch.bucketize(a.abs(), edges, out_int32=True).to(torch.uint8) | ((a < 0).to(torch.uint8) << 3)).view(n, K // 2, 2)
    return c[:, :, 0] | (c[:, :, 1] << 4), (e + 127).to(torch.uint8)


def _weights(case, g):
    """4-bit weights of a normal matrix, made in parts so that the f32 matrix stays small."""
    N, K = case["N"], case["K"]
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N, K // GROUP), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // K)
    for i in range(0, N, step):
        n = min(step, N - i)
        codes[i:i + n], scales[i:i + n] = _to_codes(_normal((n, K), g) / math.sqrt(K))
    return codes, scales


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _views(flat, sizes):
    return list(torch.split(flat, sizes))


def _block_max(t):
    return torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)).view(-1, BLOCK).abs().amax(1)


def _block_spread(scale, n):
    return scale.repeat_interleave(BLOCK)[:n]


def _to_8bit(m, r):
    """e4m3 codes and block scales of one tensor's first moment and root second moment."""
    ms = (_block_max(m) / FP8_MAX).clamp_min(SCALE_MIN)
    rs = (_block_max(r) / FP8_MAX).clamp_min(SCALE_MIN)
    mq = (m / _block_spread(ms, m.numel())).to(torch.float8_e4m3fn)
    # a positive root never becomes zero: it divides
    rq = torch.where(r > 0, (r / _block_spread(rs, r.numel())).clamp_min(FP8_TINY), torch.zeros_like(r)).to(torch.float8_e4m3fn)
    return mq, ms, rq, rs


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
    elif op == "norm_grad":
        dt = DTYPES[case["dtype"]]
        s["h"] = 2 * _stream_rows(case["rows"], case["d"], g, dt)
        s["dy"] = _normal((case["rows"], case["d"]), g, dt)
        s["dres"] = _normal((case["rows"], case["d"]), g, dt) if case["dres"] else None
        s["gain"] = 1 + 0.1 * _normal(case["d"], g, dt)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + NORM_EPS)
    elif op == "mx4":
        s["codes"], s["scales"] = _weights(case, g)
        x = _normal((case["T"], case["K"]), g)
        s["x_scale"] = None
        if case["x"] == "fp8":
            s["x_scale"] = x.abs().amax(1) / FP8_MAX
            x = x / s["x_scale"][:, None]
        s["x"] = x.to(DTYPES[case["x"]])
        s["bias"] = 0.3 * _normal(case["N"], g) if case["bias"] else None
        s["y"] = DTYPES[case["y"]]
        s["lut"] = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
        if own:  # the weights laid out once, as a serving program keeps them
            s["handle"] = s["lib"].Mx4Linear(s["codes"], s["scales"], bias=s["bias"], relu=case["relu"])
    else:
        sizes = _sizes(case)
        n = sum(sizes)
        w = 0.05 * _normal(n, g)
        grad = 1e-3 * _normal(n, g)
        grad *= torch.exp(_normal(_blocks(n), g)).repeat_interleave(BLOCK)[:n]  # parts of a model learn at different rates
        m = 0.3 * grad * _normal(n, g)
        r = grad.abs() * (0.5 + torch.rand(n, generator=g, device="cuda"))
        s["t"] = 10
        s["grad_scale"] = torch.full((1,), 0.5, device="cuda") if case["scaled"] else None
        flat = dict(p=w.to(DTYPES[case["param"]]), g=grad.to(DTYPES[case["grad"]]))
        if case["master"]:
            flat["w"] = w
        if case["bits"] == 32:
            flat.update(m=m, v=r * r)
        else:
            parts = [_to_8bit(a, b) for a, b in zip(_views(m, sizes), _views(r, sizes))]
            for k, key in enumerate(("m", "ms", "r", "rs")):
                flat[key] = torch.cat([q[k] for q in parts])
        s["flat"] = flat
        blocks = [_blocks(k) for k in sizes]
        s["parts"] = {k: _views(f, blocks if k in ("ms", "rs") else sizes) for k, f in flat.items()}
        if own:
            P = s["parts"]
            state = [P["m"], P["v"]] if case["bits"] == 32 else [P["m"], P["ms"], P["r"], P["rs"]]
            s["handle"] = s["lib"].AdamW(P["p"], master=P.get("w"), state=state, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=DECAY, step=s["t"])
    return s


# ------------------------------------------------------------------ one pass

def _norm(s):
    case = s["case"]
    x, gain = s["x"].float(), s["gain"].float()
    h = x if s["residual"] is None else x + s["residual"].float()
    rstd = torch.rsqrt(h.square().mean(1) + NORM_EPS)
    y = h * rstd[:, None] * gain
    out = [] if s["residual"] is None else [h.to(s["x"].dtype)]
    if case["out"] == "same":
        return [y.to(s["x"].dtype), rstd] + out
    scale = (y.abs().amax(1) / FP8_MAX).clamp_min(SCALE_MIN)
    return [(y / scale[:, None]).to(torch.float8_e4m3fn), scale] + out


def _norm_own(s):
    case = s["case"]
    if case["out"] == "same":
        y, h, rstd = s["lib"].rms_norm(s["x"], s["gain"], residual=s["residual"], eps=NORM_EPS)
        return [y, rstd] if s["residual"] is None else [y, rstd, h]
    q, scale, h = s["lib"].rms_norm_fp8(s["x"], s["gain"], residual=s["residual"], eps=NORM_EPS)
    return [q, scale] if s["residual"] is None else [q, scale, h]


def _norm_grad(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = s["h"].float() * rstd
    t = dy * s["gain"].float()
    dx = rstd * (t - xh * (t * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return [dx.to(s["h"].dtype), (dy * xh).sum(0)]


def _norm_grad_own(s):
    return list(s["lib"].rms_norm_backward(s["dy"], s["h"], s["gain"], s["rstd"], dres=s["dres"]))


def _mx4(s):
    case = s["case"]
    c = s["codes"]
    c = torch.stack((c & 15, c >> 4), 2).view(-1).int()
    w = s["lut"].index_select(0, c).view(case["N"], -1, GROUP)
    w = (w * torch.exp2(s["scales"].float() - 127)[:, :, None]).view(case["N"], case["K"])
    y = s["x"].float() @ w.t()
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None]
    if s["bias"] is not None:
        y = y + s["bias"]
    return (y.clamp_min(0) if case["relu"] else y).to(s["y"])


def _mx4_own(s):
    return s["handle"](s["x"], x_scale=s["x_scale"], dtype=s["y"])


def _adamw(s):
    P, t = s["parts"], s["t"] + 1
    s["t"] = t
    g = [a.float() for a in P["g"]]
    if s["grad_scale"] is not None:
        g = torch._foreach_mul(g, s["grad_scale"][0])
    bits32 = s["case"]["bits"] == 32
    if bits32:
        m, v = P["m"], P["v"]
    else:
        m = [q.float() * _block_spread(z, q.numel()) for q, z in zip(P["m"], P["ms"])]
        v = [(q.float() * _block_spread(z, q.numel())).square() for q, z in zip(P["r"], P["rs"])]
    torch._foreach_mul_(m, B1)
    torch._foreach_add_(m, g, alpha=1 - B1)
    torch._foreach_mul_(v, B2)
    torch._foreach_addcmul_(v, g, g, 1 - B2)
    root = torch._foreach_sqrt(v)
    den = torch._foreach_add(torch._foreach_div(root, math.sqrt(1 - B2 ** t)), EPS)
    w = P["w"] if "w" in P else P["p"] if P["p"][0].dtype == torch.float32 else [a.float() for a in P["p"]]
    torch._foreach_mul_(w, 1 - LR * DECAY)
    torch._foreach_addcdiv_(w, m, den, -LR / (1 - B1 ** t))
    if w is not P["p"]:
        torch._foreach_copy_(P["p"], w)
    if not bits32:
        q = [_to_8bit(a, b) for a, b in zip(m, root)]
        torch._foreach_copy_(P["ms"], [a[1] for a in q])
        torch._foreach_copy_(P["rs"], [a[3] for a in q])
        s["flat"]["m"].copy_(torch.cat([a[0] for a in q]))
        s["flat"]["r"].copy_(torch.cat([a[2] for a in q]))
    return _adamw_out(s)


def _adamw_own(s):
    s["handle"].step(s["parts"]["g"], grad_scale=s["grad_scale"])
    return _adamw_out(s)


def _adamw_out(s):
    return {k: f for k, f in s["flat"].items() if k != "g"}


PLAIN = {"norm": _norm, "norm_grad": _norm_grad, "mx4": _mx4, "adamw": _adamw}
OWN = {"norm": _norm_own, "norm_grad": _norm_grad_own, "mx4": _mx4_own, "adamw": _adamw_own}


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "mx4": _exact_mx4, "adamw": _exact_adamw}[case["op"]](s, case)


def _exact_norm(s, case):
    h = s["x"].double()
    if case["residual"]:
        h = h + s["residual"].double()
    inv = 1 / ((h * h).sum(1) / case["d"] + NORM_EPS).sqrt()
    y = s["gain"].double() * h * inv.unsqueeze(1)
    tail = [h] if case["residual"] else []
    if case["out"] == "same":
        return [y, inv] + tail
    a = y.abs().max(1).values / FP8_MAX
    return [y / a.unsqueeze(1), a] + tail


def _exact_norm_grad(s, case):
    h, dy, gain, inv = (s[k].double() for k in ("h", "dy", "gain", "rstd"))
    # d/dh of sum(dy * gain * h * inv), inv = (mean(h^2) + eps)^(-1/2): d inv / dh_j = -inv^3 h_j / d
    inv = inv.unsqueeze(1)
    dot = (dy * gain * h).sum(1, keepdim=True)
    dx = inv * dy * gain - inv ** 3 * h * dot / case["d"]
    if case["dres"]:
        dx = dx + s["dres"].double()
    return [dx, (dy * h * inv).sum(0)]


def _exact_mx4(s, case):
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double().unsqueeze(1)
    out = []
    step = max(1, (1 << 26) // case["K"])
    for i in range(0, case["N"], step):
        b = s["codes"][i:i + step]
        c = torch.empty((b.shape[0], case["K"]), dtype=torch.uint8, device=b.device)
        c[:, 0::2], c[:, 1::2] = b % 16, b // 16
        e, f = ((c // 2) % 4).double(), (c % 2).double()
        w = torch.where(e > 0, (1 + f / 2) * 2 ** (e - 1), f / 2) * (1 - 2 * (c // 8).double())
        z = 2.0 ** (s["scales"][i:i + step].double() - 127)
        out.append(x @ (w * z.repeat_interleave(GROUP, 1)).t())
    y = torch.cat(out, 1)
    if case["bias"]:
        y = y + s["bias"].double()
    return y.relu() if case["relu"] else y


def _exact_adamw(s, case):
    sizes, F, t = _sizes(case), s["flat"], s["t"] + 1
    g = F["g"].double() * (0.5 if case["scaled"] else 1.0)
    n, dev = g.numel(), g.device
    if case["bits"] == 32:
        m, v = F["m"].double(), F["v"].double()
    else:  # the block of every value: blocks start anew with each tensor
        first = torch.tensor([0] + sizes[:-1], device=dev).cumsum(0)
        start = torch.tensor([0] + [_blocks(k) for k in sizes[:-1]], device=dev).cumsum(0)
        which = torch.repeat_interleave(torch.arange(len(sizes), device=dev), torch.tensor(sizes, device=dev))
        block = start[which] + (torch.arange(n, device=dev) - first[which]) // BLOCK
        m = F["m"].double() * F["ms"].double()[block]
        v = (F["r"].double() * F["rs"].double()[block]) ** 2
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * g * g
    w = (F["w"] if case["master"] else F["p"]).double()
    w = w - LR * (DECAY * w + (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)).sqrt() + EPS))
    out = {"p": w}
    if case["master"]:
        out["w"] = w
    if case["bits"] == 32:
        return dict(out, m=m, v=v)
    r, count = v.sqrt(), F["ms"].numel()
    ms = torch.zeros(count, dtype=torch.float64, device=dev).scatter_reduce(0, block, m.abs(), "amax") / FP8_MAX
    rs = torch.zeros(count, dtype=torch.float64, device=dev).scatter_reduce(0, block, r, "amax") / FP8_MAX
    return dict(out, m=m / ms[block], ms=ms, r=r / rs[block], rs=rs)
