"""Cases for the operators at a language model's head: layer norm, linear cross entropy
over a vocabulary, and the AdamW step with 8-bit moments that updates both.

Each case is one pass of one operator.  `run` computes it in plain torch operations in
32 bits, or, with `own` set, through the package's entry points; `exact` gives the same
outputs from the definition in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-5
LR, B1, B2, ADAM_EPS, WD = 1e-4, 0.9, 0.999, 1e-8, 0.01
BLOCK = 128                  # elements that share one scale byte of the 8-bit moments
SEED = 20259                 # seed of the stochastic rounding
MIX1, MIX2 = 0x9E3779B9, 0x6A09E667
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST_NORM = 32768 * 1536     # elements of the largest listed layer norm
MOST_CE = 8192 * 2560 * 131072
MOST_ADAM = 131072 * 2560


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def listed():
    return [
        # a decoding step's sixteen tokens through one norm: launch latency
        {"name": "norm_fwd_16tok", "op": "norm_fwd", "rows": 16, "dim": 2560, "dtype": "bf16", "affine": "f32", "pad": 0},
        # a training micro-batch through one norm
        {"name": "norm_fwd_32k", "op": "norm_fwd", "rows": 32768, "dim": 1536, "dtype": "bf16", "affine": "bf16", "pad": 0},
        # its backward pass, with the weight and bias gradients over every row
        {"name": "norm_bwd_32k", "op": "norm_bwd", "rows": 32768, "dim": 1536, "dtype": "bf16", "affine": "f32", "pad": 0},
        # an odd width in 32 bits, rows cut out of a wider buffer
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 5003, "dim": 1537, "dtype": "f32", "affine": "f32", "pad": 3},
        # the losses of a few tokens (scoring an answer): the vocabulary matrix is read once
        {"name": "ce_fwd_8tok", "op": "ce_fwd", "rows": 8, "dim": 1536, "vocab": 32768, "dtype": "bf16", "grad": "mean"},
        # evaluation over a large vocabulary
        {"name": "ce_fwd_8k", "op": "ce_fwd", "rows": 8192, "dim": 2560, "vocab": 131072, "dtype": "bf16", "grad": "mean"},
        # the backward pass of a training micro-batch over the same vocabulary, mean loss
        {"name": "ce_bwd_8k", "op": "ce_bwd", "rows": 8192, "dim": 2560, "vocab": 131072, "dtype": "bf16", "grad": "mean"},
        # a ragged batch and an odd vocabulary, a weight for every token's loss
        {"name": "ce_bwd_odd", "op": "ce_bwd", "rows": 1021, "dim": 1536, "vocab": 50257, "dtype": "bf16", "grad": "rows"},
        # a small model trained in 32 bits, every size odd
        {"name": "ce_bwd_f32", "op": "ce_bwd", "rows": 1021, "dim": 1001, "vocab": 10007, "dtype": "f32", "grad": "mean"},
        # the norm weights and biases of a model's blocks: many small tensors, launch latency
        {"name": "adam_norms", "op": "adam", "tensors": 48, "small": 1536, "large": 0, "dtype": "bf16", "gdtype": "bf16"},
        # a vocabulary matrix and its norm weights
        {"name": "adam_head", "op": "adam", "tensors": 3, "small": 2560, "large": 131072 * 2560, "dtype": "bf16", "gdtype": "bf16"},
        # 32-bit parameters with 16-bit gradients, odd sizes
        {"name": "adam_f32_odd", "op": "adam", "tensors": 9, "small": 1537, "large": 50257 * 768, "dtype": "f32", "gdtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ce_fwd", "ce_bwd", "adam"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        dim = _log(rng, 16, 16384)
        dim = dim if rng.random() < 0.5 else dim // 8 * 8
        rows = _log(rng, 1, max(1, min(65536, MOST_NORM // dim)))
        return {"op": op, "rows": rows, "dim": dim, "dtype": dtype, "affine": rng.choice(["bf16", "f32", "none"]),
                "pad": rng.choice([0, 0, 8, 5])}
    if op.startswith("ce"):
        dim = _log(rng, 32, 4096)
        dim = dim if rng.random() < 0.3 else max(32, dim // 64 * 64)
        vocab = _log(rng, 1000, 131072)
        most = MOST_CE // 8 if dtype == "f32" else MOST_CE
        rows = _log(rng, 1, max(1, min(8192, most // (dim * vocab))))
        return {"op": op, "rows": rows, "dim": dim, "vocab": vocab, "dtype": dtype, "grad": rng.choice(["mean", "rows"])}
    large = _log(rng, 1000, MOST_ADAM // 2)
    return {"op": op, "tensors": rng.randint(1, 60), "small": _log(rng, 1, 16384), "large": large, "dtype": dtype,
            "gdtype": rng.choice(["bf16", "f32"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _adam_sizes(case):
    n = case["tensors"] - (1 if case["large"] else 0)
    return ([case["large"]] if case["large"] else []) + [max(1, case["small"] + 7 * (i % 3)) if case["small"] % 2 else case["small"]
                                                         for i in range(n)]


def _starts(sizes):
    """Where each tensor begins in the moments' buffers: on a block's first element."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    return at


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    s = {"case": case}
    op = case["op"]
    if op.startswith("norm"):
        n, d, dt = case["rows"], case["dim"], TYPES[case["dtype"]]
        # activations: a common offset, a scale for every channel, a few large channels
        scale = 0.5 + torch.rand(d, generator=g, device=dev) + 8.0 * (torch.rand(d, generator=g, device=dev) < 0.002)
        x = normal(n, d + case["pad"]) * 0.7 + 0.1
        x[:, :d] *= scale
        s["x"] = x.to(dt)[:, :d]
        del x
        wt = None if case["affine"] == "none" else TYPES[case["affine"]]
        s["w"] = None if wt is None else (1.0 + 0.2 * normal(d)).to(wt)
        s["b"] = None if wt is None else (0.1 * normal(d)).to(wt)
        if op == "norm_bwd":
            s["dy"] = (normal(n, d) * 1e-2).to(dt)
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = 1.0 / torch.sqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
            del xf
    elif op.startswith("ce"):
        n, d, v, dt = case["rows"], case["dim"], case["vocab"], TYPES[case["dtype"]]
        w = normal(v, d) * (2.0 / math.sqrt(d))          # logits of a spread of about 2
        labels = torch.randint(0, v, (n,), generator=g, device=dev)
        h = normal(n, d) + 2.0 * torch.rand(n, 1, generator=g, device=dev) * w[labels]   # and the label's above them
        s["h"], s["w"] = h.to(dt), w.to(dt)
        del h, w
        # a run of tokens that carry no loss (a prompt, or padding)
        quiet = (torch.arange(n, device=dev) % 16 == 5) if n > 8 else torch.zeros(n, dtype=torch.bool, device=dev)
        s["labels"] = torch.where(quiet, IGNORE, labels)
        if op == "ce_bwd":
            step = max(1, (1 << 29) // v)
            s["lse"] = torch.cat([torch.logsumexp(s["h"][i:i + step].float() @ s["w"].float().T, 1) for i in range(0, n, step)])
            s["stats"] = torch.stack([s["lse"].new_tensor(0.0), (s["labels"] != IGNORE).sum().float()])
            s["row_grad"] = torch.rand(n, generator=g, device=dev) / n if case["grad"] == "rows" else None
    else:
        sizes = _adam_sizes(case)
        at = _starts(sizes)
        s["sizes"], s["at"], s["t"] = sizes, at, 100
        pt, gt = TYPES[case["dtype"]], TYPES[case["gdtype"]]
        s["P"] = [(normal(n) * 0.02).to(pt) for n in sizes]
        s["G"] = [(normal(n) * 1e-3).to(gt) for n in sizes]
        total = at[-1]
        s["real"] = torch.cat([torch.arange(b - a, device=dev) < n for a, b, n in zip(at, at[1:], sizes)])
        key = torch.zeros(total, dtype=torch.int64, device=dev)
        s["m"], s["ms"] = _encode_m(torch.where(s["real"], normal(total) * 3e-4, 0.0), key)
        s["v"], s["vs"] = _encode_v(torch.where(s["real"], (normal(total).square() + 0.05) * 1e-6, 0.0), key)
        if own:
            import matrix_aware_optimizer_muon_gb300 as mm
            s["opt"] = mm.AdamW8(s["P"], lr=LR, betas=(B1, B2), eps=ADAM_EPS, weight_decay=WD, seed=SEED)
            s["opt"].load_state_dict({"step": s["t"], "seed": SEED, "m": s["m"], "v": s["v"], "m_scale": s["ms"], "v_scale": s["vs"]})
            del s["m"], s["v"], s["ms"], s["vs"], s["real"]
    if own and op == "norm_bwd":
        import matrix_aware_optimizer_muon_gb300 as mm
        s["ws"] = mm.alloc_layernorm_workspace(case["rows"], case["dim"])
    if own and op.startswith("ce"):
        import matrix_aware_optimizer_muon_gb300 as mm
        s["ws"] = mm.alloc_linear_ce_workspace(case["rows"], case["vocab"], case["dim"], s["h"].dtype, backward=op == "ce_bwd")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import matrix_aware_optimizer_muon_gb300 as mm
        if op == "norm_fwd":
            return mm.muon_layernorm_forward(s["x"], s["w"], s["b"], eps=EPS)
        if op == "norm_bwd":
            dx, dw, db = mm.muon_layernorm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["ws"], bias=s["b"] is not None)
            return dx, dw, db
        if op == "ce_fwd":
            return mm.muon_linear_ce_forward(s["h"], s["w"], s["labels"], s["ws"], ignore_index=IGNORE)
        if op == "ce_bwd":
            return mm.muon_linear_ce_backward(s["h"], s["w"], s["labels"], s["lse"], s["ws"], row_grad=s["row_grad"],
                                              stats=None if s["row_grad"] is not None else s["stats"], ignore_index=IGNORE)
        s["opt"].step(s["G"])
        m, v = s["opt"].moments()
        return {"P": s["P"], "m": m, "v": v}
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "ce_fwd": _ce_fwd, "ce_bwd": _ce_bwd, "adam": _adam}[op](s)


def _norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(c.square().mean(1) + EPS)
    y = c * rstd[:, None]
    if s["w"] is not None:
        y = y * s["w"].float() + s["b"].float()
    return y.to(s["x"].dtype), mean, rstd


def _norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy if s["w"] is None else dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["w"] is None:
        return dx.to(s["x"].dtype), None, None
    return dx.to(s["x"].dtype), (dy * xh).sum(0).to(s["w"].dtype), dy.sum(0).to(s["b"].dtype)


def _ce_fwd(s):
    logits = s["h"].float() @ s["w"].float().T
    top = logits.max(1).values
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    counted = s["labels"] != IGNORE
    own_logit = logits.gather(1, s["labels"].clamp(min=0)[:, None])[:, 0]
    loss = torch.where(counted, lse - own_logit, 0.0)
    count = counted.sum().float()
    return loss, lse, torch.stack([loss.sum() / count.clamp(min=1.0), count])


def _ce_bwd(s):
    h, w = s["h"].float(), s["w"].float()
    counted = s["labels"] != IGNORE
    coef = s["row_grad"] if s["row_grad"] is not None else torch.ones_like(s["lse"]) / s["stats"][1].clamp(min=1.0)
    coef = torch.where(counted, coef, 0.0)
    p = torch.exp(h @ w.T - s["lse"][:, None])
    at = torch.arange(p.shape[0], device=p.device)
    p[at, s["labels"].clamp(min=0)] -= 1.0
    p *= coef[:, None]
    return (p @ w).to(s["h"].dtype), (p.T @ h).to(s["w"].dtype)


# The 8-bit moments.  Elements of a block of 128 share a scale byte s.  A code c > 0 of the
# first moment (sign and 7 bits) or the second (8 bits) stands for the number whose 32-bit
# float bits are (c + base) << 20, base = 8 * max(s - 16, 0) or 8 * max(s - 32, 0): three
# bits of mantissa, 15.9 or 31.9 powers of two in a block; c = 0 stands for zero.
def _mix(x):
    x = x ^ (x >> 16)
    x = (x * MIX1) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * MIX2) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(total, t, dev):
    """32 random bits for every element, from the seed, the step and the element's index."""
    key = _mix(torch.tensor(SEED, device=dev) ^ _mix(torch.tensor(t, device=dev)))
    at = torch.arange(total, device=dev)
    return _mix((at & 0xFFFFFFFF) ^ _mix((key + (at >> 32)) & 0xFFFFFFFF))


def _scale(bits):
    top = bits.view(-1, BLOCK).max(1).values >> 20
    return ((top + 9) >> 3).clamp(max=255)


def _encode_m(m, r):
    r = (r & 0xFFFF).to(torch.int32)
    bits = m.view(torch.int32) & 0x7FFFFFFF
    s = _scale(bits)
    base = (8 * (s - 16).clamp(min=0)).repeat_interleave(BLOCK)
    least = ((base + 1) << 20).view(torch.float32)
    small = bits < ((base + 1) << 20)
    code = torch.where(small, (((r.float() + 0.5) * 2.0 ** -16) * least < m.abs()).to(torch.int32), ((bits + (r << 4) + 8) >> 20) - base)
    code = code.clamp(max=127)
    code = torch.where((m < 0) & (code > 0), code | 128, code)
    return code.to(torch.uint8), s.to(torch.uint8)


def _encode_v(v, r):
    r = (r >> 16).to(torch.int32)
    bits = v.view(torch.int32)
    s = _scale(bits)
    base = (8 * (s - 32).clamp(min=0)).repeat_interleave(BLOCK)
    code = torch.minimum(((bits + (r << 4) + 8) >> 20) - base, torch.full_like(bits, 255))
    code = torch.maximum(code, (bits > 0).to(torch.int32))
    return code.to(torch.uint8), s.to(torch.uint8)


def _decode_m(code, s):
    c, base = code.to(torch.int32), (8 * (s.to(torch.int32) - 16).clamp(min=0)).repeat_interleave(BLOCK)
    size = (((c & 127) + base) << 20).view(torch.float32)
    return torch.where((c & 127) == 0, torch.where(c == 128, math.nan, 0.0), torch.where(c > 127, -size, size))


def _decode_v(code, s):
    c, base = code.to(torch.int32), (8 * (s.to(torch.int32) - 32).clamp(min=0)).repeat_interleave(BLOCK)
    return torch.where(c == 0, 0.0, ((c + base) << 20).view(torch.float32))


def _flat(s, tensors):
    """The tensors one after another in 32 bits, each from a block's first element."""
    pad = [b - a - n for a, b, n in zip(s["at"], s["at"][1:], s["sizes"])]
    zero = torch.zeros(BLOCK, device=tensors[0].device)
    return torch.cat([x for t, k in zip(tensors, pad) for x in (t.float(), zero[:k])])


def _adam(s):
    s["t"] += 1
    t = s["t"]
    p, g = _flat(s, s["P"]), _flat(s, s["G"])
    m = B1 * _decode_m(s["m"], s["ms"]) + (1.0 - B1) * g
    v = B2 * _decode_v(s["v"], s["vs"]) + (1.0 - B2) * g * g
    p = p - LR * ((m / (1.0 - B1 ** t)) / (torch.sqrt(v) * (1.0 / math.sqrt(1.0 - B2 ** t)) + ADAM_EPS) + WD * p)
    r = _random(p.numel(), t, p.device)
    s["m"], s["ms"] = _encode_m(torch.where(s["real"], m, 0.0), r)
    s["v"], s["vs"] = _encode_v(torch.where(s["real"], v, 0.0), r)
    torch._foreach_copy_(s["P"], [p[a:a + n] for a, n in zip(s["at"], s["sizes"])])
    return {"P": s["P"], "m": _decode_m(s["m"], s["ms"]).to(torch.bfloat16), "v": _decode_v(s["v"], s["vs"]).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op.startswith("norm"):
        x = s["x"].double()
        w = None if s["w"] is None else s["w"].double()
        if op == "norm_fwd":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + EPS).rsqrt()
            y = (x - mean[:, None]) * rstd[:, None]
            return (y if w is None else torch.addcmul(s["b"].double(), y, w)), mean, rstd
        # dx is the product of dy with the Jacobian r (I - 11'/D - xh xh'/D) W of the rows
        dy, mean, r, d = s["dy"].double(), s["mean"].double(), s["rstd"].double(), case["dim"]
        xh = (x - mean[:, None]) * r[:, None]
        g = dy if w is None else dy * w
        dx = (g - (g.sum(1) / d)[:, None] - torch.einsum("nd,nd->n", g, xh)[:, None] * xh / d) * r[:, None]
        if w is None:
            return dx, None, None
        return dx, torch.einsum("nd,nd->d", dy, xh), dy.sum(0)
    if op.startswith("ce"):
        n, d, v = case["rows"], case["dim"], case["vocab"]
        if (2 if op == "ce_fwd" else 6) * n * d * v > 6e12:
            return None
        labels = s["labels"]
        loss = torch.zeros(n, dtype=torch.float64, device=labels.device)
        lse = torch.zeros_like(loss)
        dh = torch.zeros(n, d, dtype=torch.float64, device=labels.device) if op == "ce_bwd" else None
        w = s["w"].double()
        dw = torch.zeros_like(w) if op == "ce_bwd" else None
        counted = (labels != IGNORE).double()
        step = max(1, (1 << 28) // v)
        for i in range(0, n, step):
            h, lab = s["h"][i:i + step].double(), labels[i:i + step]
            logits = h @ w.T
            if op == "ce_fwd":
                lse[i:i + step] = torch.logsumexp(logits, 1)
                loss[i:i + step] = torch.nn.functional.cross_entropy(logits, lab, reduction="none", ignore_index=IGNORE)
                continue
            c = counted[i:i + step] * (s["row_grad"][i:i + step].double() if s["row_grad"] is not None else 1.0 / counted.sum())
            gl = c[:, None] * torch.exp(logits - s["lse"][i:i + step].double()[:, None])
            gl.scatter_add_(1, lab.clamp(min=0)[:, None], -c[:, None])
            dh[i:i + step] = gl @ w
            dw.addmm_(gl.T, h)
        if op == "ce_bwd":
            return dh, dw
        return loss, lse, torch.stack([loss.sum() / counted.sum().clamp(min=1.0), counted.sum()])
    # the moments' codes: in 64 bits a number a is 2^e f, and its place on the grid of eight
    # steps a binade is 8 (e + 127) + 8 (f - 1), rounded down after the random part is added
    t = s["t"] + 1
    m0, v0 = _decode_m(s["m"], s["ms"]).double(), _decode_v(s["v"], s["vs"]).double()
    p, g = _flat(s, s["P"]).double(), _flat(s, s["G"]).double()
    m, v = m0.lerp(g, 1.0 - B1), v0.lerp(g.square(), 1.0 - B2)
    p = p * (1.0 - LR * WD) - LR * (m / (1.0 - B1 ** t)) / ((v / (1.0 - B2 ** t)).sqrt() + ADAM_EPS)
    r = _random(p.numel(), t, p.device)
    real = s["real"].double()
    out = {"P": [p[a:a + n] for a, n in zip(s["at"], s["sizes"])]}
    for name, x, bits, codes, binades in (("m", m * real, r & 0xFFFF, 127, 16), ("v", v * real, r >> 16, 255, 32)):
        f, e = torch.frexp(x.abs())
        place = torch.where(x == 0, 0.0, torch.where(e > -126, 8.0 * (e + 126) + 8.0 * (2.0 * f - 1.0), x.abs() * 2.0 ** 129))
        top = place.view(-1, BLOCK).max(1).values.floor()
        base = (8.0 * (torch.clamp(torch.floor((top + 9) / 8), max=255) - binades).clamp(min=0)).repeat_interleave(BLOCK)
        up = (bits.double() * 16 + 8) / 2.0 ** 20

        def value(q):
            return torch.where(q < 8, q * 2.0 ** -129, (1.0 + (q % 8) / 8) * torch.exp2(torch.floor(q / 8) - 127))

        code = torch.clamp(torch.floor(place + up) - base, max=codes)
        if name == "m":
            code = torch.where(place < base + 1, ((bits.double() + 0.5) / 65536 * value(base + 1) < x.abs()).double(), code)
        else:
            code = torch.maximum(code, (x > 0).double())
        out[name] = torch.where(code > 0, value(code + base) * torch.sign(x), 0.0)
    return out


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4, "none": 0}
    if op.startswith("norm"):
        n, d, es, ws = case["rows"], case["dim"], size[case["dtype"]], size[case["affine"]]
        if op == "norm_fwd":
            return {"bytes": 2 * n * d * es + 8 * n + 2 * d * ws, "flops": 8 * n * d}
        return {"bytes": 3 * n * d * es + 8 * n + 3 * d * ws, "flops": 14 * n * d}
    if op.startswith("ce"):
        n, d, v, es = case["rows"], case["dim"], case["vocab"], size[case["dtype"]]
        if op == "ce_fwd":
            return {"bytes": (n + v) * d * es + 16 * n, "flops": 2 * n * d * v}
        return {"bytes": 2 * (n + v) * d * es + 16 * n, "flops": 6 * n * d * v}
    n = sum(_adam_sizes(case))
    # parameter and codes read and written, gradient read, the moments' values (16 bits) written
    return {"bytes": n * (2 * size[case["dtype"]] + size[case["gdtype"]] + 4 + 4) + 4 * n // BLOCK, "flops": 20 * n}
