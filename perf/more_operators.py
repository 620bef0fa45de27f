"""Cases for the operators around a language model's head that scoring and policy-gradient
training need: the root-mean-square norm with the residual's addition (and an output in 8
bits), the log probabilities of given tokens with entropy and top alternatives, and the
global norm of all gradients with clipping.

Each case is one pass of one operator.  `run` computes it in plain torch operations in 32
bits (64 where alternatives are ranked and where gradients' squares are summed), or, with
`own` set, through the package's entry points; `exact` gives the same outputs from the
definition in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-6
GROUP = 128                  # columns that share one scale of the 8-bit output
E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -100
SPARE = 16                   # alternatives that are ranked in 64 bits beside the wanted ones
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST_NORM = 32768 * 1536     # elements of the largest listed norm
MOST_HEAD = 8192 * 2560 * 131072
MOST_CLIP = 12 * 12 * 1536 * 1536


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def listed():
    return [
        # a decoding step's sixteen tokens through one norm behind a residual: launch latency
        {"name": "rms_fwd_16tok", "op": "rms_fwd", "rows": 16, "dim": 2560, "dtype": "bf16", "weight": "f32",
         "residual": True, "eight": False, "pad": 0},
        # a training micro-batch, the norm's output in 8 bits for the product that follows
        {"name": "rms_fwd8_32k", "op": "rms_fwd", "rows": 32768, "dim": 1536, "dtype": "bf16", "weight": "bf16",
         "residual": True, "eight": True, "pad": 0},
        # its backward pass: the norm's gradient joins the residual stream's
        {"name": "rms_bwd_32k", "op": "rms_bwd", "rows": 32768, "dim": 1536, "dtype": "bf16", "weight": "f32",
         "residual": True, "pad": 0},
        # an odd width in 32 bits, rows cut out of a wider buffer, no residual
        {"name": "rms_bwd_odd", "op": "rms_bwd", "rows": 5003, "dim": 1537, "dtype": "f32", "weight": "f32",
         "residual": False, "pad": 3},
        # a decoding step of eight sequences: the chosen tokens' log probabilities and eight alternatives
        {"name": "logp_fwd_8tok", "op": "logp_fwd", "rows": 8, "dim": 1536, "vocab": 32768, "dtype": "bf16", "top": 8},
        # scoring a ragged batch over an odd vocabulary, with five alternatives
        {"name": "logp_fwd_odd", "op": "logp_fwd", "rows": 1021, "dim": 1536, "vocab": 50257, "dtype": "bf16", "top": 5},
        # the log probabilities and entropies of a policy's micro-batch over a large vocabulary
        {"name": "logp_fwd_8k", "op": "logp_fwd", "rows": 8192, "dim": 2560, "vocab": 131072, "dtype": "bf16", "top": 0},
        # its policy gradient, with an entropy bonus
        {"name": "logp_bwd_8k", "op": "logp_bwd", "rows": 8192, "dim": 2560, "vocab": 131072, "dtype": "bf16", "grad": "both"},
        # a small model trained in 32 bits, every size odd
        {"name": "logp_bwd_f32", "op": "logp_bwd", "rows": 1021, "dim": 1001, "vocab": 10007, "dtype": "f32", "grad": "logprob"},
        # the gradients of a model's norms: many small tensors, launch latency
        {"name": "clip_norms", "op": "clip", "tensors": 48, "small": 1536, "large": 0, "dtype": "f32", "clip": True},
        # the matrices of twelve transformer blocks of width 1536 (each 12 * 1536^2 elements in four)
        {"name": "clip_blocks", "op": "clip", "tensors": 48, "small": 3 * 1536 * 1536, "large": 0, "dtype": "bf16", "clip": True},
        # a vocabulary matrix's gradient in 32 bits beside small ones in 16, odd sizes
        {"name": "clip_mixed_odd", "op": "clip", "tensors": 25, "small": 1537, "large": 50257 * 769, "dtype": "mixed", "clip": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "logp_fwd", "logp_bwd", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("rms"):
        dim = _log(rng, 64, 16384)
        dim = dim if rng.random() < 0.4 else dim // 8 * 8
        most = MOST_NORM // (dim if dtype == "bf16" else 2 * dim)
        case = {"op": op, "rows": _log(rng, 1, max(1, min(65536, most))), "dim": dim, "dtype": dtype,
                "weight": rng.choice(["bf16", "f32", "none"]), "residual": rng.random() < 0.6, "pad": rng.choice([0, 0, 8, 5])}
        return {**case, "eight": rng.random() < 0.5} if op == "rms_fwd" else case
    if op.startswith("logp"):
        dim = _log(rng, 32, 4096)
        dim = dim if rng.random() < 0.3 else max(32, dim // 64 * 64)
        vocab = _log(rng, 1000, 131072)
        most = MOST_HEAD // 8 if dtype == "f32" else MOST_HEAD
        rows = _log(rng, 1, max(1, min(8192, most // (dim * vocab))))
        case = {"op": op, "rows": rows, "dim": dim, "vocab": vocab, "dtype": dtype}
        if op == "logp_bwd":
            return {**case, "grad": rng.choice(["both", "both", "logprob"])}
        top = rng.choice([0, 1, 5, 8, 20])
        return {**case, "top": top if rows * dim * (top + SPARE) < 1 << 30 else 0}
    tensors = rng.randint(1, 60)
    large = _log(rng, 1000, MOST_CLIP // 4)
    return {"op": "clip", "tensors": tensors, "small": _log(rng, 1, MOST_CLIP // 4 // tensors), "large": large,
            "dtype": rng.choice(["bf16", "f32", "mixed"]), "clip": rng.random() < 0.7}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _clip_sizes(case):
    n = case["tensors"] - (1 if case["large"] else 0)
    return ([case["large"]] if case["large"] else []) + [case["small"] + (7 * (i % 3) if case["small"] % 2 else 0) for i in range(n)]


def _clip_types(case):
    n = len(_clip_sizes(case))
    return [TYPES["f32" if i % 3 == 0 else "bf16"] for i in range(n)] if case["dtype"] == "mixed" else [TYPES[case["dtype"]]] * n


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    s = {"case": case}
    op = case["op"]
    if op.startswith("rms"):
        n, d, dt = case["rows"], case["dim"], TYPES[case["dtype"]]
        # a residual stream with a scale for every channel and a few large channels, and a
        # block's output that is added to it
        scale = 0.5 + torch.rand(d, generator=g, device=dev) + 8.0 * (torch.rand(d, generator=g, device=dev) < 0.002)
        stream = normal(n, d + case["pad"])
        stream[:, :d] *= scale
        stream = stream.to(dt)[:, :d]
        s["w"] = None if case["weight"] == "none" else (1.0 + 0.2 * normal(d)).to(TYPES[case["weight"]])
        if op == "rms_fwd":
            s["x"], s["r"] = ((normal(n, d + case["pad"]) * 0.3).to(dt)[:, :d], stream) if case["residual"] else (stream, None)
        else:
            s["total"] = stream
            s["rstd"] = 1.0 / torch.sqrt(stream.float().square().mean(1) + EPS)
            s["dy"] = (normal(n, d) * 1e-2).to(dt)
            s["dtotal"] = (normal(n, d) * 1e-2).to(dt) if case["residual"] else None
            if own:
                import matrix_aware_optimizer_muon_gb300 as mm
                s["ws"] = mm.alloc_rmsnorm_workspace(n, d) if s["w"] is not None else None
    elif op.startswith("logp"):
        n, d, v, dt = case["rows"], case["dim"], case["vocab"], TYPES[case["dtype"]]
        w = normal(v, d) * (2.0 / math.sqrt(d))          # logits of a spread of about 2
        tokens = torch.randint(0, v, (n,), generator=g, device=dev)
        h = normal(n, d) + 2.0 * torch.rand(n, 1, generator=g, device=dev) * w[tokens]   # and the token's above them
        s["h"], s["w"] = h.to(dt), w.to(dt)
        del h, w
        # tokens of a prompt, which the policy did not choose
        quiet = (torch.arange(n, device=dev) % 16 == 5) if n > 8 else torch.zeros(n, dtype=torch.bool, device=dev)
        s["tokens"] = torch.where(quiet, IGNORE, tokens)
        if op == "logp_bwd":
            step = max(1, (1 << 28) // v)
            parts = [_statistics(s["h"][i:i + step].float() @ s["w"].float().T) for i in range(0, n, step)]
            s["lse"], s["entropy"] = (torch.cat(p) for p in zip(*parts))
            s["entropy"] = torch.where(quiet, 0.0, s["entropy"])
            s["g_logprob"] = normal(n) / n               # advantages
            s["g_entropy"] = torch.full((n,), 0.01 / n, device=dev) if case["grad"] == "both" else None
        if own:
            import matrix_aware_optimizer_muon_gb300 as mm
            s["ws"] = mm.alloc_linear_logprob_workspace(n, v, d, dt, top=case.get("top", 0), backward=op == "logp_bwd")
    else:
        # gradients of different sizes from tensor to tensor
        s["G"] = [(normal(n) * (1e-3 * (1 + i % 5))).to(t) for i, (n, t) in enumerate(zip(_clip_sizes(case), _clip_types(case)))]
        norm = math.sqrt(sum(float(t.double().square().sum()) for t in s["G"]))
        s["most"] = norm * (0.5 if case["clip"] else 2.0)
        if own:
            import matrix_aware_optimizer_muon_gb300 as mm
            s["ws"] = mm.alloc_clip_workspace()
    return s


def _statistics(logits):
    """(log-sum-exp, entropy) of every row."""
    top = logits.max(1, keepdim=True).values
    d = logits - top
    e = torch.exp(d)
    total = e.sum(1)
    return top[:, 0] + torch.log(total), torch.log(total) - (e * d).sum(1) / total


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if op == "clip" and s["case"]["clip"]:
        s["most"] *= 0.999       # so that every pass over the same gradients has to scale them
    if own:
        import matrix_aware_optimizer_muon_gb300 as mm
        if op == "rms_fwd" and s["case"]["eight"]:
            codes, scales, rstd, total = mm.muon_rmsnorm_forward_fp8(s["x"], s["w"], s["r"], eps=EPS)
            return {"codes": codes, "scales": scales, "rstd": rstd, "total": None if s["r"] is None else total}
        if op == "rms_fwd":
            y, rstd, total = mm.muon_rmsnorm_forward(s["x"], s["w"], s["r"], eps=EPS)
            return {"y": y, "rstd": rstd, "total": None if s["r"] is None else total}
        if op == "rms_bwd":
            return mm.muon_rmsnorm_backward(s["dy"], s["total"], s["w"], s["rstd"], s["ws"], dtotal=s["dtotal"])
        if op == "logp_fwd":
            return mm.muon_linear_logprob_forward(s["h"], s["w"], s["tokens"], s["ws"], top=s["case"]["top"], ignore_index=IGNORE)
        if op == "logp_bwd":
            return mm.muon_linear_logprob_backward(s["h"], s["w"], s["tokens"], s["lse"], s["entropy"], s["ws"],
                                                   s["g_logprob"], s["g_entropy"], ignore_index=IGNORE)
        return mm.muon_clip_grad_norm(s["G"], s["most"], s["ws"]), s["G"]
    return {"rms_fwd": _rms_fwd, "rms_bwd": _rms_bwd, "logp_fwd": _logp_fwd, "logp_bwd": _logp_bwd, "clip": _clip}[op](s)


def _grouped(y):
    """Columns in groups of 128, zeros behind the last."""
    n, d = y.shape
    k = -(-d // GROUP)
    return torch.nn.functional.pad(y, (0, k * GROUP - d)).view(n, k, GROUP)


def _rms_fwd(s):
    x = s["x"]
    # the residual stream is kept in the inputs' type, and its rounded value is what is normed
    total = x if s["r"] is None else (x.float() + s["r"].float()).to(x.dtype)
    t = total.float()
    rstd = 1.0 / torch.sqrt(t.square().mean(1) + EPS)
    y = t * rstd[:, None]
    if s["w"] is not None:
        y = y * s["w"].float()
    out = {"rstd": rstd, "total": None if s["r"] is None else total}
    if not s["case"]["eight"]:
        return {"y": y.to(x.dtype), **out}
    k = _grouped(y)
    scale = (k.abs().amax(2) / E4M3_MAX).clamp(min=LEAST_SCALE)
    q = (k / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(x.shape[0], -1)[:, :x.shape[1]]
    return {"codes": q.to(torch.float8_e4m3fn), "scales": scale, **out}


def _rms_bwd(s):
    dy, r = s["dy"].float(), s["rstd"][:, None]
    xh = s["total"].float() * r
    g = dy if s["w"] is None else dy * s["w"].float()
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    return dx.to(s["dy"].dtype), None if s["w"] is None else (dy * xh).sum(0).to(s["w"].dtype)


def _logp_fwd(s):
    h, w, k = s["h"], s["w"], s["case"]["top"]
    logits = h.float() @ w.float().T
    lse, entropy = _statistics(logits)
    counted = s["tokens"] != IGNORE
    chosen = logits.gather(1, s["tokens"].clamp(min=0)[:, None])[:, 0]
    logprob, entropy = torch.where(counted, chosen - lse, 0.0), torch.where(counted, entropy, 0.0)
    if k == 0:
        return logprob, entropy, lse, None, None
    # logits next to each other are ranked in 64 bits, equal ones by their index
    ids = logits.topk(k + SPARE, 1).indices.sort(1).values
    z = (h.double()[:, None, :] @ w[ids].double().transpose(1, 2))[:, 0, :]
    z, at = z.sort(dim=1, descending=True, stable=True)
    ids = torch.where(counted[:, None], ids.gather(1, at)[:, :k], -1)
    alternatives = torch.where(counted[:, None], z[:, :k] - lse.double()[:, None], -math.inf)
    return logprob, entropy, lse, ids, alternatives.float()


def _logp_bwd(s):
    h, w = s["h"].float(), s["w"].float()
    counted = s["tokens"] != IGNORE
    a = torch.where(counted, s["g_logprob"], 0.0)
    logp = h @ w.T - s["lse"][:, None]
    p = torch.exp(logp)
    if s["g_entropy"] is None:
        g = -a[:, None] * p
    else:
        b = torch.where(counted, s["g_entropy"], 0.0)
        g = -p * (a[:, None] + b[:, None] * (logp + s["entropy"][:, None]))
    at = torch.arange(p.shape[0], device=p.device)
    g[at, s["tokens"].clamp(min=0)] += a
    return (g @ w).to(s["h"].dtype), (g.T @ h).to(s["w"].dtype)


def _clip(s):
    grads = s["G"]
    flat = torch.cat([t.float() for t in grads])
    norm = torch.sqrt(flat.double().square().sum())
    flat = flat * torch.clamp(s["most"] / norm, max=1.0).float()
    pieces = list(zip(grads, flat.split([t.numel() for t in grads])))
    for dtype in {t.dtype for t in grads}:   # one call writes tensors of one type
        torch._foreach_copy_([t for t, _ in pieces if t.dtype == dtype], [p for t, p in pieces if t.dtype == dtype])
    return norm.float(), grads


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _e4m3(q):
    """The nearest number with a sign, 4 bits of exponent and 3 of mantissa, ties to even."""
    e = torch.frexp(q.abs()).exponent.clamp(min=-5) - 4
    return torch.ldexp(torch.round(torch.ldexp(q, -e)), e).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "rms_fwd":
        x = s["x"].double()
        total = x if s["r"] is None else x + s["r"].double()
        t = total.to(s["x"].dtype).double()
        rstd = (torch.einsum("nd,nd->n", t, t) / case["dim"] + EPS).rsqrt()
        y = torch.einsum("nd,n->nd", t, rstd)
        y = y if s["w"] is None else y * s["w"].double()
        out = {"rstd": rstd, "total": None if s["r"] is None else total}
        if not case["eight"]:
            return {"y": y, **out}
        k = _grouped(y)
        scale = torch.maximum(torch.linalg.vector_norm(k, math.inf, 2) / E4M3_MAX, torch.tensor(LEAST_SCALE, device=k.device))
        return {"codes": _e4m3(k / scale[:, :, None]).view(case["rows"], -1)[:, :case["dim"]], "scales": scale, **out}
    if op == "rms_bwd":
        # dx is the product of dy with the Jacobian r (I - xh xh'/D) W of the rows
        dy, r = s["dy"].double(), s["rstd"].double()
        xh = torch.einsum("nd,n->nd", s["total"].double(), r)
        g = dy if s["w"] is None else dy * s["w"].double()
        dx = torch.einsum("nd,n->nd", g - torch.einsum("nd,n->nd", xh, torch.einsum("nd,nd->n", g, xh) / case["dim"]), r)
        return dx if s["dtotal"] is None else dx + s["dtotal"].double(), None if s["w"] is None else torch.einsum("nd,nd->d", dy, xh)
    if op.startswith("logp"):
        n, d, v = case["rows"], case["dim"], case["vocab"]
        if (2 if op == "logp_fwd" else 6) * n * d * v > 6e12:
            return None
        w, tokens, k = s["w"].double(), s["tokens"], case.get("top", 0)
        step = max(1, (1 << 27) // v)
        rows, dw = [], torch.zeros_like(w) if op == "logp_bwd" else None
        for i in range(0, n, step):
            h, tok = s["h"][i:i + step].double(), tokens[i:i + step]
            counted, at = tok != IGNORE, tok.clamp(min=0)[:, None]
            logits = h @ w.T
            if op == "logp_fwd":
                lse = torch.logsumexp(logits, 1)
                logp = logits - lse[:, None]
                row = [torch.where(counted, logp.gather(1, at)[:, 0], 0.0),
                       torch.where(counted, torch.special.entr(torch.exp(logp)).sum(1), 0.0), lse]
                if k:
                    best, ids = logits.sort(dim=1, descending=True, stable=True)
                    row += [torch.where(counted[:, None], ids[:, :k], -1),
                            torch.where(counted[:, None], best[:, :k] - lse[:, None], -math.inf)]
                rows.append(row)
                continue
            # the Jacobians of log p[token] and of the entropy with respect to the logits
            logp = logits - s["lse"][i:i + step].double()[:, None]
            p = logp.exp()
            a = torch.where(counted, s["g_logprob"][i:i + step].double(), 0.0)[:, None]
            g = torch.zeros_like(p).scatter_(1, at, 1.0).sub_(p).mul_(a)
            if s["g_entropy"] is not None:
                b = torch.where(counted, s["g_entropy"][i:i + step].double(), 0.0)[:, None]
                g.sub_(b * p * logp).sub_(b * p * s["entropy"][i:i + step].double()[:, None])
            rows.append([g @ w])
            dw.addmm_(g.T, h)
        out = [torch.cat(x) for x in zip(*rows)]
        return (out[0], dw) if op == "logp_bwd" else (*out, *([None] * (5 - len(out))))
    most = s["most"] * (0.999 if case["clip"] else 1.0)
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(t.double()) for t in s["G"]]))
    coef = min(1.0, most / float(norm))
    return norm, [t.double() * coef for t in s["G"]]


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4, "none": 0}
    if op.startswith("rms"):
        n, d, es, ws = case["rows"], case["dim"], size[case["dtype"]], size[case["weight"]]
        if op == "rms_fwd":
            out = 1 + 4 / GROUP if case["eight"] else es
            return {"bytes": n * d * (es * (3 if case["residual"] else 1) + out) + 4 * n + d * ws, "flops": 6 * n * d}
        return {"bytes": n * d * es * (4 if case["residual"] else 3) + 4 * n + 2 * d * ws, "flops": 11 * n * d}
    if op.startswith("logp"):
        n, d, v, es = case["rows"], case["dim"], case["vocab"], size[case["dtype"]]
        if op == "logp_fwd":
            return {"bytes": (n + v) * d * es + 20 * n + 12 * n * case["top"], "flops": 2 * n * d * v}
        return {"bytes": 2 * (n + v) * d * es + 24 * n, "flops": 6 * n * d * v}
    n = sum(k * (2 if t == torch.bfloat16 else 4) for k, t in zip(_clip_sizes(case), _clip_types(case)))
    return {"bytes": n * (2 if case["clip"] else 1), "flops": 3 * sum(_clip_sizes(case))}
