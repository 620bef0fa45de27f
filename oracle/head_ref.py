"""Plain fp64 restatements of the head's operators: layer norm and RMS norm, linear cross
entropy and log probabilities, AdamW with 8-bit moments, clipping by the global norm.
Test infrastructure; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

BLOCK = 128
MIX1, MIX2 = 0x9E3779B9, 0x6A09E667


def layernorm_forward(x, w=None, b=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    y = y if w is None else y * np.asarray(w, np.float64)
    return (y if b is None else y + np.asarray(b, np.float64)), mean, rstd


def layernorm_backward(dy, x, w, mean, rstd):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    xh = (x - mean) * rstd
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def linear_ce_forward(h, w, labels, ignore_index=-100):
    """(loss, lse, mean over the rows that count, their number)."""
    z = np.asarray(h, np.float64) @ np.asarray(w, np.float64).T
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    labels = np.asarray(labels)
    loss = np.zeros(len(labels))
    for r, lab in enumerate(labels):
        if lab != ignore_index:
            loss[r] = lse[r] - z[r, lab] if 0 <= lab < z.shape[1] else np.nan
    counted = labels != ignore_index
    return loss, lse, loss[counted].sum() / max(counted.sum(), 1), int(counted.sum())


def linear_ce_logit_grad(h, w, labels, lse, coef, ignore_index=-100):
    z = np.asarray(h, np.float64) @ np.asarray(w, np.float64).T
    g = np.exp(z - np.asarray(lse, np.float64)[:, None])
    for r, lab in enumerate(np.asarray(labels)):
        if lab == ignore_index or not 0 <= lab < z.shape[1]:
            g[r] = 0.0
        else:
            g[r, lab] -= 1.0
            g[r] *= coef[r]
    return g


def linear_ce_backward(h, w, labels, lse, coef, ignore_index=-100):
    g = linear_ce_logit_grad(h, w, labels, lse, coef, ignore_index)
    return g @ np.asarray(w, np.float64), g.T @ np.asarray(h, np.float64)


def mix32(x):
    """32 random bits of a 32-bit counter."""
    x = np.asarray(x, np.uint64)
    mask = np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(MIX1)) & mask
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(MIX2)) & mask
    return x ^ (x >> np.uint64(16))


def random_bits(seed, t, index):
    key = mix32(np.uint64(seed) ^ mix32(np.uint64(t & 0xFFFFFFFF)))
    index = np.asarray(index, np.uint64)
    return mix32((index & np.uint64(0xFFFFFFFF)) ^ mix32((key + (index >> np.uint64(32))) & np.uint64(0xFFFFFFFF)))


def grid_value(q):
    """The number at place q >= 0 of the grid with eight steps a binade (linear below 2^-126)."""
    q = np.asarray(q, np.float64)
    return np.where(q < 8, q * 2.0 ** -129, (1 + (q % 8) / 8) * np.exp2(np.floor(q / 8) - 127))


def grid_place(a):
    """The real-valued place of a >= 0 on that grid."""
    a = np.asarray(a, np.float64)
    f, e = np.frexp(a)
    return np.where(a < 2.0 ** -126, a * 2.0 ** 129, 8.0 * (e + 126) + 8.0 * (2 * f - 1))


def quantise(x, bits, top_code, binades):
    """Stochastic rounding of whole blocks: (codes without sign, scale bytes, values, slack).
    slack: distance of an element's place (random part added) from the next rounding edge."""
    x = np.asarray(x, np.float64)
    place = grid_place(np.abs(x))
    scale = np.minimum(np.floor((np.floor(place.reshape(-1, BLOCK).max(1)) + 9) / 8), 255)
    base = np.repeat(8 * np.maximum(scale - binades, 0), BLOCK)
    moved = place + (np.asarray(bits, np.float64) * 16 + 8) / 2.0 ** 20
    code = np.floor(moved) - base
    slack = np.abs(moved - np.round(moved))
    if binades == 16:
        least, odds = grid_value(base + 1), (np.asarray(bits, np.float64) + 0.5) / 65536
        small = place < base + 1
        code = np.where(small, odds * least < np.abs(x), code)
        slack = np.where(small, np.abs(odds - np.abs(x) / least), slack)
    else:
        code = np.maximum(code, x > 0)
    code = np.clip(code, 0, top_code)
    return code, scale, np.where(code > 0, grid_value(code + base) * np.sign(x), 0.0), slack


def decode(codes, scales, signed):
    c = np.asarray(codes, np.int64)
    base = np.repeat(8 * np.maximum(np.asarray(scales, np.int64) - (16 if signed else 32), 0), BLOCK)
    k = c & 127 if signed else c
    v = np.where(k > 0, grid_value(k + base), 0.0)
    return np.where(c == 128, np.nan, np.where(c > 127, -v, v)) if signed else v


def adamw8_update(p, g, m, v, t, lr, beta1, beta2, eps, weight_decay):
    """New parameter and the new moments before they are rounded."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = p - lr * ((m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps) + weight_decay * p)
    return p, m, v


def rmsnorm_forward(t, w=None, eps=1e-6):
    t = np.asarray(t, np.float64)
    rstd = 1.0 / np.sqrt((t * t).mean(1) + eps)
    y = t * rstd[:, None]
    return (y if w is None else y * np.asarray(w, np.float64)), rstd


def rmsnorm_backward(dy, t, w, rstd, dtotal=None):
    dy, xh = np.asarray(dy, np.float64), np.asarray(t, np.float64) * np.asarray(rstd, np.float64)[:, None]
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dx = np.asarray(rstd, np.float64)[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    return (dx if dtotal is None else dx + np.asarray(dtotal, np.float64)), (dy * xh).sum(0)


def e4m3(q):
    """The nearest of the numbers with 4 bits of exponent and 3 of mantissa, ties to even."""
    q = np.asarray(q, np.float64)
    e = np.maximum(np.frexp(np.abs(q))[1], -5) - 4
    return np.clip(np.ldexp(np.round(np.ldexp(q, -e)), e), -448.0, 448.0)


def eight_bits(y, group=128):
    """(codes' values, scales) of rows in groups of columns."""
    y = np.asarray(y, np.float64)
    k = -(-y.shape[1] // group)
    p = np.zeros((y.shape[0], k * group))
    p[:, :y.shape[1]] = y
    scale = np.maximum(np.abs(p.reshape(-1, k, group)).max(2) / 448.0, 2.0 ** -100)
    return e4m3(p / np.repeat(scale, group, 1))[:, :y.shape[1]], scale


def logprobs(h, w, tokens, top=0, ignore_index=-100):
    """(logprob, entropy, lse, ids, alternatives) of the logits h w^T."""
    z = np.asarray(h, np.float64) @ np.asarray(w, np.float64).T
    n, v = z.shape
    m = z.max(1, keepdims=True)
    lse = m[:, 0] + np.log(np.exp(z - m).sum(1))
    p = np.exp(z - lse[:, None])
    entropy = -(p * np.where(p > 0, z - lse[:, None], 0.0)).sum(1)
    logprob = np.zeros(n)
    ids, alternatives = np.full((n, top), -1), np.full((n, top), -np.inf)
    for r in range(n):
        tok = None if tokens is None else int(tokens[r])
        if tok == ignore_index:
            entropy[r] = 0.0
            continue
        if tok is not None:
            logprob[r] = z[r, tok] - lse[r] if 0 <= tok < v else np.nan
            entropy[r] = entropy[r] if 0 <= tok < v else np.nan
        order = [c for c in np.argsort(-z[r], kind="stable") if z[r, c] > -np.inf][:top]
        ids[r, :len(order)] = order
        alternatives[r, :len(order)] = z[r, order] - lse[r]
    return logprob, entropy, lse, ids, alternatives


def logprob_logit_grad(h, w, tokens, lse, entropy, a, b, ignore_index=-100):
    """Gradient of sum_r a_r logprob_r + b_r entropy_r with respect to the logits."""
    logp = np.asarray(h, np.float64) @ np.asarray(w, np.float64).T - np.asarray(lse, np.float64)[:, None]
    p = np.exp(logp)
    g = np.zeros_like(p)
    for r, tok in enumerate(np.asarray(tokens)):
        if tok == ignore_index or not 0 <= tok < p.shape[1]:
            continue
        g[r] = -a[r] * p[r] - b[r] * p[r] * (np.where(p[r] > 0, logp[r], 0.0) + entropy[r])
        g[r, tok] += a[r]
    return g


def clip_grad_norm(grads, max_norm):
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    coef = max_norm / norm if norm > max_norm else 1.0
    return norm, [np.asarray(g, np.float64) * coef for g in grads]
