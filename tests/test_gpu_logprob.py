"""Log probabilities, entropies and alternatives on the GPU against the fp64 oracle.

Tolerances come from the arithmetic.  u = 2^-24 is fp32's rounding error, 2^-8 bf16's
half-spacing.  The tensor cores' fp32 accumulation is allowed twice fp32's rounding error for
each product of 16 terms; 32-bit operands come as three bf16 parts each, whose dropped
products are below 2^-23 of a whole one (allowed four times the error).  Exponentials are
within 4 ulp and their argument's rounding."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm
from oracle import head_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev():
    return torch.device("cuda:0")


def put(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype])
    return t.to(dev()), t.double().numpy()


def num(t):
    return t.double().cpu().numpy()


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300))))


def case(n, v, d, dt, seed):
    rng = np.random.default_rng(seed)
    w, w64 = put(rng.standard_normal((v, d)) * 2 / np.sqrt(d), dt)
    tok = rng.integers(0, v, n)
    h, h64 = put(rng.standard_normal((n, d)) + w64[tok], dt)
    tok[rng.random(n) < 0.2] = -100
    return h, h64, w, w64, torch.from_numpy(tok).to(dev()), tok


def errors(h64, w64, dt, rlse):
    """(a logit's error, the lse's, the entropy's), by row."""
    v, d = w64.shape
    z = h64 @ w64.T
    ez = ((1 if dt == "bf16" else 4) * (d / 16 + 16) * 2 * U) * (np.abs(h64) @ np.abs(w64).T).max(1)
    spread = np.abs(z).max(1) + 1
    elog = ez + (v / 32 + 64 + 4 * spread) * U + 4 * U * np.abs(rlse)
    # H = sum p (lse - z): p is within ez + elog, and so is lse - z
    p, far = np.exp(z - rlse[:, None]), np.abs(z - rlse[:, None])
    eh = (ez + elog + (v / 32 + 64 + 4 * spread) * U) * (1 + 2 * (p * far).sum(1)) + 8 * U * np.log(v + 1)
    return ez, elog, eh


def check(out, h64, w64, tok, top, dt, what):
    logprob, entropy, lse, ids, alternatives = out
    rlogp, rent, rlse, rids, ralt = ref.logprobs(h64, w64, tok, top)
    ez, elog, eh = errors(h64, w64, dt, rlse)
    within(num(lse), rlse, elog, ("lse",) + what)
    within(num(entropy), rent, eh, ("entropy",) + what)
    if tok is None:
        assert logprob is None
    else:
        within(num(logprob), rlogp, elog + ez + 2 * U * np.abs(rlse), ("logprob",) + what)
        assert np.all(num(logprob)[tok == -100] == 0) and np.all(num(entropy)[tok == -100] == 0)
    if top == 0:
        assert ids is None and alternatives is None
        return
    assert ids.dtype == torch.int64 and np.array_equal(ids.cpu().numpy(), rids), what
    got = num(alternatives)
    assert np.array_equal(np.isinf(got), np.isinf(ralt)) and np.all(got[np.isinf(got)] < 0)
    fine = np.isfinite(ralt)
    tol = (elog[:, None] + 2 * U * (np.abs(np.where(fine, ralt, 0)) + np.abs(rlse[:, None])))
    within(np.where(fine, got, 0), np.where(fine, ralt, 0), tol, ("alternatives",) + what)


SIZES = [(1, 1, 1), (1, 5, 8), (3, 2, 16), (2, 7, 3), (5, 100, 65), (8, 1000, 64), (16, 257, 72), (129, 255, 128),
         (128, 256, 64), (127, 300, 200), (257, 513, 96), (300, 1111, 321), (1, 5000, 256), (1000, 40, 40), (64, 9000, 130),
         (5, 70001, 72)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_logprobs(dt, size):
    n, v, d = size
    h, h64, w, w64, tokens, tok = case(n, v, d, dt, n + v + d)
    for top in (0, 1, 5, 32):
        ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=top, backward=False)
        out = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=top)
        assert mm.muon_check_status(ws) == mm.MUON_OK
        check(out, h64, w64, tok, top, dt, (n, v, d, top))
    none = mm.muon_linear_logprob_forward(h, w, None, ws, top=3)
    check(none, h64, w64, None, 3, dt, (n, v, d, "no tokens"))

    # gradients, from the kernel's own statistics
    _, entropy, lse, _, _ = out
    rng = np.random.default_rng(3)
    ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt])
    a, a64 = put(rng.standard_normal(n), "f32")
    b, b64 = put(rng.standard_normal(n), "f32")
    z = h64 @ w64.T
    lse64, ent64 = num(lse), num(entropy)
    ez, _, _ = errors(h64, w64, dt, lse64)
    spread = np.abs(z).max(1) + 1
    one = BF if dt == "bf16" else 0.0
    parts = 1 if dt == "bf16" else 4
    for ga, gb in ((a, b), (a, None), (None, b)):
        dh, dw = mm.muon_linear_logprob_backward(h, w, tokens, lse, entropy, ws, ga, gb)
        assert mm.muon_check_status(ws) == mm.MUON_OK
        c, e = (a64 if ga is not None else 0 * a64), (b64 if gb is not None else 0 * b64)
        g = ref.logprob_logit_grad(h64, w64, tok, lse64, ent64, c, e)
        p = np.exp(z - lse64[:, None]) * (tok != -100)[:, None]
        size_g = np.abs(c)[:, None] + np.abs(e)[:, None] * (np.abs(z - lse64[:, None]) + np.abs(ent64)[:, None])
        ep = p * (ez + (16 + 4 * spread) * U)[:, None]
        eg = ep * size_g + p * np.abs(e)[:, None] * ez[:, None] + 8 * U * p * size_g + 4 * U * np.abs(g) + \
            4 * U * (np.abs(c) * (tok != -100))[:, None]
        eg = eg + one * (np.abs(g) + eg)
        edh = eg @ np.abs(w64) + parts * (v / 16 + 64) * 2 * U * (np.abs(g) @ np.abs(w64))
        edw = eg.T @ np.abs(h64) + parts * (n / 16 + 64) * 2 * U * (np.abs(g).T @ np.abs(h64))
        within(num(dh), g @ w64, edh + one * (np.abs(g @ w64) + edh) + 1e-30, "dh")
        within(num(dw), g.T @ h64, edw + one * (np.abs(g.T @ h64) + edw) + 1e-30, "dw")
        assert not dh[tokens == -100].any()
    dh, dw = mm.muon_linear_logprob_backward(h, w, tokens, lse, None, ws)
    assert not dh.any() and not dw.any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_logprob_gradient_matches_differences(dt):
    n, v, d = 40, 333, 48
    h, h64, w, w64, tokens, tok = case(n, v, d, dt, 5)
    ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt])
    _, entropy, lse, _, _ = mm.muon_linear_logprob_forward(h, w, tokens, ws)
    rng = np.random.default_rng(1)
    (a, a64), (b, b64) = (put(rng.standard_normal(n) / n, "f32") for _ in range(2))
    dh, dw = mm.muon_linear_logprob_backward(h, w, tokens, lse, entropy, ws, a, b)

    def f(h, w):
        logp, ent, _, _, _ = ref.logprobs(h, w, tok)
        return (a64 * logp + b64 * ent).sum()

    for arg, grad, which in ((h64, num(dh), 0), (w64, num(dw), 1)):
        e = rng.standard_normal(arg.shape)
        step = 1e-4
        hi, lo = (f(*((arg + s * step * e, w64) if which == 0 else (h64, arg + s * step * e))) for s in (1, -1))
        # each entry is off by at most the rounding of g and of the result (two of 2^-8 in bf16)
        tol = (3 * BF if dt == "bf16" else 1e-5) * np.linalg.norm(grad) * np.linalg.norm(e) / np.sqrt(e.size) * 6 + 1e-6
        assert abs((hi - lo) / (2 * step) - (grad * e).sum()) < tol


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_alternatives_among_ties_and_near_ties(dt):
    """Equal logits go to the lower id, and those closer than the products' own error are
    ranked right, however many there are."""
    rng = np.random.default_rng(4)
    v, d = 3001, 136
    base = rng.standard_normal(d)
    near = base * (1 + rng.integers(-1, 2, (v, d)) * 2.0 ** -7 * (rng.random((v, d)) < 0.01))     # all within 1e-3 of each other
    some = rng.standard_normal((v, d)) * 0.1
    some[rng.permutation(v)[:40]] = base                                   # forty equal rows far above the rest
    twins = rng.standard_normal((v, d)) / np.sqrt(d)
    twins[1::2] = twins[0:-1:2]                                            # neighbours in pairs
    block = rng.standard_normal((v, d)) * 0.1
    block[320:352] = base * (1 + 2.0 ** -7 * rng.integers(0, 2, (32, d)))      # one group of 32 holds the best
    for w in (near, some, twins, block, np.zeros((v, d)), np.tile(base, (v, 1))):
        w, w64 = put(w, dt)
        h, h64 = put(np.stack([base, -base, np.zeros(d), rng.standard_normal(d), base * 1e-3]), dt)
        z = h64 @ w64.T
        ws = mm.alloc_linear_logprob_workspace(len(h64), v, d, TYPES[dt], top=32, backward=False)
        for top in (1, 8, 32):
            _, _, _, ids, alternatives = mm.muon_linear_logprob_forward(h, w, None, ws, top=top)
            got = ids.cpu().numpy()
            for r in range(len(z)):
                assert len(set(got[r])) == top and got[r].min() >= 0
                # in order, by the exact logits; rows of one value lower ids first
                zr, best = z[r][got[r]], np.sort(z[r])[::-1][:top]
                assert np.all(np.abs(zr - best) <= 2.0 ** -40 * np.abs(h64[r]) @ np.abs(w64).max(0)), (r, top)
            same = (np.abs(w64 - w64[:1]).max() == 0) or not np.any(h64[2])
            if same:
                assert np.array_equal(got[2], np.arange(top))
            if np.abs(w64 - w64[:1]).max() == 0:
                assert np.array_equal(got, np.tile(np.arange(top), (len(h64), 1)))
    # equal rows exactly: the lowest ids of them, in order
    w, w64 = put(some, dt)
    h, _ = put(base[None], dt)
    _, _, _, ids, _ = mm.muon_linear_logprob_forward(h, w, None, ws, top=32)
    want = np.flatnonzero((w64 == put(base[None], dt)[1]).all(1))[:32]
    assert np.array_equal(ids.cpu().numpy()[0], want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mask", ["lowest", "minus infinity"])
def test_masked_vocabulary(dt, mask):
    """A bias column masks entries: probability 0, no alternatives, and no gradient from them;
    a row whose every entry is masked has nothing."""
    n, v, d = 9, 700, 64
    h, h64, w, w64, tokens, tok = case(n, v, d, dt, 8)
    low = -np.inf if mask == "minus infinity" else float(torch.finfo(TYPES[dt]).min)
    allowed = np.arange(v) % 3 == 1
    allowed[300:] = False                    # whole tiles and groups masked
    h64[:, 0], w64[:, 0] = 1.0, 0.0
    keep = w64.copy()
    w64[~allowed, 0] = low
    h, _ = put(h64, dt)
    w, _ = put(w64, dt)
    tok = np.where(tok >= 0, (tok % 100) * 3 + 1, tok)
    tokens = torch.from_numpy(tok).to(dev())
    ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=32)
    out = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=32)
    few = keep[allowed]
    back = np.searchsorted(np.flatnonzero(allowed), np.where(tok < 0, 1, tok))
    logp, ent, lse, ids, alt = ref.logprobs(h64, few, np.where(tok < 0, -100, back), 32)
    ez, elog, eh = errors(h64, few, dt, lse)
    within(num(out[0]), logp, 2 * elog + ez, "logprob")
    within(num(out[1]), ent, 2 * eh, "entropy")
    where = np.where(ids >= 0, np.flatnonzero(allowed)[ids], -1)
    assert np.array_equal(out[3].cpu().numpy(), where)
    a = torch.ones(n, device=dev())
    if mask == "lowest":          # (minus infinity times a gradient of 0 is NaN in any product with W)
        dh, dw = mm.muon_linear_logprob_backward(h, w, tokens, out[2], out[1], ws, a, a)
        assert torch.isfinite(dw).all() and not dw[torch.from_numpy(~allowed).to(dev())].any()
    # fewer entries than alternatives, then none
    w64[:, 0] = low
    w64[5, 0], w64[600, 0] = 0.0, 0.0
    w, _ = put(w64, dt)
    _, ent, lse, ids, alt = mm.muon_linear_logprob_forward(h, w, None, ws, top=4)
    assert torch.isfinite(ent).all() and torch.isfinite(lse).all()
    assert bool(((ids[:, :2] == 5) | (ids[:, :2] == 600)).all()) and bool((ids[:, 2:] == -1).all())
    assert torch.isfinite(alt[:, :2]).all() and bool((alt[:, 2:] == -float("inf")).all())
    if mask == "minus infinity":
        w64[:, 0] = low
        w, _ = put(w64, dt)
        logp, ent, lse, ids, alt = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=4)
        assert bool((lse == -float("inf")).all()) and bool((ids == -1).all()) and bool((alt == -float("inf")).all())
        live = tokens != -100
        assert torch.isnan(logp[live]).all() and torch.isnan(ent[live]).all() and not logp[~live].any() and not ent[~live].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("top", [0, 5])
def test_nan_and_infinite_logits(bad, top):
    n, v, d = 6, 600, 32
    h, h64, w, w64, tokens, tok = case(n, v, d, "bf16", 3)
    tokens = torch.arange(n, device=dev())
    w = w.clone()
    w[:, 0] = 0
    w[450, 0] = 1
    h = h.clone()
    h[2, 0] = bad
    ws = mm.alloc_linear_logprob_workspace(n, v, d, top=top, backward=False)
    logp, ent, lse, ids, alt = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=top)
    others = [0, 1, 3, 4, 5]
    for t in (logp, ent, lse):
        assert torch.isnan(t[2]) and torch.isfinite(t[others]).all()
    if top:
        assert bool((ids[2] == -1).all()) and torch.isnan(alt[2]).all() and bool((ids[others] >= 0).all())


def test_peaked_and_far_apart_logits():
    """Entropies near 0 and near log v; logits thousands apart."""
    v, d = 500, 32
    w = torch.zeros(v, d, device=dev())
    w[:, 0] = torch.linspace(-300, 300, v, device=dev())
    h = torch.zeros(4, d, device=dev())
    h[0, 0], h[1, 0], h[3, 0] = 10.0, -10.0, 1e6
    ws = mm.alloc_linear_logprob_workspace(4, v, d, torch.float32, top=3)
    tokens = torch.tensor([499, 0, 7, 499], device=dev())
    logp, ent, lse, ids, alt = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=3)
    # neighbours are 12 apart: the best has all but e^-12 of the probability
    want = ref.logprobs(num(h[:3]), num(w), tokens[:3].cpu().numpy(), 3)
    assert np.allclose(num(ent[:3]), want[1], rtol=1e-3, atol=1e-6) and np.allclose(num(logp[:3]), want[0], atol=1e-3)
    assert np.array_equal(ids[:3].cpu().numpy(), want[3]) and ids[3].tolist() == [499, 498, 497]
    assert logp[3].item() == 0 and ent[3].item() == 0
    a = torch.ones(4, device=dev())
    dh, dw = mm.muon_linear_logprob_backward(h, w, tokens, lse, ent, ws, a, a)
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()
    e = torch.empty(0, d, device=dev())
    none = torch.empty(0, dtype=torch.int64, device=dev())
    logp, ent, lse, ids, alt = mm.muon_linear_logprob_forward(e, w, none, ws, top=3)
    assert logp.shape == (0,) and ids.shape == (0, 3)
    dh, dw = mm.muon_linear_logprob_backward(e, w, none, lse, ent, ws, lse, ent)
    assert dh.shape == (0, d) and not dw.any()


def test_tokens():
    """All ignored; out of range; an ignore_index inside the vocabulary; the last column."""
    n, v, d = 20, 300, 64
    h, h64, w, w64, tokens, tok = case(n, v, d, "bf16", 11)
    ws = mm.alloc_linear_logprob_workspace(n, v, d, top=2)
    none = torch.full_like(tokens, -100)
    logp, ent, lse, ids, alt = mm.muon_linear_logprob_forward(h, w, none, ws, top=2)
    assert not logp.any() and not ent.any() and torch.isfinite(lse).all()
    assert bool((ids == -1).all()) and bool((alt == -float("inf")).all())
    nan = torch.full((n,), float("nan"), device=dev())
    dh, dw = mm.muon_linear_logprob_backward(h, w, none, nan, nan, ws, nan, nan)
    assert not dh.any() and not dw.any()
    odd = tokens.clone()
    odd[3], odd[4], odd[5] = v, -1, v - 1
    logp, ent, lse, ids, alt = mm.muon_linear_logprob_forward(h, w, odd, ws, top=2)
    for t in (logp, ent):
        assert torch.isnan(t[3]) and torch.isnan(t[4]) and torch.isfinite(t[5])
    assert torch.isfinite(lse).all() and bool((ids[3:6] >= 0).all())
    one = torch.ones(n, device=dev())
    dh, dw = mm.muon_linear_logprob_backward(h, w, odd, lse, ent, ws, one, one)
    assert not dh[3].any() and not dh[4].any() and dh[5].any() and torch.isfinite(dw).all()
    zero = torch.where(tokens == -100, 0, tokens)
    logp, _, _, _, _ = mm.muon_linear_logprob_forward(h, w, zero, ws, ignore_index=0)
    assert not logp[zero == 0].any() and logp[zero != 0].all()


@pytest.mark.parametrize("dt,d,pad", [("bf16", 64, 0), ("bf16", 72, 24), ("bf16", 61, 0), ("f32", 64, 0), ("f32", 61, 2)])
def test_rows_without_a_token_may_hold_anything(dt, d, pad):
    """NaN and infinities in rows whose token is ignored or out of range change no gradient."""
    n, v = 140, 300
    h, h64, w, w64, tokens, tok = case(n, v, d, dt, 12)
    tokens = tokens.clone()
    tokens[::3], tokens[7] = -100, v + 5
    dead = (tokens < 0) | (tokens >= v)
    big = torch.zeros(n, d + pad, dtype=h.dtype, device=dev())
    clean = torch.where(dead[:, None], 0.0, h.float()).to(h.dtype)
    junk = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38], device=dev()).repeat(n * d // 4 + 1)[:n * d]
    big[:, :d] = torch.where(dead[:, None], junk.view(n, d), h.float()).to(h.dtype)
    big = big[:, :d]
    ws = mm.linear_logprob_workspace_for(big, w, tokens, top=4)
    got, want = (mm.muon_linear_logprob_forward(x, w, tokens, ws, top=4) for x in (big, clean))
    assert all(torch.equal(p[~dead], q[~dead]) for p, q in zip(got, want))
    one = torch.ones(n, device=dev())
    a, b = (mm.muon_linear_logprob_backward(x, w, tokens, o[2], o[1], ws, one, one) for x, o in ((big, got), (clean, want)))
    assert all(torch.equal(p, q) and bool(torch.isfinite(p).all()) for p, q in zip(a, b))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_and_alignment(dt):
    for n, v, d, pad, off in ((33, 200, 64, 8, 0), (33, 200, 64, 5, 0), (20, 77, 50, 3, 1), (9, 130, 128, 0, 1)):
        h, h64, w, w64, tokens, tok = case(n, v, d, dt, n)
        hb, wb = (torch.full((off + k * (d + pad) + 8,), float("nan"), dtype=h.dtype, device=dev()) for k in (n, v))
        hv, wv = (t[off:off + k * (d + pad)].view(k, d + pad)[:, :d] for t, k in ((hb, n), (wb, v)))
        hv.copy_(h)
        wv.copy_(w)
        ws = mm.linear_logprob_workspace_for(hv, wv, tokens, top=6)
        packed = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=6)
        a, b = mm.muon_linear_logprob_forward(hv, wv, tokens, ws, top=6), mm.muon_linear_logprob_forward(h, w, tokens, packed, top=6)
        for out in (a, b):
            check(out, h64, w64, tok, 6, dt, (n, v, d, pad, off))
        one = torch.ones(n, device=dev())
        c = mm.muon_linear_logprob_backward(hv, wv, tokens, b[2], b[1], ws, one, one)
        e = mm.muon_linear_logprob_backward(h, w, tokens, b[2], b[1], packed, one, one)
        if n > 16:       # tiles of copies: the same bits (few rows are read where they lie, and summed in another order)
            assert all(torch.equal(p, q) for p, q in zip(a[:4], b[:4])) and all(torch.equal(p, q) for p, q in zip(c, e))
        for p, q in zip(c, e):
            assert torch.linalg.norm((p - q).float()) <= (2 * BF if dt == "bf16" else 1e-5) * torch.linalg.norm(q.float())


def test_repeats_other_streams_graphs_and_pieces():
    n, v, d = 300, 10007, 130
    h, h64, w, w64, tokens, tok = case(n, v, d, "bf16", 21)
    one = torch.ones(n, device=dev())

    def both(ws, stream=None):
        out = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=5, stream=stream)
        return out + mm.muon_linear_logprob_backward(h, w, tokens, out[2], out[1], ws, one, one, stream=stream)

    ws = mm.alloc_linear_logprob_workspace(n, v, d, top=5)
    want = both(ws)
    ws[256:].fill_(255)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(ws, s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    only = mm.muon_linear_logprob_backward(h, w, tokens, want[2], want[1], ws, one, one, need_dw=False)
    assert only[1] is None and torch.equal(only[0], want[5])
    only = mm.muon_linear_logprob_backward(h, w, tokens, want[2], want[1], ws, one, one, need_dh=False)
    assert only[0] is None and torch.equal(only[1], want[6])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both(ws)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want))
    # queued without a wait between them, with short limits for the kernels' own waits
    mm.muon_debug_set(0, 200)
    try:
        for _ in range(150):
            got = both(ws)
        assert mm.muon_check_status(ws) == mm.MUON_OK
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        # the vocabulary in pieces: the same gradients but for the order of dh's sums
        mm.muon_debug_set(4 * mm.MUON_DEBUG_CE_PIECE, 0)
        wp = mm.alloc_linear_logprob_workspace(n, v, d, top=5)
        got = both(wp)
        assert mm.muon_check_status(wp) == mm.MUON_OK
    finally:
        mm.muon_debug_set(0, 0)
    assert torch.equal(got[6], want[6])
    assert np.linalg.norm(num(got[5]) - num(want[5])) < BF * np.linalg.norm(num(want[5]))


def test_expired_wait_shows_in_every_output():
    n, v, d = 40, 600, 64
    h, h64, w, w64, tokens, tok = case(n, v, d, "bf16", 6)
    one = torch.ones(n, device=dev())
    for top in (0, 3):
        ws = mm.alloc_linear_logprob_workspace(n, v, d, top=top)
        want = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=top)
        wantg = mm.muon_linear_logprob_backward(h, w, tokens, want[2], want[1], ws, one, one)
        mm.muon_debug_set(mm.MUON_DEBUG_STALL_PRODUCER, 50)
        try:
            out = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=top)
        finally:
            mm.muon_debug_set(0, 0)
        grads = mm.muon_linear_logprob_backward(h, w, tokens, want[2], want[1], ws, one, one)
        for t in (*out[:3], *grads):
            assert torch.isnan(t).all()
        if top:
            assert bool((out[3] == -1).all()) and torch.isnan(out[4][tokens != -100]).all()
        assert mm.muon_check_status(ws) == mm.MUON_ERR_TIMEOUT
        got = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=top)
        gotg = mm.muon_linear_logprob_backward(h, w, tokens, want[2], want[1], ws, one, one)
        assert all(p is q or torch.equal(p, q) for p, q in zip(got + gotg, want + wantg))


def test_past_32_bit_offsets():
    """Rows 2^25 elements apart in both operands."""
    n, v, d, apart = 40, 90, 96, 1 << 25
    h, h64, w, w64, tokens, tok = case(n, v, d, "bf16", 2)
    big = torch.zeros((n + v) * apart, dtype=torch.bfloat16, device=dev()).view(n + v, apart)
    hv, wv = big[:n, :d], big[n:, :d]
    hv.copy_(h)
    wv.copy_(w)
    one = torch.ones(n, device=dev())
    ws = mm.linear_logprob_workspace_for(hv, wv, tokens, top=4)
    a, b = mm.muon_linear_logprob_forward(hv, wv, tokens, ws, top=4), mm.muon_linear_logprob_forward(h, w, tokens, ws, top=4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a, b = (mm.muon_linear_logprob_backward(x, y, tokens, a[2], a[1], ws, one, one) for x, y in ((hv, wv), (h, w)))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_logprobs_function(dt):
    """Under autograd: a policy's loss against torch's own derivatives in 64 bits."""
    torch.manual_seed(2)
    n, v, d = 24, 301, 40
    h = torch.randn(3, n // 3, d, device=dev()).to(TYPES[dt]).requires_grad_()
    w = (torch.randn(v, d, device=dev()) * 0.3).to(TYPES[dt]).requires_grad_()
    tokens = torch.randint(0, v, (3, n // 3), device=dev())
    tokens[1, 2] = -100
    adv = torch.randn(3, n // 3, device=dev())
    h6, w6 = h.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    lp6 = torch.log_softmax(h6 @ w6.T, -1)
    live = tokens != -100
    logp6 = torch.where(live, lp6.gather(-1, tokens.clamp(min=0)[..., None])[..., 0], 0.0)
    ent6 = torch.where(live, -(lp6.exp() * lp6).sum(-1), 0.0)
    tol = 4 * BF if dt == "bf16" else 1e-4
    for how in ("both", "logprob", "entropy"):
        logp, ent, ids, alt = mm.linear_logprobs(h, w, tokens, top=3)
        assert logp.shape == tokens.shape and ids.shape == (*tokens.shape, 3) and not alt.requires_grad
        assert torch.allclose(logp.double(), logp6, atol=1e-4) and torch.allclose(ent.double(), ent6, atol=1e-4)
        first, second = (-(adv * logp).mean(), -0.1 * ent.mean()), (-(adv * logp6).mean(), -0.1 * ent6.mean())
        a, b = {"both": (sum(first), sum(second)), "logprob": (first[0], second[0]), "entropy": (first[1], second[1])}[how]
        got, want = torch.autograd.grad(a, (h, w)), torch.autograd.grad(b, (h6, w6), retain_graph=True)
        for p, q in zip(got, want):
            assert p.shape == q.shape and torch.linalg.norm(p.double() - q) < tol * torch.linalg.norm(q)
    logp, ent = mm.linear_logprobs(h, w, tokens)
    (g,) = torch.autograd.grad(logp.sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        g.sum().backward()
