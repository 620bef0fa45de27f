"""RMS norm, log probabilities and clipping without a GPU: the fp64 oracle against independent
facts, the C entry points' refusals and workspace sizes, the differentiable forms with their
kernels replaced by the formulas."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from matrix_aware_optimizer_muon_gb300 import clip, functional, head
from oracle import head_ref as ref

FAKE = 1 << 20   # an aligned address that nothing reads


@pytest.fixture(scope="session")
def lib():
    from matrix_aware_optimizer_muon_gb300 import _lib
    from matrix_aware_optimizer_muon_gb300 import build as b
    if not os.path.exists(_lib.LIB_PATH):
        b.build()
    return _lib.load_library()


def differences(f, arg, grad, step=1e-6, tol=1e-6):
    for i in np.ndindex(arg.shape):
        old = arg[i]
        arg[i] = old + step
        hi = f()
        arg[i] = old - step
        lo = f()
        arg[i] = old
        assert abs((hi - lo) / (2 * step) - grad[i]) < tol


def test_rmsnorm_gradient_matches_differences():
    rng = np.random.default_rng(0)
    t, dy, dt, w = rng.standard_normal((3, 7)), rng.standard_normal((3, 7)), rng.standard_normal((3, 7)), rng.standard_normal(7)

    def f():
        return (ref.rmsnorm_forward(t, w)[0] * dy).sum() + (t * dt).sum()

    dx, dw = ref.rmsnorm_backward(dy, t, w, ref.rmsnorm_forward(t, w)[1], dt)
    differences(f, t, dx)
    differences(f, w, dw)


def test_logprob_gradient_matches_differences():
    rng = np.random.default_rng(1)
    h, w = rng.standard_normal((4, 5)), rng.standard_normal((6, 5))
    tok, a, b = np.array([2, -100, 5, 0]), rng.standard_normal(4), rng.standard_normal(4)

    def f():
        logp, ent, _, _, _ = ref.logprobs(h, w, tok)
        return (a * logp + b * ent).sum()

    _, ent, lse, _, _ = ref.logprobs(h, w, tok)
    g = ref.logprob_logit_grad(h, w, tok, lse, ent, a, b)
    differences(f, h, g @ w)
    differences(f, w, g.T @ h)
    assert not g[1].any()


def test_logprobs_are_torch_log_softmax():
    rng = np.random.default_rng(2)
    h, w, tok = rng.standard_normal((5, 8)), rng.standard_normal((40, 8)), rng.integers(0, 40, 5)
    logp, ent, lse, ids, alt = ref.logprobs(h, w, tok, 6)
    want = torch.log_softmax(torch.from_numpy(h @ w.T), 1)
    assert np.allclose(logp, want.numpy()[np.arange(5), tok]) and np.allclose(ent, torch.distributions.Categorical(logits=want).entropy())
    best, at = want.topk(6, 1)
    assert np.array_equal(ids, at.numpy()) and np.allclose(alt, best.numpy())
    # equal logits: the lower index first; masked entries are no alternatives
    w[7] = w[3]
    h[0] = w[3] * 9
    assert ref.logprobs(h, w, tok, 2)[3][0].tolist() == [3, 7]
    z = np.full((1, 4), -np.inf)
    z[0, 2] = 1.0
    _, ent, _, ids, alt = ref.logprobs(np.ones((1, 1)), z.T, None, 3)
    assert ids[0].tolist() == [2, -1, -1] and alt[0, 0] == 0 and ent[0] == 0


def test_e4m3_is_torchs():
    x = np.concatenate([np.linspace(-460, 460, 20001), 2.0 ** np.linspace(-12, 9, 999), [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(x), want)
    assert np.all(np.abs(ref.e4m3(x) - np.clip(x, -448, 448)) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10))


def test_clip_is_torchs():
    rng = np.random.default_rng(3)
    grads = [rng.standard_normal(n) for n in (3, 50, 1)]
    for most in (0.5, 100.0):
        ps = [torch.zeros(len(g), dtype=torch.float64).requires_grad_() for g in grads]
        for p, g in zip(ps, grads):
            p.grad = torch.from_numpy(g.copy())
        want = torch.nn.utils.clip_grad_norm_(ps, most)
        norm, out = ref.clip_grad_norm(grads, most)
        assert abs(norm - want.item()) < 1e-12 and all(np.allclose(o, p.grad, rtol=1e-5) for o, p in zip(out, ps))


def test_rmsnorm_refusals(lib):
    def fwd(x=FAKE, r=None, y=FAKE, t=None, codes=None, scales=None, rstd=FAKE, w=None, rows=2, dim=8, ld=8, xdt=1, wdt=0,
            eps=1e-6, ldt=8, ldc=8, ldr=8):
        return lib.muon_rmsnorm_forward(x, ld, r, ldr, w, rows, dim, xdt, wdt, eps, t, ldt, y, 8, codes, ldc, scales, rstd, None)

    assert fwd(rows=0) == 0
    for bad in (dict(x=None), dict(y=None), dict(rows=-1), dict(dim=0), dict(ld=7), dict(eps=-1.0), dict(eps=float("nan")),
                dict(x=FAKE + 1), dict(y=FAKE + 1), dict(rstd=FAKE + 2), dict(w=FAKE + 2), dict(codes=FAKE), dict(scales=FAKE),
                dict(codes=FAKE, scales=FAKE + 2), dict(codes=FAKE, scales=FAKE, ldc=7), dict(t=FAKE), dict(r=FAKE, ldr=7),
                dict(r=FAKE, t=FAKE + 64, ldt=7), dict(r=FAKE, t=FAKE, y=FAKE), dict(r=FAKE + 1), dict(dim=(1 << 30) + 1)):
        assert fwd(**bad) == -1, bad
    assert fwd(xdt=2) == -2 and fwd(wdt=7) == -2
    big = ctypes.c_size_t(-1).value
    assert lib.muon_rmsnorm_workspace_size(3, 0) == big and lib.muon_rmsnorm_workspace_size(-1, 8) == big
    assert 0 < lib.muon_rmsnorm_workspace_size(3, 8) < big

    def bwd(dy=FAKE, t=FAKE, rstd=FAKE, dx=FAKE, rows=2, dim=8, dw=None, ws=None, nws=0, ld=8, xdt=1, dt=None, ldd=8):
        return lib.muon_rmsnorm_backward(dy, ld, t, 8, None, rstd, dt, ldd, rows, dim, xdt, 0, dx, 8, dw, ws, nws, None)

    assert bwd(rows=0) == 0
    for bad in (dict(dy=None), dict(t=None), dict(rstd=None), dict(dx=None), dict(ld=7), dict(dim=0), dict(dt=FAKE, ldd=7),
                dict(dt=FAKE + 1), dict(dy=FAKE + 1), dict(rstd=FAKE + 2), dict(dw=FAKE + 2)):
        assert bwd(**bad) == -1, bad
    assert bwd(xdt=3) == -2
    assert bwd(dw=FAKE) == -3 and bwd(dw=FAKE, ws=FAKE + 64, nws=1 << 30) == -3 and bwd(dw=FAKE, ws=FAKE, nws=8) == -3


def _args(**kw):
    d = dict(H=FAKE, W=FAKE, labels=FAKE, rows=4, vocab=16, dim=8, ldh=8, ldw=8, dtype=1, ignore_index=-100)
    d.update(kw)
    return head.MuonLinearCe(*[d[f[0]] for f in head.MuonLinearCe._fields_])


def test_logprob_refusals(lib):
    big = ctypes.c_size_t(-1).value
    size = lambda a, top, b: lib.muon_linear_logprob_workspace_size(ctypes.byref(a), top, b)  # noqa: E731
    assert 0 < size(_args(), 0, 0) <= size(_args(), 8, 0) and size(_args(), 8, 0) <= size(_args(), 8, 1) < big
    assert size(_args(), -1, 0) == big and size(_args(), 33, 0) == big and size(_args(), 32, 0) < big
    for dtype in (0, 1):                       # a workspace serves fewer rows, too
        for vocab in (1, 700, 38911, 38912, 50000):
            for backward in (0, 1):
                sizes = [size(_args(rows=n, vocab=vocab, dtype=dtype), 4, backward) for n in range(40)]
                assert sizes == sorted(sizes), (dtype, vocab, backward)

    def fwd(a, top=3, logp=FAKE, ent=FAKE, lse=FAKE, ids=FAKE, alt=FAKE, ws=FAKE, n=1 << 40):
        return lib.muon_linear_logprob_forward(ctypes.byref(a), top, logp, ent, lse, ids, alt, ws, n, None)

    def bwd(a, lse=FAKE, ent=FAKE, ga=FAKE, gb=FAKE, dH=FAKE, dW=FAKE, ws=FAKE, n=1 << 40):
        return lib.muon_linear_logprob_backward(ctypes.byref(a), lse, ent, ga, gb, dH, dW, ws, n, None)

    for bad in (dict(rows=-1), dict(vocab=0), dict(dim=0), dict(ldh=7), dict(ldw=7), dict(rows=1 << 31)):
        assert size(_args(**bad), 1, 1) == big and fwd(_args(**bad)) == -1 and bwd(_args(**bad)) == -1, bad
    for bad in (dict(H=None), dict(W=None), dict(H=FAKE + 1), dict(W=FAKE + 1), dict(labels=FAKE + 4)):
        assert fwd(_args(**bad)) == -1 and bwd(_args(**bad)) == -1, bad
    assert bwd(_args(labels=None)) == -1                              # a gradient needs tokens
    assert fwd(_args(dtype=9)) == -2 and bwd(_args(dtype=9)) == -2
    for bad in (dict(top=-1), dict(top=33), dict(logp=None), dict(ent=None), dict(lse=None), dict(ids=None), dict(alt=None),
                dict(logp=FAKE + 2), dict(ids=FAKE + 4), dict(alt=FAKE + 1)):
        assert fwd(_args(), **bad) == -1, bad
    for bad in (dict(lse=None), dict(ent=None), dict(lse=FAKE + 2), dict(ga=FAKE + 2), dict(gb=FAKE + 2), dict(dH=FAKE + 1)):
        assert bwd(_args(), **bad) == -1, bad
    for ws, n in ((None, 1 << 40), (FAKE + 16, 1 << 40), (FAKE, 255)):
        assert fwd(_args(), ws=ws, n=n) == -3 and bwd(_args(), ws=ws, n=n) == -3
    assert fwd(_args(), n=size(_args(), 3, 0) - 1) == -3 and bwd(_args(), n=size(_args(), 0, 1) - 1) == -3


def _grads(*entries):
    a = np.zeros(len(entries), dtype=clip._GRAD)
    for i, e in enumerate(entries):
        a["G"][i], a["numel"][i], a["dtype"][i] = e
    return a


def test_clip_refusals(lib):
    def call(arr, n=None, most=1.0, norm=FAKE, ws=FAKE, nws=1 << 20):
        return lib.muon_clip_grad_norm(None if arr is None else arr.ctypes.data, len(arr) if n is None else n, most, norm, ws, nws, None)

    one = _grads((FAKE, 10, 0))
    assert call(None, n=1) == -1 and call(one, n=-1) == -1
    for bad in (dict(most=-1.0), dict(most=float("nan")), dict(norm=None), dict(norm=FAKE + 2)):
        assert call(one, **bad) == -1, bad
    for e in ((0, 10, 0), (FAKE, -1, 0), (FAKE + 2, 10, 0), (FAKE + 1, 10, 1)):
        assert call(_grads(e)) == -1, e
    assert call(_grads((FAKE, 10, 2))) == -2 and call(_grads((FAKE, 1 << 42, 0))) == -2
    for bad in (dict(ws=None), dict(ws=FAKE + 4), dict(nws=lib.muon_clip_workspace_size() - 1)):
        assert call(one, **bad) == -3, bad
    # tensors that share memory are not scaled twice
    for pair in (((FAKE, 10, 0), (FAKE, 10, 0)), ((FAKE + 36, 5, 0), (FAKE, 10, 0)), ((FAKE, 8, 1), (FAKE + 14, 1, 1))):
        assert call(_grads(*pair)) == -1, pair
        assert call(_grads(*pair), most=math.inf) == -6          # (no GPU here)
    assert call(_grads((FAKE, 10, 0), (FAKE + 40, 10, 0), (FAKE, 0, 0))) == -6


def test_python_refusals():
    import matrix_aware_optimizer_muon_gb300 as mm
    x, tok = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: mm.muon_rmsnorm_forward(x), lambda: mm.muon_rmsnorm_forward_fp8(x), lambda: mm.rms_norm(x),
                 lambda: mm.muon_rmsnorm_backward(x, x, None, x[:, 0]), lambda: mm.muon_linear_logprob_forward(x, x, tok, x),
                 lambda: mm.muon_linear_logprob_forward(x, x, None, x), lambda: mm.muon_linear_logprob_backward(x, x, tok, x[0], None, x),
                 lambda: mm.linear_logprobs(x, x, tok), lambda: mm.muon_clip_grad_norm([x], 1.0, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mm.MuonError):
        mm.muon_linear_ce_workspace_size(4, 0, 8)


class _Gpu(torch.Tensor):
    gpu = 0
    is_cuda = True

    def get_device(self):
        return self.gpu


def _on_gpu(t, gpu):
    t = t.as_subclass(_Gpu)
    t.gpu = gpu
    return t


def test_tensors_of_another_gpu_and_other_shapes_are_refused(monkeypatch):
    monkeypatch.setattr(head, "_current_device", lambda: 0)
    for m in (head, clip):
        monkeypatch.setattr(m, "load_library", lambda: pytest.fail("reached the library"))
    f = {"x": torch.zeros(4, 8), "r": torch.zeros(4, 8), "w": torch.zeros(8), "rstd": torch.zeros(4), "dy": torch.zeros(4, 8),
         "dt": torch.zeros(4, 8), "ws": torch.zeros(512, dtype=torch.uint8), "h": torch.zeros(4, 8), "v": torch.zeros(16, 8),
         "tok": torch.zeros(4, dtype=torch.int64), "lse": torch.zeros(4), "ent": torch.zeros(4), "ga": torch.zeros(4),
         "gb": torch.zeros(4)}
    calls = {
        "x w r": lambda x, w, r: head.muon_rmsnorm_forward(x, w, r),
        "x w": lambda x, w: head.muon_rmsnorm_forward_fp8(x, w),
        "dy x w rstd ws dt": lambda *a: head.muon_rmsnorm_backward(*a),
        "h v tok": lambda *a: head.linear_logprob_workspace_for(*a),
        "h v tok ws": lambda *a: head.muon_linear_logprob_forward(*a),
        "h v tok lse ent ws ga gb": lambda *a: head.muon_linear_logprob_backward(*a),
    }
    for names, call in calls.items():
        names = names.split()
        for moved in [*[{n} for n in names], set(names)]:
            with pytest.raises(ValueError, match="current CUDA device"):
                call(*[_on_gpu(f[n].clone(), 1 if n in moved else 0) for n in names])
    on = {k: _on_gpu(t, 0) for k, t in f.items()}
    with pytest.raises(ValueError, match="same shape"):
        head.muon_rmsnorm_forward(on["x"], None, _on_gpu(torch.zeros(1, 8), 0))
    with pytest.raises(ValueError, match="same shape"):
        head.muon_rmsnorm_forward(on["x"], None, _on_gpu(torch.zeros(4, 8, dtype=torch.bfloat16), 0))
    with pytest.raises(ValueError, match="same shape"):
        head.muon_rmsnorm_backward(on["dy"], on["x"], None, on["rstd"], dtotal=_on_gpu(torch.zeros(1, 8), 0))
    with pytest.raises(TypeError):
        head.muon_linear_logprob_backward(on["h"], on["v"], on["tok"], on["lse"], on["ent"], on["ws"],
                                          _on_gpu(torch.zeros(4, dtype=torch.float64), 0))
    with pytest.raises(ValueError):
        head.muon_linear_logprob_forward(on["h"], _on_gpu(torch.zeros(16, 9), 0), None, on["ws"])


@pytest.fixture
def plain(monkeypatch):
    """The kernels' formulas in place of the kernels."""
    seen = []

    def rms_forward(x, weight=None, residual=None, eps=1e-6, stream=None, need_total=True):
        t = x if residual is None else x + residual
        rstd = torch.rsqrt(t.square().mean(1) + eps)
        y = t * rstd[:, None]
        return y if weight is None else y * weight, rstd, t

    def rms_backward(dy, total, weight, rstd, ws=None, dtotal=None, stream=None, weight_grad=True):
        seen.append(("rms", weight_grad, dtotal is not None))
        xh = total * rstd[:, None]
        g = dy if weight is None else dy * weight
        dx = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
        return dx if dtotal is None else dx + dtotal, (dy * xh).sum(0) if weight is not None and weight_grad else None

    def forward(h, w, tokens, ws, top=0, ignore_index=-100, stream=None):
        logp = torch.log_softmax(h @ w.T, 1)
        live = tokens != ignore_index
        one = torch.where(live, logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0], 0.0)
        ent = torch.where(live, -(logp.exp() * logp).sum(1), 0.0)
        best = logp.topk(top, 1) if top else (None, None)
        return one, ent, torch.logsumexp(h @ w.T, 1), best[1], best[0]

    def backward(h, w, tokens, lse, entropy, ws, g_logprob=None, g_entropy=None, ignore_index=-100, need_dh=True, need_dw=True, stream=None):
        seen.append(("logprob", g_logprob is not None, g_entropy is not None))
        a, b = (np.zeros(len(lse)) if g is None else g.double().numpy() for g in (g_logprob, g_entropy))
        g = torch.from_numpy(ref.logprob_logit_grad(h.numpy(), w.numpy(), tokens.numpy(), lse.numpy(), entropy.numpy(), a, b, ignore_index))
        return (g @ w if need_dh else None), (g.T @ h if need_dw else None)

    monkeypatch.setattr(head, "muon_rmsnorm_forward", rms_forward)
    monkeypatch.setattr(head, "muon_rmsnorm_backward", rms_backward)
    monkeypatch.setattr(head, "muon_linear_logprob_forward", forward)
    monkeypatch.setattr(head, "muon_linear_logprob_backward", backward)
    monkeypatch.setattr(head, "alloc_rmsnorm_workspace", lambda *a, **k: None)
    monkeypatch.setattr(head, "linear_logprob_workspace_for", lambda *a, **k: None)
    return seen


def _leaves():
    torch.manual_seed(0)
    x, r = (torch.randn(2, 5, 12, dtype=torch.float64).requires_grad_() for _ in range(2))
    w, v = torch.randn(12, dtype=torch.float64).requires_grad_(), torch.randn(30, 12, dtype=torch.float64).requires_grad_()
    tokens = torch.randint(0, 30, (2, 5))
    tokens[0, 1] = -100
    return x, r, w, v, tokens


def test_first_derivatives_are_the_formulas(plain):
    x, r, w, v, tokens = _leaves()
    a, b, c = (torch.randn(2, 5, dtype=torch.float64) for _ in range(3))

    def loss(norm, logprobs):
        y, t = norm(x, w, r)
        logp, ent = logprobs(y, v, tokens)
        return (a * logp + b * ent).sum() + (c[..., None] * t).sum()

    def norm(x, w, r):
        t = x + r
        return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w, t

    def logprobs(y, v, tokens):
        logp = torch.log_softmax(y @ v.T, -1)
        live = tokens != -100
        return (torch.where(live, logp.gather(-1, tokens.clamp(min=0)[..., None])[..., 0], 0.0),
                torch.where(live, -(logp.exp() * logp).sum(-1), 0.0))

    got = torch.autograd.grad(loss(functional.rms_norm, functional.linear_logprobs), (x, r, w, v))
    want = torch.autograd.grad(loss(norm, logprobs), (x, r, w, v))
    # (the gradients of log probability and entropy pass through fp32)
    assert all(torch.allclose(p, q, rtol=1e-5, atol=1e-6) for p, q in zip(got, want))


def test_only_what_is_asked_for(plain):
    x, r, w, v, tokens = _leaves()
    y, t = functional.rms_norm(x, w, r)
    (g,) = torch.autograd.grad(t.sum(), r)
    assert torch.equal(g, torch.ones_like(r)) and not plain
    y, t = functional.rms_norm(x.detach(), w.detach(), r)
    torch.autograd.grad(y.sum(), r)
    assert plain.pop() == ("rms", False, False)
    logp, ent, ids, alt = functional.linear_logprobs(y, v, tokens, top=4)
    assert ids.shape == alt.shape == (2, 5, 4) and not ids.requires_grad and not alt.requires_grad
    torch.autograd.grad(ent.sum(), v)
    assert plain.pop() == ("logprob", False, True)
    # x and residual may be one tensor
    y, t = functional.rms_norm(x, w, x)
    (g,) = torch.autograd.grad(t.sum(), x)
    assert torch.equal(g, torch.full_like(x, 2.0))


def test_second_derivatives_are_refused_not_wrong(plain):
    x, r, w, v, tokens = _leaves()
    y, t = functional.rms_norm(x, w, r)
    logp, ent = functional.linear_logprobs(y, v, tokens)
    for out, leaf in ((y.square().sum(), x), (t.sum() + y.sum(), r), (logp.sum(), v), (ent.sum(), v)):
        (g,) = torch.autograd.grad(out, leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="second derivatives"):
            g.sum().backward()


@pytest.mark.parametrize("shape", [(3, 2, 12), (6, 12), (1, 6, 12), (2, 3, 1, 12)])
def test_residuals_of_other_shapes_are_refused(plain, shape):
    """As many rows of one width are not one shape: the gradient would have x's."""
    x = torch.randn(2, 3, 12)
    with pytest.raises(ValueError, match="shape"):
        functional.rms_norm(x, None, torch.randn(shape))
    functional.rms_norm(x, None, torch.randn(2, 3, 12))


def test_tokens_of_another_shape_are_refused(plain):
    """Tokens of h's leading shape, or either of them flat; as many in another order would be
    other rows' tokens."""
    h, w = torch.randn(2, 3, 12), torch.randn(30, 12)
    tokens = torch.arange(6).view(2, 3)
    for bad in (tokens.t(), tokens.view(3, 2), tokens.view(1, 6), tokens.view(2, 3, 1)):
        with pytest.raises(ValueError, match="tokens"):
            functional.linear_logprobs(h, w, bad)
    want = functional.linear_logprobs(h, w, tokens)
    for a, b in ((h.view(6, 12), tokens), (h, tokens.view(6)), (h.view(6, 12), tokens.view(6))):
        got = functional.linear_logprobs(a, w, b)
        assert got[0].shape == b.shape and all(torch.equal(p.reshape(-1), q.reshape(-1)) for p, q in zip(got, want))


def test_a_norm_behind_a_residual_keeps_their_sum_alone(plain):
    """x and the residual are free after the forward pass: the sum is all the gradient needs."""
    x, r, w, _, _ = _leaves()
    kept = []

    def pack(t):
        kept.append(t)
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        y, t = functional.rms_norm(x, w, r)
    at = {k.untyped_storage().data_ptr() for k in kept}
    assert not at & {x.untyped_storage().data_ptr(), r.untyped_storage().data_ptr()}
    assert sum(k.numel() >= x.numel() for k in kept) == 1
    # and may be written over before the backward pass
    want = torch.autograd.grad((functional.rms_norm(x, w, r)[0] * y.detach()).sum(), (x, r, w))
    out = (y * y.detach()).sum()
    with torch.no_grad():
        x.zero_(), r.zero_()
    got = torch.autograd.grad(out, (x, r, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def _workspace_size(rows, vocab, dim, f32, top, backward, ldw=None):
    a = head.MuonLinearCe(None, None, None, rows, vocab, dim, dim, ldw or dim, 0 if f32 else 1, -100)
    return head._logprob_workspace_size(a, top, backward)


def test_a_few_rows_need_no_copy_of_w(lib):
    """Their kernels read W where it lies, in any type and alignment."""
    v, d = 32768, 1536
    for rows in (1, 8):
        assert _workspace_size(rows, v, d, True, 8, False) < 4 << 20 < v * d
        assert _workspace_size(rows, v, d, True, 8, True) < 48 << 20        # shares of dH, a CTA each
    assert _workspace_size(2, v, d, False, 8, False, ldw=d + 3) < 4 << 20
    assert _workspace_size(40, v, d, True, 8, False) > 6 * v * d            # (by tiles: three parts of W)


def test_a_workspace_for_more_rows_is_no_smaller(lib):
    for f32 in (False, True):
        for v, d in ((900, 96), (50257, 1536), (1000, 4096), (128, 40)):
            for top in (0, 4):
                for backward in (False, True):
                    sizes = [_workspace_size(n, v, d, f32, top, backward) for n in (1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64)]
                    assert sizes == sorted(sizes), (f32, v, d, top, backward, sizes)
