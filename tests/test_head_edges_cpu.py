"""The head's host side without a GPU: the differentiable forms with their kernels replaced by
the formulas, and refusals that depend on where tensors live."""
import pytest
import torch

from matrix_aware_optimizer_muon_gb300 import functional, head


def _ln_forward(x, weight=None, bias=None, eps=1e-5, stream=None):
    mean = x.float().mean(1)
    rstd = 1 / torch.sqrt((x.float() - mean[:, None]).square().mean(1) + eps)
    y = (x.float() - mean[:, None]) * rstd[:, None]
    y = y if weight is None else y * weight.float()
    return (y if bias is None else y + bias.float()).to(x.dtype), mean, rstd


def _ln_backward(dy, x, weight, mean, rstd, ws=None, bias=True, stream=None, weight_grad=True):
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    g = dy.float() if weight is None else dy.float() * weight.float()
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return (dx.to(x.dtype), None if weight is None or not weight_grad else (dy.float() * xh).sum(0).to(weight.dtype),
            dy.float().sum(0) if bias else None)


def _ce_forward(h, w, labels, ws, ignore_index=-100, stream=None):
    z = h @ w.T
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, labels[:, None])[:, 0]
    return loss, lse, torch.stack([loss.mean(), torch.tensor(float(len(loss)))])


def _ce_backward(h, w, labels, lse, ws, stats=None, upstream=None, need_dh=True, need_dw=True, **_):
    g = torch.exp(h @ w.T - lse[:, None])
    g[torch.arange(len(labels)), labels] -= 1
    g = g * upstream / stats[1]
    return g @ w if need_dh else None, g.T @ h if need_dw else None


@pytest.fixture
def plain(monkeypatch):
    calls = []

    def kept(name, f):
        def g(*a, **k):
            calls.append((name, k))
            return f(*a, **k)
        monkeypatch.setattr(head, name, g)

    kept("muon_layernorm_forward", _ln_forward)
    kept("muon_layernorm_backward", _ln_backward)
    kept("muon_linear_ce_forward", _ce_forward)
    kept("muon_linear_ce_backward", _ce_backward)
    monkeypatch.setattr(head, "alloc_layernorm_workspace", lambda *a, **k: None)
    monkeypatch.setattr(head, "linear_ce_workspace_for", lambda *a, **k: None)
    return calls


def test_first_derivatives_are_the_formulas(plain):
    torch.manual_seed(0)
    x, w, b = torch.randn(6, 24, requires_grad=True), torch.randn(24, requires_grad=True), torch.randn(24, requires_grad=True)
    v, labels = torch.randn(40, 24, requires_grad=True), torch.arange(6)
    got = torch.autograd.grad(functional.linear_cross_entropy(functional.layer_norm(x, w, b), v, labels), (x, w, b, v))
    y = torch.nn.functional.layer_norm(x, (24,), w, b)
    want = torch.autograd.grad(torch.nn.functional.cross_entropy(y @ v.T, labels), (x, w, b, v))
    assert all(torch.allclose(p, q, atol=1e-5) for p, q in zip(got, want))


@pytest.mark.parametrize("train", [(True, False, False), (True, True, False), (True, False, True), (False, True, True)])
def test_layer_norm_sums_columns_only_for_what_is_trained(plain, train):
    torch.manual_seed(0)
    t = [torch.randn(s, requires_grad=r) for s, r in zip(((6, 24), (24,), (24,)), train)]
    functional.layer_norm(*t).square().sum().backward()
    name, asked = plain[-1]
    assert name == "muon_layernorm_backward" and bool(asked["weight_grad"]) == train[1] and bool(asked["bias"]) == train[2]
    got = [x.grad for x in t]
    t = [x.detach().requires_grad_(r) for x, r in zip(t, train)]
    torch.nn.functional.layer_norm(t[0], (24,), t[1], t[2]).square().sum().backward()
    for g, x in zip(got, t):
        assert (g is None) == (x.grad is None) and (g is None or torch.allclose(g, x.grad, atol=1e-4))


def test_second_derivatives_are_refused_not_wrong(plain):
    """A penalty on the gradient needs the backward pass's own derivative, which there is none of."""
    x, w = torch.randn(5, 16, requires_grad=True), torch.randn(16, requires_grad=True)
    v, labels = torch.randn(30, 16, requires_grad=True), torch.arange(5)
    for loss in (functional.layer_norm(x, w).square().sum(), functional.linear_cross_entropy(x, v, labels)):
        g, = torch.autograd.grad(loss, x, create_graph=True)
        with pytest.raises(RuntimeError):
            (g.square().sum() + x.sum()).backward()


class _Gpu(torch.Tensor):
    """A tensor that says it lives on a GPU (the one in .gpu)."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.gpu


def _on_gpu(t, gpu):
    t = t.as_subclass(_Gpu)
    t.gpu = gpu
    return t


def test_tensors_of_another_gpu_are_refused(monkeypatch):
    """Operands on two GPUs, or all on one that is not current, never reach the library."""
    monkeypatch.setattr(head, "_current_device", lambda: 0)
    monkeypatch.setattr(head, "load_library", lambda: pytest.fail("reached the library"))
    f = {"x": torch.zeros(4, 8), "w": torch.zeros(8), "b": torch.zeros(8), "mean": torch.zeros(4), "rstd": torch.zeros(4),
         "dy": torch.zeros(4, 8), "ws": torch.zeros(512, dtype=torch.uint8), "h": torch.zeros(4, 8), "v": torch.zeros(16, 8),
         "labels": torch.zeros(4, dtype=torch.int64), "lse": torch.zeros(4), "row_grad": torch.zeros(4),
         "stats": torch.zeros(2), "upstream": torch.zeros(1)}
    calls = {
        "x w b": lambda x, w, b: head.muon_layernorm_forward(x, w, b),
        "dy x w mean rstd ws": lambda *a: head.muon_layernorm_backward(*a),
        "h v labels": lambda *a: head.linear_ce_workspace_for(*a),
        "h v labels ws": lambda *a: head.muon_linear_ce_forward(*a),
        "h v labels lse ws row_grad stats upstream": lambda *a: head.muon_linear_ce_backward(*a),
    }
    for names, call in calls.items():
        names = names.split()
        for moved in [*[{n} for n in names], set(names)]:
            with pytest.raises(ValueError, match="current CUDA device"):
                call(*[_on_gpu(f[n].clone(), 1 if n in moved else 0) for n in names])
