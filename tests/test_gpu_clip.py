"""The global gradient norm and clipping on the GPU against the fp64 oracle, and the step it
belongs to: norm, log probabilities, their gradients, clipping, update.

u = 2^-24.  Up to 64 squares are added in fp32 (64 u of their sum, half of that of its root),
everything above in 64 bits; the factor and the product round once each, the result once more
to bf16 (2^-8)."""
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


def check(tensors, wants, max_norm, ws, what):
    norm = mm.muon_clip_grad_norm(tensors, max_norm, ws)
    rnorm, clipped = ref.clip_grad_norm(wants, np.inf if max_norm is None else max_norm)
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(norm.item() - rnorm) <= 36 * U * rnorm, what
    for t, before, want in zip(tensors, wants, clipped):
        if max_norm is None or rnorm < max_norm * (1 - 40 * U):
            assert np.array_equal(num(t), before), what
        else:
            one = BF if t.dtype == torch.bfloat16 else 0.0
            tiny = 2.0 ** -133 if one else 2.0 ** -149
            assert np.all(np.abs(num(t) - want) <= (one + 40 * U) * np.abs(want) * 1.01 + tiny), what


SIZES = [[1], [3, 1, 7], [8, 16, 2048], [16384], [16385, 16383], [8191, 8192, 8193], [100003], [5, 0, 40000, 0, 1],
         [0], list(range(1, 60)), [300001, 7, 1536, 1537]]


@pytest.mark.parametrize("dt", ["bf16", "f32", "mixed"])
def test_clip(dt):
    ws = mm.alloc_clip_workspace()
    for sizes in SIZES:
        for factor in (None, 0.3, 3.0, 0.0):
            rng = np.random.default_rng(5)
            pairs = [put(rng.standard_normal(n) * (1 + i % 4), ("bf16", "f32")[i % 2] if dt == "mixed" else dt)
                     for i, n in enumerate(sizes)]
            tensors, wants = [p[0] for p in pairs], [p[1] for p in pairs]
            norm = np.sqrt(sum((w ** 2).sum() for w in wants))
            check(tensors, wants, None if factor is None else factor * norm, ws, (dt, sizes, factor))


@pytest.mark.parametrize("off", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_clip_views_of_one_buffer(dt, off):
    """Gradients that lie next to each other at any offset; what is around them stays."""
    sizes, at = [9, 16384, 1, 33333, 6], off
    buf, want = put(np.random.default_rng(off).standard_normal(sum(sizes) + off + 11), dt)
    tensors, wants, inside = [], [], np.zeros(len(want), bool)
    for n in sizes:
        tensors.append(buf[at:at + n])
        wants.append(want[at:at + n].copy())
        inside[at:at + n] = True
        at += n + 1
    check(tensors, wants, 1.0, mm.alloc_clip_workspace(), (dt, off))
    assert np.array_equal(num(buf)[~inside], want[~inside])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e25, 1e19, 1e-19, 1e-25, 1e-37])
def test_clip_of_numbers_whose_squares_leave_fp32(dt, size):
    rng = np.random.default_rng(6)
    pairs = [put(rng.standard_normal(n) * size, dt) for n in (700, 40001)] + [put(np.zeros(5000), dt)]
    tensors, wants = [p[0] for p in pairs], [p[1] for p in pairs]
    check(tensors, wants, 50.0 * size, mm.alloc_clip_workspace(), (dt, size))
    # large and small ones together
    pairs = [put(rng.standard_normal(3000) * s, dt) for s in (size, 1.0)]
    check([p[0] for p in pairs], [p[1] for p in pairs], None, mm.alloc_clip_workspace(), (dt, size, "both"))


def test_clip_many_tensors():
    """More tensors than a launch's table holds, the same bits twice."""
    rng = np.random.default_rng(7)
    sizes = [int(n) for n in rng.integers(1, 400, 2203)]
    sizes[5], sizes[1500] = 70001, 0
    pairs = [put(rng.standard_normal(n), ("bf16", "f32")[i % 2]) for i, n in enumerate(sizes)]
    tensors, wants = [p[0] for p in pairs], [p[1] for p in pairs]
    ws = mm.alloc_clip_workspace()
    ws.fill_(255)
    a, b = mm.muon_clip_grad_norm(tensors, None, ws), mm.muon_clip_grad_norm(tensors, None, ws)
    assert torch.equal(a, b) and mm.muon_launch_count() == 4
    check(tensors, wants, 1.5, ws, "many")


def test_clip_nonfinite_and_limits():
    ws = mm.alloc_clip_workspace()
    inf = float("inf")
    for dt in (torch.float32, torch.bfloat16):
        g = [torch.tensor([1.0, inf, 2.0], device=dev(), dtype=dt), torch.ones(9, device=dev(), dtype=dt)]
        norm = mm.muon_clip_grad_norm(g, None, ws)
        assert norm.item() == inf and g[0][0] == 1
        norm = mm.muon_clip_grad_norm(g, 1.0, ws)
        assert norm.item() == inf and g[0][0] == 0 and torch.isnan(g[0][1]) and not g[1].any()
        g = [torch.tensor([1.0, float("nan")], device=dev(), dtype=dt), torch.ones(9, device=dev(), dtype=dt)]
        assert torch.isnan(mm.muon_clip_grad_norm(g, None, ws)) and g[1].all() and not torch.isnan(g[1]).any()
        assert torch.isnan(mm.muon_clip_grad_norm(g, 1.0, ws)) and torch.isnan(g[1]).all()
    # a norm beyond fp32 that is finite in 64 bits still clips
    g = [torch.full((4,), 3e38, device=dev())]
    assert mm.muon_clip_grad_norm(g, 1.0, ws).item() == inf
    assert torch.allclose(g[0], torch.full((4,), 0.5, device=dev()))
    zero = [torch.zeros(5, device=dev())]
    assert mm.muon_clip_grad_norm(zero, 0.0, ws).item() == 0 and not zero[0].any()
    assert mm.muon_clip_grad_norm([], 1.0, ws).item() == 0


def test_clip_refusals():
    ws = mm.alloc_clip_workspace()
    a = torch.ones(10, device=dev())
    for bad in ([a, a], [a, a[3:]], [a[2:5], a]):
        with pytest.raises(mm.MuonError):
            mm.muon_clip_grad_norm(bad, 1.0, ws)
        assert mm.muon_clip_grad_norm(bad, None, ws).item() > 0      # the norm alone may count elements twice
    assert torch.equal(a, torch.ones_like(a))
    for bad, kind in (([torch.ones(4)], ValueError), ([torch.ones(4, 4, device=dev()).t()[1:]], ValueError),
                      ([torch.ones(4, device=dev(), dtype=torch.float16)], TypeError)):
        with pytest.raises(kind):
            mm.muon_clip_grad_norm(bad, 1.0, ws)
    for most in (-1.0, float("nan")):
        with pytest.raises(mm.MuonError):
            mm.muon_clip_grad_norm([a], most, ws)
    with pytest.raises(mm.MuonError):
        mm.muon_clip_grad_norm([a], 1.0, ws[:64])


def test_clip_on_another_stream_and_in_a_graph():
    ws = mm.alloc_clip_workspace()
    g = [torch.randn(50000, device=dev()), torch.randn(777, device=dev()).bfloat16()]
    copies = [t.clone() for t in g]
    want = mm.muon_clip_grad_norm(g, 1.0, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = [t.clone() for t in copies]
    torch.cuda.synchronize()
    norm = mm.muon_clip_grad_norm(b, 1.0, ws, stream=s)
    s.synchronize()
    assert torch.equal(norm, want) and all(torch.equal(p, q) for p, q in zip(b, g))
    b = [t.clone() for t in copies]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = mm.muon_clip_grad_norm(b, 1.0, ws)
    for t, c in zip(b, copies):
        t.copy_(c)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, want) and all(torch.equal(p, q) for p, q in zip(b, g))
    graph.replay()
    torch.cuda.synchronize()
    assert abs(norm.item() - 1.0) < 1e-2


@pytest.mark.parametrize("bits", [8, 32])
def test_periodic_muon_clips_all_its_gradients(bits):
    """A clipped step is the step of the clipped gradients."""
    torch.manual_seed(3)
    def fresh():
        torch.manual_seed(3)
        weights = [torch.randn(64, 96, device=dev()), torch.randn(128, 64, device=dev())]
        aux = [torch.randn(50, device=dev()), torch.randn(12, 10, device=dev())]
        return weights, aux

    (w1, a1), (w2, a2) = fresh(), fresh()
    one = mm.PeriodicMuon(w1, aux_params=a1, aux_bits=bits, max_grad_norm=2.0)
    two = mm.PeriodicMuon(w2, aux_params=a2, aux_bits=bits)
    assert one.grad_norm is None
    ws = mm.alloc_clip_workspace()
    for step in range(4):
        g, ga = [torch.randn_like(w) * (10.0 ** -step) for w in w1], [torch.randn(50, device=dev()), torch.randn(10, 12, device=dev()).t()]
        h, ha = [t.clone() for t in g], [t.contiguous().clone() for t in ga]
        norm = mm.muon_clip_grad_norm(h + ha, 2.0, ws)
        one.step(g, ga)
        two.step(h, ha)
        assert torch.equal(one.grad_norm, norm)
        assert all(torch.equal(p, q) for p, q in zip(w1 + a1, w2 + a2))
        assert all(torch.equal(p, q) for p, q in zip(g, h))
    # a refused step (two gradients share memory) changes nothing
    before, keep = [t.clone() for t in w1 + a1], g[0].clone()
    with pytest.raises(mm.MuonError):
        one.step(g, [g[0].view(-1)[:50], ga[1]])
    assert all(torch.equal(p, q) for p, q in zip(w1 + a1, before)) and torch.equal(g[0], keep) and one.step_count == 4


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_policy_step(dt):
    """The operators in a row, as a policy-gradient step runs them, against 64 bits: residual and
    norm, log probabilities and entropies, their gradients, clipping, the update."""
    torch.manual_seed(4)
    n, d, v = 96, 64, 517
    t = TYPES[dt]
    x = torch.randn(n, d, device=dev()).to(t)
    r = torch.randn(n, d, device=dev()).to(t)
    proj = (torch.randn(d, d, device=dev()) / 8).to(t).requires_grad_()
    gain = (1 + 0.1 * torch.randn(d, device=dev())).requires_grad_()
    vocab = (torch.randn(v, d, device=dev()) / 8).to(t).requires_grad_()
    tokens = torch.randint(0, v, (n,), device=dev())
    tokens[:7] = -100
    adv = torch.randn(n, device=dev())
    live = (tokens != -100)
    leaves = [proj, gain, vocab]

    def loss_of(logp, ent):
        return -((adv * logp).sum() + 0.01 * ent.sum()) / live.sum()

    y, total = mm.rms_norm(x @ proj.T, gain, r)
    logp, ent = mm.linear_logprobs(y.to(t), vocab, tokens)
    loss = loss_of(logp, ent) + 1e-3 * total.float().square().mean()
    grads = [g.contiguous() for g in torch.autograd.grad(loss, leaves)]

    p6, g6, v6 = (u.detach().double().requires_grad_() for u in leaves)
    t6 = x.double() @ p6.T + r.double()
    y6 = t6 * torch.rsqrt(t6.square().mean(1, keepdim=True) + 1e-6) * g6
    lp6 = torch.log_softmax(y6 @ v6.T, 1)
    logp6 = torch.where(live, lp6.gather(1, tokens.clamp(min=0)[:, None])[:, 0], 0.0)
    ent6 = torch.where(live, -(lp6.exp() * lp6).sum(1), 0.0)
    loss6 = loss_of(logp6, ent6) + 1e-3 * t6.square().mean()
    grads6 = torch.autograd.grad(loss6, (p6, g6, v6))
    # bf16 rounds x proj, total, y, g and the gradients, each by 2^-8 of its numbers at most
    tol = 6 * BF if dt == "bf16" else 1e-4
    assert abs(loss.item() - loss6.item()) < tol * (1 + abs(loss6.item()))
    for a, b in zip(grads, grads6):
        assert torch.linalg.norm(a.double() - b) < tol * torch.linalg.norm(b)
    norm6 = torch.sqrt(sum(b.square().sum() for b in grads6)).item()

    opt = mm.PeriodicMuon([proj.detach()], K=3, aux_params=[vocab.detach(), gain.detach()], aux_bits=8, max_grad_norm=norm6 / 4)
    before = [u.detach().clone() for u in leaves]
    opt.step(grads[:1], [grads[2], grads[1]])
    assert opt.check() == mm.MUON_OK and abs(opt.grad_norm.item() - norm6) < tol * norm6
    scaled = torch.sqrt(sum(g.double().square().sum() for g in grads)).item()
    assert abs(scaled - norm6 / 4) < 2 * BF * norm6
    assert all(not torch.equal(a, b.detach()) for a, b in zip(before, leaves))
