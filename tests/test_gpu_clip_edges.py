"""Clipping at the ends of its types' range, and where the optimizer calls it."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev():
    return torch.device("cuda:0")


def test_first_clipped_step_on_another_stream():
    """Memory that the current stream has given back and still reads is not the step's: what a step
    on another stream needs there is made beforehand, or on that stream."""
    torch.manual_seed(2)
    weights, aux = [torch.randn(64, 96, device=dev())], [torch.randn(50, device=dev())]
    twins = [t.clone() for t in weights], [t.clone() for t in aux]
    grads = [torch.randn(64, 96, device=dev()), torch.randn(50, device=dev())]
    again = [g.clone() for g in grads]
    opt = mm.PeriodicMuon(weights, aux_params=aux, max_grad_norm=0.5)
    one = mm.PeriodicMuon(twins[0], aux_params=twins[1], max_grad_norm=0.5)
    size = mm.alloc_clip_workspace().numel()
    out = [torch.zeros(size, dtype=torch.uint8, device=dev()) for _ in range(32)]
    held = [torch.full_like(o, 7) for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(100_000_000)
    for i in range(len(out)):
        out[i].copy_(held[i])
    held.clear()
    opt.step(grads[:1], grads[1:], stream=side)
    torch.cuda.synchronize()
    assert all(bool((o == 7).all()) for o in out)
    one.step(again[:1], again[1:])
    torch.cuda.synchronize()
    assert torch.equal(opt.grad_norm, one.grad_norm)
    assert all(torch.equal(a, b) for a, b in zip(weights + aux + grads, twins[0] + twins[1] + again))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size, max_norm", [(1e38, 1.0), (1e38, 1e-3), (1e37, 1e-9), (1e20, 1e-25), (1.0, 1e-38), (1e-3, 1e-30)])
def test_factors_below_the_smallest_normal_number(dt, size, max_norm):
    """max_norm / norm down to 2^-150 and below keeps its bits: a clipped number is off by the norm's
    36 roundings at most (64 squares in fp32), the factor's, the product's and its type's."""
    rng = np.random.default_rng(1)
    for n in (63, 4099):
        g = torch.from_numpy(rng.uniform(-3, 3, n) * size).to(dev(), TYPES[dt])
        before = g.double().cpu().numpy()
        norm = np.sqrt((before ** 2).sum())
        got = mm.muon_clip_grad_norm([g], max_norm, mm.alloc_clip_workspace())
        assert norm > 3.4028235677973366e38 and np.isinf(got.item()) or abs(got.item() - norm) <= 36 * 2.0 ** -24 * norm
        want = before * (max_norm / norm)
        one = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
        tiny = 2.0 ** -133 if dt == "bf16" else 2.0 ** -149
        off = np.abs(g.double().cpu().numpy() - want)
        assert np.all(off <= (one + 40 * 2.0 ** -24) * np.abs(want) + 1.01 * tiny), float((off / np.abs(want)).max())


@pytest.mark.parametrize("bits", [8, 32])
def test_gradients_that_are_not_contiguous_are_clipped_in_place(bits):
    torch.manual_seed(5)
    w = [torch.randn(64, 96, device=dev())]
    aux = [torch.randn(12, 10, device=dev()), torch.randn(40, device=dev()), torch.randn(6, 8, device=dev()), torch.randn(16, device=dev())]
    opt = mm.PeriodicMuon(w, aux_params=aux, aux_bits=bits, max_grad_norm=0.5)
    wide = torch.randn(40, 3, device=dev())
    one = torch.randn(8, device=dev())
    ga = [torch.randn(10, 12, device=dev()).t(), wide[:, 1], one.expand(6, 8), torch.randn(16, device=dev())]
    g = [torch.randn(64, 96, device=dev())]
    before, others = [t.double().clone() for t in g + ga], wide.clone()
    norm = torch.sqrt(sum(t.square().sum() for t in before)).item()
    opt.step(g, ga)
    assert abs(opt.grad_norm.item() - norm) <= 36 * 2.0 ** -24 * norm
    for t, b in zip(g + ga, before):
        want = b * (0.5 / norm)
        assert torch.all((t.double() - want).abs() <= 40 * 2.0 ** -24 * want.abs())
    assert torch.equal(wide[:, ::2], others[:, ::2])           # its neighbours stay


@pytest.mark.parametrize("bits", [8, 32])
def test_a_clipped_step_captured_first(bits):
    """The first step of an optimizer inside a capture, its gradients changed between replays; the norm on
    the device is the replayed step's."""
    def fresh():
        torch.manual_seed(6)
        return [torch.randn(64, 96, device=dev())], [torch.randn(12, 10, device=dev()), torch.randn(40, device=dev())]

    (w1, a1), (w2, a2) = fresh(), fresh()
    one = mm.PeriodicMuon(w1, aux_params=a1, aux_bits=bits, max_grad_norm=0.5)
    two = mm.PeriodicMuon(w2, aux_params=a2, aux_bits=bits, max_grad_norm=0.5)
    g, ga = [torch.randn(64, 96, device=dev())], [torch.randn(10, 12, device=dev()).t(), torch.randn(40, device=dev())]
    keep = [t.clone() for t in g + ga]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one.step(g, ga)
    for scale in (1.0, 3.0):
        for t, k in zip(g + ga, keep):
            t.copy_(k * scale)
        for p, q in zip(w1 + a1 + one.M + one.aux_m + one.aux_v, w2 + a2 + two.M + two.aux_m + two.aux_v):
            p.copy_(q)
        if bits == 8:
            one.aux8.load_state_dict(two.aux8.state_dict())
        two.step_count = 0
        h, ha = [t.clone() for t in g], [ga[0].t().clone().t(), ga[1].clone()]
        graph.replay()
        two.step(h, ha)
        torch.cuda.synchronize()
        assert torch.equal(one.grad_norm, two.grad_norm)
        assert all(torch.equal(p, q) for p, q in zip(w1 + a1 + g + ga, w2 + a2 + h + ha))
