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
