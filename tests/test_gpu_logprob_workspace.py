"""Log probabilities in workspaces that are no larger than they say, with a guard behind each."""
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm
from matrix_aware_optimizer_muon_gb300 import head

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("top", [0, 4])
def test_exact_workspaces(dt, pad, top):
    v, d = 900, 96
    torch.manual_seed(1)
    w = (torch.randn(v, d + pad, device=dev()) / 4).to(dt)[:, :d]
    roomy = head.linear_logprob_workspace_for(torch.zeros(64, d, device=dev(), dtype=dt), w, None, top)
    for n in (1, 2, 3, 4, 5, 8, 9, 16, 17, 64):
        h = torch.randn(n, d, device=dev()).to(dt)
        tok = torch.randint(0, v, (n,), device=dev())
        one = torch.ones(n, device=dev())
        for backward in (False, True):
            size = head.linear_logprob_workspace_for(h, w, tok, top, backward).numel()
            assert size <= roomy.numel()                 # (one for more rows serves these, too)
            buffer = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=dev())
            buffer[:256] = 0
            ws = buffer[:size]
            a, b = (mm.muon_linear_logprob_forward(h, w, tok, s, top=top) for s in (ws, roomy))
            assert all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))
            if backward:
                p, q = (mm.muon_linear_logprob_backward(h, w, tok, a[2], a[1], s, one, one) for s in (ws, roomy))
                assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
            assert bool((buffer[size:] == 0xA5).all())
            if size > 256:
                with pytest.raises(mm.MuonError):
                    mm.muon_linear_logprob_forward(h, w, tok, torch.zeros(256, dtype=torch.uint8, device=dev()), top=top)
