"""Calls around RMS norm, log probabilities and clipping that their own tests do not make:
captured before any other call, on tensors past 2^31 elements, by two streams at once, with a
workspace made for more rows, in a model whose parameters are frozen."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm
from oracle import head_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def dev():
    return torch.device("cuda:0")


FIRST = """
import torch, matrix_aware_optimizer_muon_gb300 as mm
torch.cuda.init()
mm.muon_init()
dev = "cuda:0"
x = torch.randn(40, 520, device=dev).bfloat16()
odd = torch.randn(40, 521, device=dev)
w = torch.randn(700, 520, device=dev).bfloat16()
tok = torch.arange(40, device=dev)
one = torch.ones(40, device=dev)
gain = torch.ones(520, device=dev)
ws, wf = mm.alloc_linear_logprob_workspace(40, 700, 520, top=3), mm.alloc_linear_logprob_workspace(2, 700, 520, top=3)
wr, wc = mm.alloc_rmsnorm_workspace(40, 520), mm.alloc_clip_workspace()
grads = [torch.randn(5000, device=dev), torch.randn(70, device=dev).bfloat16()]
keep = [g.clone() for g in grads]
torch.cuda.synchronize()

def step():
    out = []
    y, rstd, total = mm.muon_rmsnorm_forward(x, gain, x)
    out += [y, *mm.muon_rmsnorm_forward_fp8(x, gain, x)[:2], mm.muon_rmsnorm_forward(odd)[0], *mm.muon_rmsnorm_backward(x, total, gain, rstd, wr)]
    for n, s in ((40, ws), (2, wf)):
        lp, ent, lse, ids, alt = mm.muon_linear_logprob_forward(y[:n], w, tok[:n], s, top=3)
        out += [lp, ent, ids, alt, *mm.muon_linear_logprob_backward(y[:n], w, tok[:n], lse, ent, s, one[:n], one[:n])]
    out.append(mm.muon_clip_grad_norm(grads, 1.0, wc))
    return out

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
for t, k in zip(grads, keep):
    t.copy_(k)
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out + grads]
for t, k in zip(grads, keep):
    t.copy_(k)
want = step() + grads
torch.cuda.synchronize()
assert all(torch.equal(a.float(), b.float()) for a, b in zip(got, want))
print("captured first")
"""


def test_captured_before_any_other_call():
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_clip_past_32_bit_offsets():
    """A tensor of more than 2^31 elements, and its neighbour in the same launch."""
    n = (1 << 31) + 12345
    big = torch.full((n,), 0.5, dtype=torch.bfloat16, device=dev())
    small = torch.full((1000,), 3.0, device=dev())
    ws = mm.alloc_clip_workspace()
    want = np.sqrt(0.25 * n + 9000.0)
    norm = mm.muon_clip_grad_norm([small, big], float(want / 2), ws)
    # (64 squares in fp32, the rest in 64 bits)
    assert abs(norm.item() - want) <= 36 * 2.0 ** -24 * want
    assert bool((big == 0.25).all()) and torch.allclose(small, torch.full_like(small, 1.5), rtol=1e-6)


def test_two_streams_at_once():
    """Each stream with its own workspace: the results are those of one after the other."""
    n, v, d = 200, 5000, 264
    torch.manual_seed(0)
    sets = []
    for i in range(2):
        x = torch.randn(n, d, device=dev()).bfloat16()
        w = (torch.randn(v, d, device=dev()) / 8).bfloat16()
        sets.append((x, w, torch.randint(0, v, (n,), device=dev()), torch.randn(d, device=dev()), torch.ones(n, device=dev()),
                     mm.alloc_linear_logprob_workspace(n, v, d, top=4), mm.alloc_rmsnorm_workspace(n, d), mm.alloc_clip_workspace()))

    def chain(x, w, tok, gain, one, ws, wr, wc):
        y, rstd, total = mm.muon_rmsnorm_forward(x, gain, x)
        lp, ent, lse, ids, alt = mm.muon_linear_logprob_forward(y, w, tok, ws, top=4)
        dy, dw = mm.muon_linear_logprob_backward(y, w, tok, lse, ent, ws, one, one)
        dx, dg = mm.muon_rmsnorm_backward(dy, total, gain, rstd, wr)
        return lp, ent, ids, alt, mm.muon_clip_grad_norm([dx, dw, dg], 1.0, wc), dx, dw, dg

    want = [chain(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        got = []
        for s, a in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(chain(*a))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for a, b in zip(got, want) for p, q in zip(a, b))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_workspace_for_more_rows_serves_a_few(dt):
    v, d = 900, 96
    torch.manual_seed(1)
    w = (torch.randn(v, d, device=dev()) / 4).to(dt)
    ws = mm.alloc_linear_logprob_workspace(64, v, d, dt, top=4)
    for n in (1, 2, 5, 16, 64):
        h = torch.randn(n, d, device=dev()).to(dt)
        tok = torch.randint(0, v, (n,), device=dev())
        one = torch.ones(n, device=dev())
        own = mm.alloc_linear_logprob_workspace(n, v, d, dt, top=4)
        a, b = (mm.muon_linear_logprob_forward(h, w, tok, s, top=4) for s in (ws, own))
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        if ws.numel() >= own.numel():
            a, b = (mm.muon_linear_logprob_backward(h, w, tok, a[2], a[1], s, one, one) for s in (ws, own))
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_frozen_parameters():
    """Gradients only for what is trained, and for nothing else."""
    torch.manual_seed(2)
    x, r = (torch.randn(20, 48, device=dev()) for _ in range(2))
    w, v = torch.randn(48, device=dev()), torch.randn(300, 48, device=dev()) / 4
    tok = torch.randint(0, 300, (20,), device=dev())
    full = None
    for train in ((1, 1, 1, 1), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1)):
        leaves = [t.clone().requires_grad_(bool(f)) for t, f in zip((x, r, w, v), train)]
        y, total = mm.rms_norm(leaves[0], leaves[2], leaves[1])
        logp, ent = mm.linear_logprobs(y, leaves[3], tok)
        (logp.sum() + 0.1 * ent.sum() + total.square().sum()).backward()
        got = [t.grad for t in leaves]
        full = full or got
        assert all((g is None) if not f else torch.allclose(g, q, rtol=1e-5, atol=1e-6) for g, q, f in zip(got, full, train))


def test_residual_broadcast_is_refused():
    x = torch.randn(4, 8, device=dev())
    for bad in (torch.randn(1, 8, device=dev()), torch.randn(4, 8, device=dev()).bfloat16(), torch.randn(4, 9, device=dev())):
        with pytest.raises(ValueError):
            mm.rms_norm(x, None, bad)
    with pytest.raises(ValueError):
        mm.linear_logprobs(x, torch.randn(5, 8, device=dev()), torch.zeros(3, dtype=torch.int64, device=dev()))
    with pytest.raises(mm.MuonError):
        mm.linear_logprobs(x, torch.randn(5, 8, device=dev()), torch.zeros(4, dtype=torch.int64, device=dev()), top=33)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_more_alternatives_than_entries(dt):
    for n in (2, 40):
        h, w = torch.randn(n, 24, device=dev()).to(dt), torch.randn(5, 24, device=dev()).to(dt)
        tok = torch.zeros(n, dtype=torch.int64, device=dev())
        ws = mm.alloc_linear_logprob_workspace(n, 5, 24, dt, top=32)
        _, _, lse, ids, alt = mm.muon_linear_logprob_forward(h, w, tok, ws, top=32)
        want = ref.logprobs(h.double().cpu().numpy(), w.double().cpu().numpy(), tok.cpu().numpy(), 32)
        assert np.array_equal(ids.cpu().numpy(), want[3]) and bool((alt[:, 5:] == -float("inf")).all())
