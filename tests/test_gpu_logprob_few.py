"""The log probabilities of a few rows, which have kernels of their own: the calls around
them (streams, graphs, a workspace that others use, rows far apart), with the tolerances of
the other tests."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm
from oracle import head_ref as ref
from tests.test_gpu_logprob import BF, TYPES, case, check, dev, num

pytestmark = pytest.mark.gpu


def both(h, w, tokens, ws, one, top=4, stream=None):
    out = mm.muon_linear_logprob_forward(h, w, tokens, ws, top=top, stream=stream)
    return out + mm.muon_linear_logprob_backward(h, w, tokens, out[2], out[1], ws, one, one, stream=stream)


def same(a, b):
    return all(p is q or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 4, 8, 9, 16, 17])
def test_around_the_limits_of_rows(dt, n):
    """Each number of rows that has a kernel of its own, and the next one."""
    for v, d in ((300, 64), (129, 200), (4099, 37)):
        h, h64, w, w64, tokens, tok = case(n, v, d, dt, n + v)
        ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=4)
        one = torch.ones(n, device=dev())
        out = both(h, w, tokens, ws, one)
        check(out[:5], h64, w64, tok, 4, dt, (n, v, d))
        g = ref.logprob_logit_grad(h64, w64, tok, num(out[2]), num(out[1]), np.ones(n), np.ones(n))
        tol = 3 * BF if dt == "bf16" else 1e-5      # g's rounding (in tiles) and the result's, or fp32's sums
        for got, want in ((out[5], g @ w64), (out[6], g.T @ h64)):
            assert np.linalg.norm(num(got) - want) <= tol * np.linalg.norm(want) + 1e-30
        assert mm.muon_check_status(ws) == mm.MUON_OK


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 3])
def test_repeats_streams_and_graphs(dt, n):
    v, d = 5003, 130
    h, h64, w, w64, tokens, tok = case(n, v, d, dt, 3)
    tokens = tokens.clamp(min=0)
    one = torch.ones(n, device=dev())
    ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=4)
    want = both(h, w, tokens, ws, one)
    ws[256:].fill_(255)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(h, w, tokens, ws, one, stream=s)
    s.synchronize()
    assert same(got, want)
    for need in ("dh", "dw"):
        a = mm.muon_linear_logprob_backward(h, w, tokens, want[2], want[1], ws, one, one, need_dh=need == "dh", need_dw=need == "dw")
        assert same([a[0]], [want[5]]) if need == "dh" else same([a[1]], [want[6]])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both(h, w, tokens, ws, one)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert same(out, want)
    for _ in range(100):
        got = both(h, w, tokens, ws, one)
    assert same(got, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_without_a_token_may_hold_anything(dt):
    n, v, d = 3, 700, 72
    h, h64, w, w64, tokens, tok = case(n, v, d, dt, 5)
    tokens = torch.tensor([5, -100, v + 3], device=dev())
    bad = h.clone()
    bad[1], bad[2] = float("nan"), float("inf")
    clean = h.clone()
    clean[1:] = 0
    one = torch.ones(n, device=dev())
    ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=4)
    a, b = (both(x, w, tokens, ws, one) for x in (bad, clean))
    assert same([t[:1] for t in a[:5]], [t[:1] for t in b[:5]]) and same(a[5:], b[5:])
    assert torch.isfinite(a[6]).all() and not a[5][1:].any() and a[5][0].any()
    assert a[0][1] == 0 and a[1][1] == 0 and torch.isnan(a[0][2]) and torch.isnan(a[1][2])


def test_a_lost_wait_of_another_call_shows():
    """A workspace whose status nobody has read writes NaN here, too."""
    v, d = 600, 64
    h, h64, w, w64, tokens, tok = case(40, v, d, "bf16", 6)
    ws = mm.alloc_linear_logprob_workspace(40, v, d, top=4)
    one = torch.ones(1, device=dev())
    few = (h[:1].contiguous(), w, torch.tensor([3], device=dev()))
    want = both(*few, ws, one)
    mm.muon_debug_set(mm.MUON_DEBUG_STALL_PRODUCER, 50)
    try:
        mm.muon_linear_logprob_forward(h, w, tokens, ws)
    finally:
        mm.muon_debug_set(0, 0)
    out = both(*few, ws, one)
    assert all(torch.isnan(out[i]).all() for i in (0, 1, 2, 4, 5, 6)) and bool((out[3] == -1).all())
    assert mm.muon_check_status(ws) == mm.MUON_ERR_TIMEOUT
    assert same(both(*few, ws, one), want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_past_32_bit_offsets_and_unaligned(dt):
    """Rows 2^25 elements apart, and rows that start off every word."""
    n, v, d, apart = 2, 90, 96, 1 << 25
    h, h64, w, w64, tokens, tok = case(n, v, d, dt, 2)
    tokens = torch.tensor([7, 80], device=dev())
    one = torch.ones(n, device=dev())
    for stride, off in ((apart, 0), (d + 3, 1)):
        big = torch.zeros((n + v) * stride + off, dtype=h.dtype, device=dev())
        rows = big[off:].view(n + v, stride)
        hv, wv = rows[:n, :d], rows[n:, :d]
        hv.copy_(h)
        wv.copy_(w)
        ws = mm.linear_logprob_workspace_for(hv, wv, tokens, top=4)
        a, b = both(hv, wv, tokens, ws, one), both(h, w, tokens, ws, one)
        assert torch.equal(a[3], b[3])
        check(a[:5], h64, w64, tokens.cpu().numpy(), 4, dt, (stride, off))
        for p, q in zip(a[5:], b[5:]):
            assert torch.linalg.norm((p - q).float()) <= (2 * BF if dt == "bf16" else 1e-5) * torch.linalg.norm(q.float())
        del big, rows, hv, wv


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("v, d, pad, shift", [(38911, 40, 0, 0), (38912, 40, 0, 0), (38913, 24, 0, 0), (1625, 2241, 0, 0),
                                              (33, 519, 5, 0), (700, 512, 3, 1), (31, 8, 0, 3), (40001, 17, 2, 5), (150, 1001, 0, 7), (97, 768, 1, 2)])
def test_blocks_and_alignments(dt, v, d, pad, shift):
    """Vocabularies around the one that is read in longer blocks, and rows of W that begin anywhere."""
    for n in (1, 2):
        h, h64, w, w64, tokens, tok = case(n, v, d, dt, v + d + n)
        flat = torch.full((v * (d + pad) + shift + 8,), float("nan"), dtype=w.dtype, device=dev())
        wv = flat[shift:shift + v * (d + pad)].view(v, d + pad)[:, :d]
        wv.copy_(w)
        ws = mm.linear_logprob_workspace_for(h, wv, tokens, top=32)
        one = torch.ones(n, device=dev())
        out = both(h, wv, tokens, ws, one, top=32)
        check(out[:5], h64, w64, tok, 32, dt, (n, v, d, pad, shift))
        g = ref.logprob_logit_grad(h64, w64, tok, num(out[2]), num(out[1]), np.ones(n), np.ones(n))
        tol = 3 * BF if dt == "bf16" else 1e-5
        for got, want in ((out[5], g @ w64), (out[6], g.T @ h64)):
            assert np.linalg.norm(num(got) - want) <= tol * np.linalg.norm(want) + 1e-30


@pytest.mark.parametrize("v, d, pad", [(300, 8, 0), (38911, 40, 8), (38912, 96, 0), (1625, 1000, 0), (17, 520, 16), (128, 2048, 0),
                                       (31000, 136, 24), (500, 3520, 0), (500, 3560, 8)])
@pytest.mark.parametrize("n", [1, 3, 8, 9, 16, 17, 31, 32, 33])
def test_words_of_few_rows(n, v, d, pad):
    """Rows of W in whole words, as matrix instructions take them: all numbers of rows, a row's ends
    inside a step; H in words and off them."""
    h, h64, w, w64, tokens, tok = case(n, v, d, "bf16", v + d + n)
    wide = torch.full((v, d + pad), float("nan"), dtype=w.dtype, device=dev())
    wide[:, :d] = w
    odd = torch.full((n, d + 3), float("nan"), dtype=h.dtype, device=dev())
    odd[:, :d] = h
    for hv in (h, odd[:, :d]):
        ws = mm.linear_logprob_workspace_for(hv, wide[:, :d], tokens, top=32)
        out = mm.muon_linear_logprob_forward(hv, wide[:, :d], tokens, ws, top=32)
        check(out, h64, w64, tok, 32, "bf16", (n, v, d, pad))
        assert mm.muon_check_status(ws) == mm.MUON_OK


@pytest.mark.parametrize("v", [1000, 40000])
@pytest.mark.parametrize("n", [5, 16])
def test_words_with_numbers_that_are_none(n, v):
    """A NaN in a row of H is that row's alone; a row of W that the logits mask with minus infinity has
    probability 0; the first call of a size may be a captured one; two streams at once give one's bits."""
    d = 136
    h, h64, w, w64, tokens, tok = case(n, v, d, "bf16", n + v)
    h, h64 = h.abs(), np.abs(h64)                 # so that a row of W of minus infinity makes a logit of it
    h[:, -1], h64[:, -1] = 1, 1
    gone = np.array([0, 31, v // 2, v - 1])
    w[torch.from_numpy(gone).to(dev())], w64[gone] = float("-inf"), -1e30
    tok[np.isin(tok, gone)] = 1
    tok[1] = 2
    tokens.copy_(torch.from_numpy(tok))
    h = h.clamp(min=2.0 ** -20)
    h64 = num(h)
    spaces = [mm.alloc_linear_logprob_workspace(n, v, d, top=6) for _ in range(2)]
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        held = mm.muon_linear_logprob_forward(h, w, tokens, spaces[0], top=6)
    graph.replay()
    torch.cuda.synchronize()
    keep = np.ones(v, bool)
    keep[gone] = False
    back = np.flatnonzero(keep)
    small = np.where(tok >= 0, np.searchsorted(back, np.maximum(tok, 0)), tok)
    rlogp, rent, rlse, rids, ralt = ref.logprobs(h64, w64[keep], small, 6)
    ids = held[3].cpu().numpy()
    assert not np.isin(ids, gone).any()
    ids = np.where(ids < 0, ids, np.searchsorted(back, ids))     # an ignored row has none
    check(held[:3] + (torch.from_numpy(ids).to(dev()), held[4]), h64, w64[keep], small, 6, "bf16", (n, v, "masked"))
    s.wait_stream(torch.cuda.current_stream())
    one = mm.muon_linear_logprob_forward(h, w, tokens, spaces[0], top=6)
    two = mm.muon_linear_logprob_forward(h, w, tokens, spaces[1], top=6, stream=s)
    torch.cuda.synchronize()
    assert same(one, held) and same(two, held)
    bad = h.clone()
    bad[0, 3] = float("nan")
    out = mm.muon_linear_logprob_forward(bad, w, tokens, spaces[0], top=6)
    assert same([x[1:] for x in out], [x[1:] for x in held])
    assert tok[0] == -100 or bool(torch.isnan(out[0][0]) and torch.isnan(out[1][0]))
    assert bool(torch.isnan(out[2][0]))
    for ws in spaces:
        assert mm.muon_check_status(ws) == mm.MUON_OK
