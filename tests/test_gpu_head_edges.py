"""Edges of the head's operators on the GPU: extreme values, failures that have to show, long
sums, several pieces of the vocabulary, many rows.

Tolerances are derived as in test_gpu_head.py."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm
from oracle import head_ref as ref
from test_gpu_head import BF, TYPES, U, ce_case, ce_tolerances, compare_codes, dev, num, padded, put, strided, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gdt", ["bf16", "f32"])
@pytest.mark.parametrize("pdt", ["bf16", "f32"])
def test_adamw8_steps_for_large_gradients(pdt, gdt):
    """Second moments up to the end of fp32's range (2e37), next to ordinary and to tiny ones,
    move their parameters like any others."""
    rng = np.random.default_rng(41)
    sizes = [16, 300, 2048, 5001]
    P0 = [put(rng.standard_normal(k) * 0.02, pdt) for k in sizes]
    opt = mm.AdamW8([p for p, _ in P0], lr=1e-3, betas=(0.9, 0.999), weight_decay=0.05, seed=7)
    ref_p = [q for _, q in P0]
    for t in range(1, 4):
        m8, v8 = (num(x) for x in opt.moments())
        G = [put(rng.standard_normal(k) * 10.0 ** rng.choice([-25.0, -3.0, 15.0, 16.0, 17.0, 18.0, 19.0], k), gdt) for k in sizes]
        opt.step([g for g, _ in G])
        for i, k in enumerate(sizes):
            a = opt.starts[i]
            m0, v0 = m8[a:a + k], v8[a:a + k]
            g = G[i][1]
            p, m, v = ref.adamw8_update(ref_p[i], g, m0, v0, t, 1e-3, 0.9, 0.999, 1e-8, 0.05)
            got = num(opt.params[i])
            # a square below fp32's range is 0 in fp32: with eps = 1e-8 nothing of it shows
            step = 1e-3 * ((0.9 * np.abs(m0) + 0.1 * np.abs(g)) / (1 - 0.9 ** t) / (np.sqrt(v / (1 - 0.999 ** t)) + 1e-8))
            tol = 16 * U * (np.abs(ref_p[i]) + step) + (BF * 1.01 * np.abs(p) if pdt == "bf16" else 0) + 1e-12
            within(got, p, tol, ("p", k, t))
            ref_p[i] = got


def test_linear_ce_expired_wait_shows_in_every_output():
    """When a wait runs out (test flag: no loads are issued) loss, lse, statistics and both
    gradients are NaN, also for a caller that has no workspace to ask."""
    for n, v, d in ((24, 3000, 64), (600, 700, 96)):       # dH summed over ranges of K, and not
        h, h64, w, w64, labels, lab = ce_case(n, v, d, "bf16", 6)
        ws = mm.alloc_linear_ce_workspace(n, v, d)
        want = mm.muon_linear_ce_forward(h, w, labels, ws)
        grads = mm.muon_linear_ce_backward(h, w, labels, want[1], ws, stats=want[2])
        hr, wr = h.clone().requires_grad_(), w.clone().requires_grad_()
        good = mm.linear_cross_entropy(hr, wr, labels)
        mm.muon_debug_set(mm.MUON_DEBUG_STALL_PRODUCER, 20)
        try:
            lost = mm.muon_linear_ce_forward(h, w, labels, ws)
            assert all(bool(torch.isnan(t).all()) for t in lost)
            assert mm.muon_check_status(ws) == mm.MUON_ERR_TIMEOUT
            for need in ((True, True), (True, False), (False, True)):
                lost = mm.muon_linear_ce_backward(h, w, labels, want[1], ws, stats=want[2], need_dh=need[0], need_dw=need[1])
                assert all(t is None or bool(torch.isnan(t).all()) for t in lost)
                assert mm.muon_check_status(ws) == mm.MUON_ERR_TIMEOUT
            assert torch.isnan(mm.linear_cross_entropy(hr, wr, labels))
            good.backward()
            assert bool(torch.isnan(hr.grad).all()) and bool(torch.isnan(wr.grad).all())
        finally:
            mm.muon_debug_set(0, 0)
        got = mm.muon_linear_ce_forward(h, w, labels, ws)
        again = mm.muon_linear_ce_backward(h, w, labels, got[1], ws, stats=got[2])
        assert mm.muon_check_status(ws) == mm.MUON_OK
        assert all(torch.equal(p, q) for p, q in zip(want + grads, got + again))


@pytest.mark.parametrize("bits", [8, 32])
def test_periodic_muon_copies_gradients_on_the_stream_that_reads_them(bits):
    """Gradients that are not contiguous, and a stream of the caller's, while the current stream
    is busy and its freed memory is written again."""
    gen = torch.Generator(device=dev())
    gen.manual_seed(3)
    W0 = torch.randn(64, 96, generator=gen, device=dev()).bfloat16()
    A0 = [torch.randn(s, generator=gen, device=dev()) for s in ((1000, 700), (33, 65))]
    G = [torch.randn(64, 96, generator=gen, device=dev()).bfloat16()]
    GA = [torch.randn(*reversed(a.shape), generator=gen, device=dev()).T for a in A0]

    def run(stream):
        W, A = [W0.clone()], [a.clone() for a in A0]
        opt = mm.PeriodicMuon(W, aux_params=A, aux_bits=bits, aux_lr=1e-2)
        torch.cuda.synchronize()
        if stream is None:
            opt.step(G, [g.contiguous() for g in GA])
        else:
            torch.cuda._sleep(100_000_000)
            opt.step(G, GA, stream=stream)
            for g in GA:                          # what the step let go of is given out again
                torch.full_like(g.contiguous(), float("nan"))
        torch.cuda.synchronize()
        return W + A

    assert all(torch.equal(a, b) for a, b in zip(run(None), run(torch.cuda.Stream())))


def test_streams_given_as_handles():
    """0 is the default stream, any other number the stream it is the handle of: outputs and
    copies are made on the very stream the kernels run on."""
    from matrix_aware_optimizer_muon_gb300 import head
    side = torch.cuda.Stream()
    for stream, handle in ((0, 0), (side.cuda_stream, side.cuda_stream), (side, side.cuda_stream), (torch.cuda.default_stream(), 0)):
        with torch.cuda.stream(torch.cuda.Stream()), head._on(stream):
            assert torch.cuda.current_stream().cuda_stream == handle
    x = torch.randn(50, 64, device=dev())
    want = mm.muon_layernorm_forward(x)
    torch.cuda.synchronize()
    for stream in (0, side.cuda_stream):
        got = mm.muon_layernorm_forward(x, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("bits", [8, 32])
def test_periodic_muon_refuses_before_it_changes_anything(bits):
    W = [torch.randn(64, 96, device=dev()).bfloat16()]
    A = [torch.randn(300, device=dev()), torch.randn(40, device=dev())]
    opt = mm.PeriodicMuon(W, aux_params=A, aux_bits=bits)
    g, ga = [torch.randn_like(W[0])], [torch.randn_like(a) for a in A]
    opt.step(g, ga)
    w, a, m = W[0].clone(), [x.clone() for x in A], opt.M[0].clone()

    def refused(grads):
        with pytest.raises((ValueError, TypeError, mm.MuonError)):
            opt.step(g, grads)
        torch.cuda.synchronize()
        assert torch.equal(W[0], w) and torch.equal(opt.M[0], m) and opt.step_count == 1

    refused(ga[:1])
    refused([ga[0], ga[1][:39]])
    refused([ga[0], ga[1].cpu()])
    refused([ga[0], ga[1].bfloat16()])
    refused([ga[0], ga[1].half()])
    keep = opt.aux[1].data
    for bad in (keep.bfloat16(), keep.cpu(), keep[:39], torch.zeros(80, device=dev())[::2]):
        opt.aux[1].data = bad
        refused(ga)
    opt.aux[1].data = keep
    assert all(torch.equal(x, y) for x, y in zip(A, a))
    opt.step(g, ga)
    assert opt.step_count == 2 and not torch.equal(W[0], w)


def test_periodic_muon_refuses_a_state_before_it_copies_any():
    def make(rows, k):
        return mm.PeriodicMuon([torch.ones(rows, 96, device=dev()).bfloat16()], aux_params=[torch.ones(k, device=dev())], aux_bits=8)

    opt = make(64, 300)
    opt.step([torch.ones(64, 96, device=dev()).bfloat16()], [torch.ones(300, device=dev())])
    m, codes = opt.M[0].clone(), opt.aux8.m.clone()
    for other in (make(64, 700), make(65, 300)):
        with pytest.raises(ValueError):
            opt.load_state_dict(other.state_dict())
        assert torch.equal(opt.M[0], m) and torch.equal(opt.aux8.m, codes) and opt.step_count == 1


def test_layer_norm_bias_without_weight_has_its_own_precision():
    rng = np.random.default_rng(3)
    n, d = 777, 96
    x, _ = put(rng.standard_normal((n, d)), "bf16")
    dy, dy64 = put(rng.standard_normal((n, d)), "bf16")
    b, _ = put(rng.standard_normal(d), "f32")
    x.requires_grad_(), b.requires_grad_()
    mm.layer_norm(x, None, b).backward(dy)
    assert b.grad.dtype == torch.float32
    within(num(b.grad), dy64.sum(0), (n + 8) * U * np.abs(dy64).sum(0), "db")


@pytest.mark.parametrize("train", [(True, False, False), (True, True, False), (True, False, True), (False, True, True)])
def test_layer_norm_of_frozen_parameters(train):
    """Column sums are left out where no gradient is wanted; the other gradients keep their bits."""
    rng = np.random.default_rng(5)
    n, d = 500, 200
    vals = [rng.standard_normal(s) for s in ((n, d), d, d)]
    dy, _ = put(rng.standard_normal((n, d)), "f32")

    def grads(flags):
        t = [put(a, "f32")[0].requires_grad_(f) for a, f in zip(vals, flags)]
        mm.layer_norm(*t).backward(dy)
        return [x.grad for x in t]

    for got, want, f in zip(grads(train), grads((True, True, True)), train):
        assert (got is None) == (not f) and (got is None or torch.equal(got, want))
    x, w = put(vals[0], "f32")[0], put(vals[1], "f32")[0]
    _, mean, rstd = mm.muon_layernorm_forward(x, w)
    dx, dw, db = mm.muon_layernorm_backward(dy, x, w, mean, rstd, bias=False, weight_grad=False)
    assert dw is None and db is None and mm.muon_launch_count() == 1


def test_adamw8_parameters_of_two_types():
    """A bf16 matrix beside fp32 vectors: each gets, bit for bit, what it gets among its like."""
    rng = np.random.default_rng(8)
    sizes, kinds = [5000, 300, 129, 700], ["bf16", "f32", "bf16", "f32"]
    vals = [rng.standard_normal(k) * 0.02 for k in sizes]
    grads = [[rng.standard_normal(k) * 1e-3 for k in sizes] for _ in range(3)]

    def run(types, gtypes, resume_at=None):
        P = [put(x, t)[0] for x, t in zip(vals, types)]
        opt = mm.AdamW8(P, lr=1e-2, weight_decay=0.1, seed=3)
        for s, g in enumerate(grads):
            if s == resume_at:
                sd = opt.state_dict()
                opt = mm.AdamW8(P, lr=1e-2, weight_decay=0.1)
                opt.load_state_dict(sd)
            opt.step([put(x, t)[0] for x, t in zip(g, gtypes)])
        return P, opt.moments()

    P, (m, v) = run(kinds, kinds)
    R, (mr, vr) = run(kinds, kinds, resume_at=2)
    assert all(torch.equal(p, r) for p, r in zip(P, R)) and torch.equal(m, mr) and torch.equal(v, vr)
    at = 0
    starts = mm.AdamW8([torch.zeros(k, device=dev()) for k in sizes]).starts
    for kind in ("bf16", "f32"):
        Q, (mq, vq) = run([kind] * 4, [kind] * 4)
        for i in range(4):
            if kinds[i] == kind:
                s = slice(starts[i], starts[i + 1])
                assert torch.equal(P[i], Q[i]) and torch.equal(m[s], mq[s]) and torch.equal(v[s], vq[s])
                at += 1
    assert at == 4
    # one type for gradients of one type of parameters
    opt = mm.AdamW8([put(x, t)[0] for x, t in zip(vals, kinds)])
    with pytest.raises(ValueError):
        opt.step([put(x, t)[0] for x, t in zip(grads[0], ["bf16", "f32", "f32", "f32"])])
    assert opt.step_count == 0
    W = [torch.randn(64, 96, device=dev()).bfloat16()]
    A = [put(x, t)[0] for x, t in zip(vals, kinds)]
    both = mm.PeriodicMuon(W, aux_params=A, aux_bits=8)
    before = [a.clone() for a in A]
    both.step([torch.randn_like(W[0])], [put(x, t)[0] for x, t in zip(grads[0], kinds)])
    assert all(not torch.equal(a, b) for a, b in zip(A, before))


def test_linear_ce_backward_long_sums():
    """dW over 2^22 rows whose products all have one sign: the tensor cores' truncation must
    not pile up.  W = 0, so every probability is 2^-8 exactly and dW[v] = 2^-8 sum_r h[r] for a
    column that is no row's label.  Between take-overs of the sums lie 2^16 products at most,
    2^12 additions of 16 products with an error of 2u each; then a rounding to bf16."""
    n, v, d = 1 << 22, 256, 64
    gen = torch.Generator(device=dev())
    gen.manual_seed(1)
    h = (torch.rand(n, d, generator=gen, device=dev()) + 0.5).bfloat16()
    w = torch.zeros(v, d, device=dev(), dtype=torch.bfloat16)
    labels = torch.randint(0, v // 2, (n,), generator=gen, device=dev())
    ws = mm.alloc_linear_ce_workspace(n, v, d)
    lse = torch.full((n,), float(np.log(256.0)), device=dev())
    _, dw = mm.muon_linear_ce_backward(h, w, labels, lse, ws, need_dh=False)
    assert mm.muon_check_status(ws) == mm.MUON_OK
    want = num(h.double().sum(0)) / 256
    within(num(dw[v // 2:]), np.broadcast_to(want, (v // 2, d)), np.broadcast_to((BF + 4096 * 2 * U + 64 * U) * want, (v // 2, d)),
           "dw")


def test_linear_ce_backward_long_vocabulary():
    """dH of few rows over a vocabulary of 2^21 entries, all products of one sign."""
    n, v, d = 40, 1 << 21, 64
    gen = torch.Generator(device=dev())
    gen.manual_seed(2)
    h = torch.zeros(n, d, device=dev(), dtype=torch.bfloat16)
    w = (torch.rand(v, d, generator=gen, device=dev()) + 0.5).bfloat16()
    labels = torch.zeros(n, dtype=torch.int64, device=dev())
    ws = mm.alloc_linear_ce_workspace(n, v, d)
    lse = torch.full((n,), float(np.log(256.0)), device=dev())
    dh, _ = mm.muon_linear_ce_backward(h, w, labels, lse, ws, need_dw=False)
    assert mm.muon_check_status(ws) == mm.MUON_OK
    want = num(w.double().sum(0)) / 256 - num(w[0])
    within(num(dh), np.broadcast_to(want, (n, d)), np.broadcast_to((BF + 4096 * 2 * U + 64 * U) * want, (n, d)), "dh")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mask", ["lowest", "minus infinity"])
def test_linear_ce_vocabulary_masked_by_a_bias_column(dt, mask):
    """Entries shut out by the type's lowest value (or minus infinity) in a column that every
    hidden state holds 1 in: their logits vanish, the others' loss is what it is without them."""
    n, v, d = 70, 700, 64
    h, h64, w, w64, labels, lab = ce_case(n, v, d, dt, 12)
    low = torch.finfo(TYPES[dt]).min if mask == "lowest" else float("-inf")
    shut = np.arange(v) % 5 == 2
    h[:, -1] = 1.0
    w[:, -1] = torch.from_numpy(np.where(shut, low, 0.0)).to(dev(), w.dtype)
    lab = np.where((lab >= 0) & shut[lab], lab - 1, lab)
    labels = torch.from_numpy(lab).to(dev())
    ws = mm.alloc_linear_ce_workspace(n, v, d, TYPES[dt])
    loss, lse, stats = mm.muon_linear_ce_forward(h, w, labels, ws)
    h64, w64 = num(h), num(w)
    keep = np.flatnonzero(~shut)
    place = np.where(lab >= 0, np.searchsorted(keep, np.maximum(lab, 0)), lab)
    rloss, rlse, rmean, count = ref.linear_ce_forward(h64, w64[keep], place)
    ez = ce_tolerances(h64, w64[keep], dt)
    spread = np.abs(h64 @ w64[keep].T).max(1) + 1
    elog = ez + (v / 32 + 64 + 4 * spread) * U + 4 * U * np.abs(rlse)
    within(num(lse), rlse, elog, "lse")
    within(num(loss), rloss, elog + ez + 2 * U * np.abs(rlse), "loss")
    if mask == "lowest":
        dh, dw = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats)
        assert torch.isfinite(dh).all() and torch.isfinite(dw).all() and not dw[torch.from_numpy(shut).to(dev())].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_linear_ce_nan_and_infinite_logits_stay_nan(bad):
    for dt in ("bf16", "f32"):
        h, h64, w, w64, labels, lab = ce_case(20, 300, 64, dt, 13)
        h[3, 5], w[:, 5] = bad, 1.0
        loss, lse, _ = mm.muon_linear_ce_forward(h, w, labels.clamp(min=0), mm.alloc_linear_ce_workspace(20, 300, 64, TYPES[dt]))
        assert torch.isnan(loss[3]) and torch.isnan(lse[3])
        rest = torch.arange(20, device=dev()) != 3
        assert torch.isfinite(loss[rest]).all() and torch.isfinite(lse[rest]).all()


def test_second_derivatives_are_refused():
    x = torch.randn(5, 64, device=dev(), requires_grad=True)
    w = torch.randn(64, device=dev(), requires_grad=True)
    g, = torch.autograd.grad(mm.layer_norm(x, w).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (g.square().sum() + x.sum()).backward()
    v = torch.randn(100, 64, device=dev(), requires_grad=True)
    labels = torch.arange(5, device=dev())
    g, = torch.autograd.grad(mm.linear_cross_entropy(x, v, labels), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (g.square().sum() + x.sum()).backward()


def pieces_of(v, columns):
    """The pieces that so many columns a piece make of v entries: of one size, as far as tiles of 256 allow."""
    n = -(-v // columns)
    size = -(-(-(-v // n)) // 256) * 256
    return -(-v // size)


PIECE_SIZES = [(1, 3000, 40), (5, 3111, 65), (64, 3001, 257), (129, 3300, 96), (257, 4001, 200), (300, 3107, 321), (700, 5050, 130),
               (1000, 3000, 32)]


@pytest.mark.parametrize("columns", [256, 512])
@pytest.mark.parametrize("size", PIECE_SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_ce_backward_in_pieces(dt, size, columns):
    """Six pieces of the vocabulary or more, the last one short: g in two buffers in turn, dH's
    running sums over them, offsets into W, labels of other pieces, launches of all three
    products, dH's ranges of K (few rows) and none."""
    n, v, d = size
    npieces = pieces_of(v, columns)
    assert npieces >= 6
    h, h64, w, w64, labels, lab = ce_case(n, v, d, dt, n + v + d)
    plain = mm.alloc_linear_ce_workspace(n, v, d, TYPES[dt])
    _, lse, stats = mm.muon_linear_ce_forward(h, w, labels, plain)
    rg, rg64 = put(np.random.default_rng(3).random(n), "f32")
    whole = mm.muon_linear_ce_backward(h, w, labels, lse, plain, row_grad=rg)
    mm.muon_debug_set(mm.MUON_DEBUG_CE_PIECE * (columns // 256), 0)
    try:
        ws = mm.alloc_linear_ce_workspace(n, v, d, TYPES[dt])
        ws[256:].fill_(255)                       # NaN in every sum that is not written first
        dh, dw = mm.muon_linear_ce_backward(h, w, labels, lse, ws, row_grad=rg)
        # a launch a piece and one more, the operands' copies and the last kernel
        assert npieces + 2 <= mm.muon_launch_count() <= npieces + 4
        assert mm.muon_check_status(ws) == mm.MUON_OK
        again = mm.muon_linear_ce_backward(h, w, labels, lse, ws, row_grad=rg)
        only = (mm.muon_linear_ce_backward(h, w, labels, lse, ws, row_grad=rg, need_dw=False)[0],
                mm.muon_linear_ce_backward(h, w, labels, lse, ws, row_grad=rg, need_dh=False)[1])
        mean = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats, grad_scale=3.0)
        assert mm.muon_check_status(ws) == mm.MUON_OK
    finally:
        mm.muon_debug_set(0, 0)
    assert torch.equal(dw, whole[1])              # a column's sum over rows does not depend on the pieces
    assert all(torch.equal(p, q) for p, q in zip((dh, dw), again)) and all(torch.equal(p, q) for p, q in zip((dh, dw), only))
    lse64, z = num(lse), h64 @ w64.T
    ez = ce_tolerances(h64, w64, dt)
    spread = np.abs(z).max(1) + 1
    count = max((lab != -100).sum(), 1)
    for got, coef in (((dh, dw), rg64), (mean, np.full(n, 3.0 / count))):
        g = ref.linear_ce_logit_grad(h64, w64, lab, lse64, coef)
        counted = (lab != -100) * coef
        eg = counted[:, None] * np.exp(z - lse64[:, None]) * (ez + (16 + 4 * spread) * U)[:, None] + 8 * U * np.abs(g) + \
            4 * U * counted[:, None]
        parts, one = (1, BF) if dt == "bf16" else (4, 0.0)
        if dt == "bf16":
            eg = eg + BF * (np.abs(g) + eg)
        # an fp32 addition a piece on top of a whole vocabulary's sum
        edh = eg @ np.abs(w64) + parts * (v / 16 + 64 + npieces) * 2 * U * (np.abs(g) @ np.abs(w64))
        edw = eg.T @ np.abs(h64) + parts * (n / 16 + 64) * 2 * U * (np.abs(g).T @ np.abs(h64))
        within(num(got[0]), g @ w64, edh + one * (np.abs(g @ w64) + edh) + 1e-30, "dh")
        within(num(got[1]), g.T @ h64, edw + one * (np.abs(g.T @ h64) + edw) + 1e-30, "dw")
        assert not got[0][labels == -100].any()


def test_linear_ce_backward_in_pieces_on_their_own():
    """The pieces of 268 million logits that a larger case makes without any flag."""
    n, v, d = 4096, 131073, 48
    gen = torch.Generator(device=dev())
    gen.manual_seed(5)
    w = (torch.randn(v, d, generator=gen, device=dev()) * 2 / d ** 0.5).bfloat16()
    labels = torch.randint(0, v, (n,), generator=gen, device=dev())
    h = (torch.randn(n, d, generator=gen, device=dev()) + w[labels].float()).bfloat16()
    labels[::7] = -100
    ws = mm.alloc_linear_ce_workspace(n, v, d)
    _, lse, stats = mm.muon_linear_ce_forward(h, w, labels, ws)
    got = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats)
    # H's copy, a launch a piece and one more, the last kernel
    assert mm.muon_launch_count() == pieces_of(v, 65536) + 3 and mm.muon_check_status(ws) == mm.MUON_OK
    check_ce_backward_on_gpu(h, w, labels, lse, got)


def test_linear_ce_backward_more_tiles_than_the_table_holds():
    """A launch of two products whose 13282 and more tiles go round robin."""
    n, v, d = 8, 1_700_003, 512
    gen = torch.Generator(device=dev())
    gen.manual_seed(6)
    w = (torch.randn(v, d, generator=gen, device=dev()) * 2 / d ** 0.5).bfloat16()
    labels = torch.randint(0, v, (n,), generator=gen, device=dev())
    h = (torch.randn(n, d, generator=gen, device=dev()) + 2 * w[labels].float()).bfloat16()
    labels[3] = -100
    ws = mm.alloc_linear_ce_workspace(n, v, d)
    _, lse, stats = mm.muon_linear_ce_forward(h, w, labels, ws)
    got = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats)
    assert mm.muon_check_status(ws) == mm.MUON_OK
    check_ce_backward_on_gpu(h, w, labels, lse, got)


def check_ce_backward_on_gpu(h, w, labels, lse, got):
    """The mean loss's gradients against 64 bits on the GPU, bf16, the vocabulary in slices."""
    h64, live = h.double(), (labels != -100).double()
    n, v, c = h.shape[0], w.shape[0], live / live.sum()
    dh, edh = torch.zeros_like(h64), torch.zeros_like(h64)
    at = torch.arange(n, device=h.device)
    step = (1 << 27) // n
    for a in range(0, v, step):
        wp = w[a:a + step].double()
        z = h64 @ wp.T
        p = torch.exp(z - lse.double()[:, None])
        here = (labels >= a) & (labels < a + step)
        g = p.clone()
        g[at[here], labels[here] - a] -= 1
        g *= c[:, None]
        ez = (h.shape[1] / 16 + 16) * 2 * U * (h64.abs() @ wp.abs().T)
        eg = c[:, None] * p * (ez + (20 + 4 * z.abs()) * U) + 8 * U * g.abs() + 4 * U * c[:, None]
        eg += BF * (g.abs() + eg)
        dh += g @ wp
        edh += eg @ wp.abs() + (v / 16 + 64) * 2 * U * (g.abs() @ wp.abs())
        dw, edw = g.T @ h64, eg.T @ h64.abs() + (n / 16 + 64) * 2 * U * (g.abs().T @ h64.abs())
        bad = (got[1][a:a + step].double() - dw).abs() > edw + BF * (dw.abs() + edw) + 1e-30
        assert not bad.any(), ("dw", a, int(bad.sum()))
    bad = (got[0].double() - dh).abs() > edh + BF * (dh.abs() + edh) + 1e-30
    assert not bad.any(), ("dh", int(bad.sum()))


ROW_CASES = [(6000, 1536, "bf16", 0), (6000, 1544, "bf16", 0), (5000, 1540, "f32", 0), (5003, 1537, "f32", 3),
             (6001, 1537, "bf16", 1), (2000, 8192, "bf16", 0), (1500, 8192, "f32", 0), (9000, 520, "bf16", 8), (9000, 1000, "f32", 0),
             (12000, 300, "f32", 5), (2500, 5001, "bf16", 0), (600, 12288, "bf16", 0), (500, 9001, "f32", 1)]


@pytest.mark.parametrize("n,d,xdt,pad", ROW_CASES)
def test_layernorm_backward_many_rows_a_group(n, d, xdt, pad):
    """Eight rows or more through each of the backward pass's row groups: its ring of copies
    wraps, the barriers' buffers alternate, sums run on."""
    rng = np.random.default_rng(n + d)
    x, x64 = put(rng.standard_normal((n, d)) * 2 + 0.5, xdt)
    dy, dy64 = put(rng.standard_normal((n, d)), xdt)
    w, w64 = put(1 + 0.3 * rng.standard_normal(d), "f32")
    xs, dys = strided(x, pad), strided(dy, pad)
    y, mean, rstd = mm.muon_layernorm_forward(xs, w, w)
    ws = mm.alloc_layernorm_workspace(n, d)
    dx, dw, db = mm.muon_layernorm_backward(dys, xs, w, mean, rstd, ws)
    ws.fill_(255)
    again = mm.muon_layernorm_backward(dys, xs, w, mean, rstd, ws)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))
    check_layernorm(xdt, n, d, x64, dy64, w64, w64, (y, mean, rstd), (dx, dw, db))


@pytest.mark.parametrize("off", [1, 2, 3, 5])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_layernorm_unaligned_views_to_their_own_precision(xdt, off):
    rng = np.random.default_rng(off)
    n, d = 9, 1536
    flat, f64 = put(rng.standard_normal(off + n * d) * 2 + 0.5, xdt)
    dflat, d64 = put(rng.standard_normal(off + n * d), xdt)
    wf, wf64 = put(1 + 0.3 * rng.standard_normal(off + d), "f32")
    x, dy, w = flat[off:].view(n, d), dflat[off:].view(n, d), wf[off:]
    y, mean, rstd = mm.muon_layernorm_forward(x, w, w)
    got = mm.muon_layernorm_backward(dy, x, w, mean, rstd, mm.alloc_layernorm_workspace(n, d))
    check_layernorm(xdt, n, d, f64[off:].reshape(n, d), d64[off:].reshape(n, d), wf64[off:], wf64[off:], (y, mean, rstd), got)


def check_layernorm(xdt, n, d, x64, dy64, w64, b64, forward, backward):
    """test_layernorm's bounds, with an fp32 weight and bias."""
    (y, mean, rstd), (dx, dw, db) = forward, backward
    gam, one = (d / 32 + 32) * U, BF if xdt == "bf16" else 0.0
    ry, rmean, rrstd = ref.layernorm_forward(x64, w64, b64, 1e-5)
    emean = gam * np.abs(x64).mean(1) + U * np.abs(rmean)
    within(num(mean), rmean, emean, "mean")
    cen = np.abs(x64 - rmean[:, None])
    ev = (2 * (emean[:, None] + U * cen) * cen).mean(1) + emean ** 2 + gam * (cen ** 2).mean(1)
    er = rrstd * (0.5 * ev * rrstd ** 2 + 8 * U)
    within(num(rstd), rrstd, er, "rstd")
    exh = (emean[:, None] + U * cen) * rrstd[:, None] + cen * er[:, None]
    ey = exh * np.abs(w64) + 4 * U * (np.abs(ry) + cen * rrstd[:, None] * np.abs(w64)) + one * np.abs(ry)
    within(num(y), ry, ey * 1.01 + 1e-30, "y")
    m64, r64 = num(mean), num(rstd)
    rdx, rdw, rdb = ref.layernorm_backward(dy64, x64, w64, m64, r64)
    xh, g = (x64 - m64[:, None]) * r64[:, None], dy64 * w64
    eg, exh = 2 * U * np.abs(g), 3 * U * np.abs(xh)
    c1, c2 = np.abs(g).mean(1, keepdims=True), np.abs(g * xh).mean(1, keepdims=True)
    edx = r64[:, None] * (eg + (gam + 4 * U) * c1 + np.abs(xh) * (gam + 8 * U) * c2 + exh * c2 +
                          4 * U * (np.abs(g) + c1 + np.abs(xh) * c2)) + one * np.abs(rdx)
    within(num(dx), rdx, edx * 1.01 + 1e-30, "dx")
    within(num(dw), rdw, (n + 8) * U * np.abs(dy64 * xh).sum(0) + 1e-30, "dw")
    within(num(db), rdb, (n + 8) * U * np.abs(dy64).sum(0) + 1e-30, "db")


def test_layernorm_past_32_bit_offsets():
    """More than 2^31 elements: the last rows are, bit for bit, what they are by themselves."""
    n, d, k = 2_200_003, 1024, 500
    gen = torch.Generator(device=dev())
    gen.manual_seed(8)
    x = torch.empty(n, d, device=dev(), dtype=torch.bfloat16).normal_(generator=gen)
    w = torch.rand(d, generator=gen, device=dev()) + 0.5
    y, mean, rstd = mm.muon_layernorm_forward(x, w, w)
    ws = mm.alloc_layernorm_workspace(n, d)
    dx, dw, db = mm.muon_layernorm_backward(y, x, w, mean, rstd, ws)
    for s in (slice(0, k), slice(n - k, n)):
        part = mm.muon_layernorm_forward(x[s], w, w)
        assert all(torch.equal(a, b) for a, b in zip(part, (y[s], mean[s], rstd[s])))
        assert torch.equal(mm.muon_layernorm_backward(y[s], x[s], w, mean[s], rstd[s], ws)[0], dx[s])
    sums = [torch.zeros(d, dtype=torch.float64, device=dev()) for _ in range(4)]
    for a in range(0, n, 1 << 18):
        g = y[a:a + (1 << 18)].double()
        p = g * (x[a:a + (1 << 18)].double() - mean[a:a + (1 << 18), None].double()) * rstd[a:a + (1 << 18), None].double()
        for t, q in zip(sums, (p, p.abs(), g, g.abs())):
            t += q.sum(0)
    # a CTA's running sums take its share of the rows, then at most 152 lines are added
    rows = n / 152 + 152 + 8
    within(num(dw), num(sums[0]), rows * U * num(sums[1]), "dw")
    within(num(db), num(sums[2]), rows * U * num(sums[3]), "db")


def test_linear_ce_past_32_bit_offsets():
    """H, then W, of more than 2^31 elements, and rows of H further apart than they are long."""
    gen = torch.Generator(device=dev())
    gen.manual_seed(9)
    d, k = 2048, 256
    wide = torch.empty(1_050_003, d, device=dev(), dtype=torch.bfloat16).normal_(generator=gen)
    few = torch.empty(300, d, device=dev(), dtype=torch.bfloat16).normal_(std=0.05, generator=gen)
    n = wide.shape[0]
    labels = torch.randint(0, 300, (n,), generator=gen, device=dev())
    ws = mm.alloc_linear_ce_workspace(n, 300, d)
    loss, lse, _ = mm.muon_linear_ce_forward(wide, few, labels, ws)
    dh, dw = mm.muon_linear_ce_backward(wide, few, labels, lse, ws)
    assert mm.muon_check_status(ws) == mm.MUON_OK
    for s in (slice(0, k), slice(n - k, n)):
        p = mm.muon_linear_ce_forward(wide[s], few, labels[s], ws)
        assert torch.equal(p[0], loss[s]) and torch.equal(p[1], lse[s])
        q = mm.muon_linear_ce_backward(wide[s], few, labels[s], lse[s], ws, need_dw=False)[0]
        assert torch.linalg.norm(q.float() - dh[s].float()) <= 2 * BF * torch.linalg.norm(q.float())
    want = torch.zeros(300, d, dtype=torch.float64, device=dev())
    for a in range(0, n, 1 << 16):
        h = wide[a:a + (1 << 16)].double()
        g = torch.exp(h @ few.double().T - lse[a:a + (1 << 16), None].double())
        g[torch.arange(len(h), device=dev()), labels[a:a + (1 << 16)]] -= 1
        want += g.T @ h
    assert torch.linalg.norm(dw.double() - want) <= 2 * BF * torch.linalg.norm(want)
    del dh, dw
    # the other way round: 300 rows against the long matrix as the vocabulary
    labels = torch.randint(n - 1000, n, (300,), generator=gen, device=dev())
    ws = mm.alloc_linear_ce_workspace(300, n, d)
    loss, lse, _ = mm.muon_linear_ce_forward(few, wide, labels, ws)
    dh, dw = mm.muon_linear_ce_backward(few, wide, labels, lse, ws)
    assert mm.muon_check_status(ws) == mm.MUON_OK
    z = torch.cat([few.double() @ wide[a:a + (1 << 16)].double().T for a in range(0, n, 1 << 16)], 1)
    rl = torch.logsumexp(z, 1)
    assert (lse - rl).abs().max() < 1e-4 and (loss - (rl - z.gather(1, labels[:, None])[:, 0])).abs().max() < 1e-4
    g = torch.exp(z - lse.double()[:, None])
    g[torch.arange(300, device=dev()), labels] -= 1
    want = sum(g[:, a:a + (1 << 16)] @ wide[a:a + (1 << 16)].double() for a in range(0, n, 1 << 16))
    assert torch.linalg.norm(dh.double() - want) <= 2 * BF * torch.linalg.norm(want)
    for s in (slice(0, 5000), slice(n - 5000, n)):
        want = g[:, s].T @ few.double()
        assert torch.linalg.norm(dw[s].double() - want) <= 2 * BF * torch.linalg.norm(want)
    # rows 2^25 elements apart
    del wide, dh, dw, z, g, want
    buf = torch.empty(70 << 25, device=dev(), dtype=torch.bfloat16)
    far = buf.view(70, 1 << 25)[:, 8:8 + d]
    far.copy_(few[:70])
    labels = torch.randint(0, 300, (70,), generator=gen, device=dev())
    ws = mm.linear_ce_workspace_for(far, few, labels)
    got = mm.muon_linear_ce_forward(far, few, labels, ws)
    got += mm.muon_linear_ce_backward(far, few, labels, got[1], ws, stats=got[2])
    near = far.clone()
    want = mm.muon_linear_ce_forward(near, few, labels, ws)
    want += mm.muon_linear_ce_backward(near, few, labels, want[1], ws, stats=want[2])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_adamw8_past_32_bit_offsets():
    """More than 2^32 elements in one parameter, and another behind it: the oracle's update and
    its random bits at both ends and around 2^31 and 2^32."""
    n = (1 << 32) + 70_003
    gen = torch.Generator(device=dev())
    gen.manual_seed(10)
    p = torch.full((n,), 0.5, device=dev(), dtype=torch.bfloat16)
    g = torch.empty(n, device=dev(), dtype=torch.bfloat16).normal_(std=1e-3, generator=gen)
    p2, g2 = p[:5000].clone(), g[:5000].clone()
    opt = mm.AdamW8([p, p2], lr=1e-2, betas=(0.9, 0.999), seed=99)
    opt.step([g, g2])
    m, v = opt.moments()
    for q, grad, first, spots in ((p, g, 0, (0, (1 << 31) - 640, (1 << 32) - 640, n - n % 128 - 1152)), (p2, g2, opt.starts[1], (0, 3712))):
        for a in spots:
            k = min(1280, q.numel() - a)
            x = num(grad[a:a + k])
            want, em, ev = ref.adamw8_update(np.full(k, 0.5), x, 0.0, 0.0, 1, 1e-2, 0.9, 0.999, 1e-8, 0.0)
            within(num(q[a:a + k]), want, 16 * U + BF * 1.01 * np.abs(want), ("p", a))
            blocks = -(-k // 128) * 128
            at = first + a
            bits = ref.random_bits(99, 1, at + np.arange(blocks)).astype(np.int64)
            compare_codes(opt.m[at:at + blocks].cpu().numpy(), opt.m_scale[at // 128:(at + blocks) // 128].cpu().numpy(), padded(em),
                          bits & 0xFFFF, 127, 16, 4 * U, ("m", a))
            compare_codes(opt.v[at:at + blocks].cpu().numpy(), opt.v_scale[at // 128:(at + blocks) // 128].cpu().numpy(), padded(ev),
                          bits >> 16, 255, 32, 8 * U, ("v", a))
            assert np.array_equal(num(m[at:at + blocks]), ref.decode(opt.m[at:at + blocks].cpu().numpy(),
                                                                     opt.m_scale[at // 128:(at + blocks) // 128].cpu().numpy(), True))
            assert np.array_equal(num(v[at:at + blocks]), ref.decode(opt.v[at:at + blocks].cpu().numpy(),
                                                                     opt.v_scale[at // 128:(at + blocks) // 128].cpu().numpy(), False))
