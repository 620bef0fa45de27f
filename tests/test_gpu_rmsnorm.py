"""RMS norm behind a residual's addition, its 8-bit output and its gradient, on the GPU
against the fp64 oracle.

Tolerances come from the arithmetic.  u = 2^-24 is fp32's rounding error, 2^-8 bf16's
half-spacing, 2^-4 e4m3's (2^-10 of the scale below its smallest normal number).  Every
kernel keeps at least 32 running sums a row, so a sum over a row of D is within (D/32 + 32) u
of the sum of its terms' magnitudes."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm
from oracle import head_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


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


def strided(t, pad, off=0):
    """The same values as rows of a wider buffer that starts `off` elements late."""
    if not pad and not off:
        return t
    n, d = t.shape
    b = torch.full((off + n * (d + pad),), float("nan"), dtype=t.dtype, device=t.device)
    b = b[off:].view(n, d + pad)[:, :d]
    b.copy_(t)
    return b


def check_forward(x, x64, w, w64, r, r64, xdt, what):
    one = BF if xdt == "bf16" else U
    n, d = x64.shape
    y, rstd, total = mm.muon_rmsnorm_forward(x, w, r, eps=EPS)
    if r is not None:
        within(num(total), x64 + r64, 1.01 * one * np.abs(x64 + r64), ("total",) + what)
    else:
        assert total is x
    t64 = num(total)
    ry, rrstd = ref.rmsnorm_forward(t64, w64, EPS)
    rel = 0.5 * ((d / 32 + 32) * U + 2 * U) + 4 * U        # of rstd = v^-1/2
    within(num(rstd), rrstd, rel * rrstd, ("rstd",) + what)
    within(num(y), ry, (rel + 3 * U + (BF if xdt == "bf16" else 0)) * np.abs(ry) * 1.01, ("y",) + what)
    # 8 bits, from the same inputs
    codes, scales, rstd8, total8 = mm.muon_rmsnorm_forward_fp8(x, w, r, eps=EPS)
    # (rows that start off a 16-byte boundary add their squares in another order here: the bound
    # holds for any order, so it holds for both)
    within(num(rstd8), rrstd, rel * rrstd, ("rstd8",) + what)
    assert torch.equal(total8, total)
    rq, rscale = ref.eight_bits(ry)
    within(num(scales), rscale, (rel + 6 * U) * rscale, ("scale",) + what)
    s = np.repeat(num(scales), 128, 1)[:, :d]
    value = num(codes.float()) * s
    within(value, ry, np.maximum(2.0 ** -4 * np.abs(ry), 2.0 ** -10 * s) * 1.001 + (rel + 8 * U) * np.abs(ry), ("codes",) + what)
    return rstd, total


def check_backward(dy, dy64, total, w, w64, rstd, dt, dt64, xdt, wdt, what):
    t64, r64 = num(total), num(rstd)
    n, d = t64.shape
    ws = mm.alloc_rmsnorm_workspace(n, d) if w is not None else None
    dx, dw = mm.muon_rmsnorm_backward(dy, total, w, rstd, ws, dtotal=dt)
    rdx, rdw = ref.rmsnorm_backward(dy64, t64, w64, r64, dt64)
    xh = t64 * r64[:, None]
    g = np.abs(dy64 * (w64 if w is not None else 1.0))
    c = (g * np.abs(xh)).mean(1, keepdims=True)
    ec = ((d / 32 + 32) * U + 6 * U) * c
    e = r64[:, None] * (2 * U * g + np.abs(xh) * (ec + 4 * U * c) + 3 * U * (g + np.abs(xh) * c)) + 2 * U * np.abs(rdx)
    e = e + 2 * U * (np.abs(dt64) if dt is not None else 0.0)
    within(num(dx), rdx, 1.01 * (e + (BF if xdt == "bf16" else 0.0) * np.abs(rdx)) + 1e-30, ("dx",) + what)
    if w is None:
        assert dw is None
    else:
        one = BF if wdt == "bf16" else 0.0
        within(num(dw), rdw, 1.01 * ((n + 8) * U * np.abs(dy64 * xh).sum(0) + one * np.abs(rdw)) + 1e-30, ("dw",) + what)


SIZES = [(1, 1), (3, 1), (1, 2), (5, 3), (1, 7), (7, 31), (2, 32), (9, 33), (4, 64), (33, 127), (5, 128), (3, 129), (5, 255),
         (3, 256), (6, 257), (160, 512), (2, 1000), (311, 1024), (3, 1025), (17, 1536), (2, 2047), (5, 2560), (3, 4096),
         (2, 4099), (4, 5120), (3, 8192), (2, 8200), (2, 12288), (3, 16384), (1, 16391), (2, 40000), (1, 65536), (2, 70000)]


@pytest.mark.parametrize("pad", [0, 8, 5])
@pytest.mark.parametrize("wdt", ["bf16", "f32", None])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_rmsnorm(xdt, residual, wdt, pad):
    rng = np.random.default_rng(7)
    for n, d in SIZES:
        x, x64 = put(rng.standard_normal((n, d)) * 2, xdt)
        r, r64 = put(rng.standard_normal((n, d)) * 3, xdt) if residual else (None, None)
        w, w64 = put(1 + 0.3 * rng.standard_normal(d), wdt) if wdt else (None, None)
        x, r = strided(x, pad), strided(r, pad) if residual else None
        rstd, total = check_forward(x, x64, w, w64, r, r64, xdt, (n, d))
        dy, dy64 = put(rng.standard_normal((n, d)), xdt)
        dt, dt64 = put(rng.standard_normal((n, d)), xdt) if residual else (None, None)
        check_backward(strided(dy, pad), dy64, strided(total, pad), w, w64, rstd, dt, dt64, xdt, wdt, (n, d))


@pytest.mark.parametrize("off", [1, 2, 3, 5])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_rmsnorm_unaligned_views(xdt, off):
    """Rows and weights that start off every vector boundary."""
    rng = np.random.default_rng(9)
    for n, d in ((5, 64), (40, 250), (7, 1536), (3, 9001)):
        x, x64 = put(rng.standard_normal((n, d)), xdt)
        r, r64 = put(rng.standard_normal((n, d)), xdt)
        dy, dy64 = put(rng.standard_normal((n, d)), xdt)
        w, w64 = put(np.concatenate([np.full(off, np.nan), 1 + 0.2 * rng.standard_normal(d)]), "f32")
        w, w64 = w[off:], w64[off:]
        rstd, total = check_forward(strided(x, 3, off), x64, w, w64, strided(r, 1, off), r64, xdt, (n, d))
        check_backward(strided(dy, 2, off), dy64, strided(total, 5, off), w, w64, rstd, strided(r, 7, off), r64, xdt, "f32", (n, d))


ROW_CASES = [(20011, 192, "bf16", 0), (5003, 1537, "f32", 3), (3001, 1536, "bf16", 0), (4001, 100, "f32", 0),
             (2000, 2562, "bf16", 0), (700, 8192, "bf16", 0), (500, 8193, "bf16", 0), (400, 12288, "f32", 0)]


@pytest.mark.parametrize("n,d,xdt,pad", ROW_CASES)
def test_rmsnorm_many_rows_and_repeatability(n, d, xdt, pad):
    """More rows than run at once; the same inputs give the same bits, whatever the workspace held."""
    rng = np.random.default_rng(8)
    x, x64 = put(rng.standard_normal((n, d)), xdt)
    r, r64 = put(rng.standard_normal((n, d)), xdt)
    dy, dy64 = put(rng.standard_normal((n, d)), xdt)
    w, w64 = put(1 + 0.3 * rng.standard_normal(d), "f32")
    x, r, dy = strided(x, pad), strided(r, pad), strided(dy, pad)
    rstd, total = check_forward(x, x64, w, w64, r, r64, xdt, (n, d))
    check_backward(dy, dy64, total, w, w64, rstd, r, r64, xdt, "f32", (n, d))
    ws = mm.alloc_rmsnorm_workspace(n, d)
    a = mm.muon_rmsnorm_backward(dy, total, w, rstd, ws, dtotal=r)
    ws.fill_(255)
    b = mm.muon_rmsnorm_backward(dy, total, w, rstd, ws, dtotal=r)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rmsnorm_options():
    """total left out; dx without the weight's gradient needs no workspace; empty batches."""
    x, r = (torch.randn(6, 300, device=dev()) for _ in range(2))
    w = torch.randn(300, device=dev())
    y, rstd, total = mm.muon_rmsnorm_forward(x, w, r)
    y2, rstd2, none = mm.muon_rmsnorm_forward(x, w, r, need_total=False)
    assert none is None and torch.equal(y, y2) and torch.equal(rstd, rstd2)
    big, wide = torch.randn(2, 70001, device=dev()), torch.randn(2, 70001, device=dev())
    assert torch.equal(mm.muon_rmsnorm_forward(big, None, wide)[0], mm.muon_rmsnorm_forward(big, None, wide, need_total=False)[0])
    dx, dw = mm.muon_rmsnorm_backward(x, total, w, rstd, weight_grad=False)
    assert dw is None and torch.equal(dx, mm.muon_rmsnorm_backward(x, total, w, rstd, mm.alloc_rmsnorm_workspace(6, 300))[0])
    with pytest.raises(mm.MuonError):
        mm.muon_rmsnorm_backward(x, total, w, rstd)
    with pytest.raises(mm.MuonError):
        mm.muon_rmsnorm_backward(x, total, w, rstd, mm.alloc_rmsnorm_workspace(6, 300)[:256])
    e = torch.empty(0, 40, device=dev())
    y, rstd, total = mm.muon_rmsnorm_forward(e, w[:40], e)
    assert y.shape == (0, 40) and rstd.shape == (0,) and total.shape == (0, 40)
    codes, scales, _, _ = mm.muon_rmsnorm_forward_fp8(e)
    assert codes.shape == (0, 40) and scales.shape == (0, 1)
    dx, dw = mm.muon_rmsnorm_backward(e, e, w[:40], rstd, mm.alloc_rmsnorm_workspace(0, 40))
    assert dx.shape == (0, 40) and dw.shape == (40,) and not dw.any()


def test_rmsnorm_in_place():
    """Through the C entry point: total over the residual or x, y over x, dx over dy or dtotal."""
    lib = mm.load_library()
    for d in (64, 77, 1536, 9000, 70000):
        for dt in (torch.bfloat16, torch.float32):
            code = mm.MUON_DTYPE_BF16 if dt == torch.bfloat16 else mm.MUON_DTYPE_F32
            x, r, dy, dtot = (torch.randn(5, d, device=dev()).to(dt) for _ in range(4))
            y, rstd, total = mm.muon_rmsnorm_forward(x, None, r)
            for keep in ("r", "x"):
                a, b = x.clone(), r.clone()
                t, o = (b, a) if keep == "r" else (a, torch.empty_like(a))
                assert lib.muon_rmsnorm_forward(a.data_ptr(), d, b.data_ptr(), d, None, 5, d, code, code, 1e-6, t.data_ptr(), d,
                                                o.data_ptr(), d, None, 0, None, None, torch.cuda.current_stream().cuda_stream) == 0
                assert torch.equal(t, total) and torch.equal(o, y)
            want, _ = mm.muon_rmsnorm_backward(dy, total, None, rstd, dtotal=dtot)
            for over in (0, 1):
                a, b = dy.clone(), dtot.clone()
                o = b if over else a
                assert lib.muon_rmsnorm_backward(a.data_ptr(), d, total.data_ptr(), d, None, rstd.data_ptr(), b.data_ptr(), d, 5, d,
                                                 code, code, o.data_ptr(), d, None, None, 0,
                                                 torch.cuda.current_stream().cuda_stream) == 0
                assert torch.equal(o, want)
            w = torch.randn(d, device=dev())
            ws = mm.alloc_rmsnorm_workspace(5, d)
            want, wantw = mm.muon_rmsnorm_backward(dy, total, w, rstd, ws, dtotal=dtot)
            a, dw = dy.clone(), torch.empty_like(w)
            assert lib.muon_rmsnorm_backward(a.data_ptr(), d, total.data_ptr(), d, w.data_ptr(), rstd.data_ptr(), dtot.data_ptr(), d, 5, d,
                                             code, 0, a.data_ptr(), d, dw.data_ptr(), ws.data_ptr(), ws.numel(),
                                             torch.cuda.current_stream().cuda_stream) == 0
            assert torch.equal(a, want) and torch.equal(dw, wantw)


def test_rmsnorm_zeros_extremes_and_nonfinite():
    x = torch.zeros(4, 300, device=dev())
    x[1] = 1e-30
    x[2] = 1e15
    x[3, 5] = 7.0
    w = torch.full((300,), 2.0, device=dev())
    y, rstd, _ = mm.muon_rmsnorm_forward(x, w, eps=1e-6)
    assert not y[0].any() and abs(rstd[0].item() - 1000) < 1e-3 and torch.allclose(y[2], w) and torch.isfinite(y).all()
    codes, scales, _, _ = mm.muon_rmsnorm_forward_fp8(x, w, eps=1e-6)
    c = codes.float()
    assert scales.shape == (4, 3)
    assert not c[0].any() and torch.equal(scales[0], torch.full((3,), 2.0 ** -100, device=dev()))
    assert torch.equal(scales[3, 1:], torch.full((2,), 2.0 ** -100, device=dev())) and c[3, 5] == 448
    assert torch.equal(c[2], torch.full((300,), 448.0, device=dev()))
    # numbers so small that a group's scale is held: they round to codes of that scale
    t = torch.full((1, 256), 1e-28, device=dev())
    codes, scales, _, _ = mm.muon_rmsnorm_forward_fp8(t, None, eps=1.0)
    assert torch.equal(scales, torch.full((1, 2), 2.0 ** -100, device=dev()))
    want = torch.from_numpy(ref.e4m3(num(t) * 2.0 ** 100)).to(dev()).float()
    assert torch.equal(codes.float(), want) and want.any()
    # a NaN or infinity stays in its row
    x = torch.randn(5, 300, device=dev())
    x[1, 3], x[3, 200] = float("nan"), float("inf")
    y, _, _ = mm.muon_rmsnorm_forward(x, w)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3, 200]) and torch.isfinite(y[[0, 2, 4]]).all()
    codes, scales, _, _ = mm.muon_rmsnorm_forward_fp8(x, w)
    c = codes.float()
    assert torch.isnan(c[1]).all() and torch.isnan(scales[1]).all() and torch.isnan(scales[3, 1]) and torch.isnan(c[3, 200])
    assert torch.isfinite(c[[0, 2, 4]]).all() and not c[3, :128].any() and torch.isnan(c[3, 128:256]).all()


def test_rmsnorm_streams_graphs_and_second_derivatives():
    x, r, dy = (torch.randn(70, 520, device=dev(), dtype=torch.bfloat16) for _ in range(3))
    w = torch.randn(520, device=dev())
    ws = mm.alloc_rmsnorm_workspace(70, 520)

    def both(stream=None):
        y, rstd, total = mm.muon_rmsnorm_forward(x, w, r, stream=stream)
        return (y, rstd, total, *mm.muon_rmsnorm_forward_fp8(x, w, r, stream=stream)[:2],
                *mm.muon_rmsnorm_backward(dy, total, w, rstd, ws, dtotal=dy, stream=stream))

    def same(a, b):
        return all(torch.equal(p.float(), q.float()) for p, q in zip(a, b))

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(s)
    s.synchronize()
    assert same(got, want)
    handle = both(s.cuda_stream)
    s.synchronize()
    assert same(handle, want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    x.mul_(2)
    dy.add_(1)
    g.replay()
    torch.cuda.synchronize()
    assert same(out, both())
    a, b = x.float().requires_grad_(), w.clone().requires_grad_()
    y, t = mm.rms_norm(a, b, r.float())
    (da,) = torch.autograd.grad((y * y).sum() + t.sum(), a, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        da.sum().backward()


@pytest.mark.parametrize("shape", [(3, 4, 96), (5, 96), (96,)])
def test_rms_norm_function(shape):
    """Under autograd: against torch's own derivatives in 64 bits, each output used or not."""
    torch.manual_seed(1)
    x, r = (torch.randn(*shape, device=dev()).requires_grad_() for _ in range(2))
    w = torch.randn(96, device=dev()).requires_grad_()
    cy, ct = torch.randn(*shape, device=dev()), torch.randn(*shape, device=dev())

    def plain(x, w, t):
        y = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)
        return y * w

    for use_y, use_t in ((1, 1), (1, 0), (0, 1)):
        y, t = mm.rms_norm(x, w, r)
        got = torch.autograd.grad((y * cy).sum() * use_y + (t * ct).sum() * use_t if use_y and use_t else
                                  (y * cy).sum() if use_y else (t * ct).sum(), (x, r, w), allow_unused=True)
        x6, r6, w6 = (v.detach().double().requires_grad_() for v in (x, r, w))
        t6 = x6 + r6
        want = torch.autograd.grad((plain(x6, w6, t6) * cy).sum() * use_y + (t6 * ct).sum() * use_t, (x6, r6, w6))
        for p, q in zip(got, want):
            assert (p is None and not q.any()) or torch.allclose(p.double(), q, rtol=1e-4, atol=1e-4)
    y = mm.rms_norm(x, w)
    (dx,) = torch.autograd.grad(y, x, cy.expand_as(y))
    x6 = x.detach().double().requires_grad_()
    (want,) = torch.autograd.grad((plain(x6, w.double(), x6) * cy).sum(), x6)
    assert torch.allclose(dx.double(), want, rtol=1e-4, atol=1e-4)
    # a broadcast gradient, and transposed rows
    (dx,) = torch.autograd.grad(mm.rms_norm(x, w).sum(), x)
    (want,) = torch.autograd.grad(plain(x6, w.double(), x6).sum(), x6)
    assert torch.allclose(dx.double(), want, rtol=1e-4, atol=1e-4)


def test_rmsnorm_past_32_bit_offsets():
    """Rows 2^25 elements apart, and past 2^31 elements."""
    n, d, apart = 70, 96, 1 << 25
    big = torch.zeros(n * apart, dtype=torch.bfloat16, device=dev())
    rows = big.view(n, apart)[:, :d]
    x, x64 = put(np.random.default_rng(2).standard_normal((n, d)), "bf16")
    rows.copy_(x)
    w = torch.ones(d, device=dev())
    a, b = mm.muon_rmsnorm_forward(rows, w, rows), mm.muon_rmsnorm_forward(x, w, x)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ws = mm.alloc_rmsnorm_workspace(n, d)
    p, q = (mm.muon_rmsnorm_backward(v, v, w, a[1], ws, dtotal=v) for v in (rows, x))
    assert all(torch.equal(u, v) for u, v in zip(p, q))
    c, e = mm.muon_rmsnorm_forward_fp8(rows, w), mm.muon_rmsnorm_forward_fp8(x, w)
    assert torch.equal(c[0].float(), e[0].float()) and torch.equal(c[1], e[1])
