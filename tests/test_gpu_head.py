"""The head's operators on the GPU against the fp64 oracle.

Tolerances come from the arithmetic, not from runs.  u = 2^-24 is fp32's rounding error,
2^-8 bf16's half-spacing.  A sum of n fp32 terms in any order is within n*u of the sum of
their magnitudes; every kernel here keeps at least 32 running sums a row, so n is D/32 + 32
for a row of D.  The tensor cores' fp32 accumulation is allowed twice fp32's rounding error
(2u, truncation) for each product of 16 terms."""
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
    """(tensor of that dtype on the GPU, the values it holds in fp64)"""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype])
    return t.to(dev()), t.double().numpy()


def num(t):
    return t.double().cpu().numpy()


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300))))


def strided(t, pad):
    """The same values as rows of a wider buffer."""
    if not pad:
        return t
    b = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


# ------------------------------------------------------------------ layer norm
NORM_SIZES = [(1, 1), (3, 1), (1, 2), (5, 3), (1, 7), (7, 31), (2, 32), (9, 33), (4, 64), (33, 127), (5, 255), (3, 256),
              (6, 257), (160, 512), (2, 1000), (311, 1024), (3, 1025), (17, 1536), (2, 2047), (5, 2560), (3, 4096),
              (2, 4099), (4, 5120), (3, 8192), (2, 8200), (2, 12288), (3, 16384), (1, 16391), (2, 40000), (1, 65536)]


@pytest.mark.parametrize("pad", [0, 8, 5])
@pytest.mark.parametrize("wdt", ["bf16", "f32", None])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_layernorm(xdt, wdt, pad):
    rng = np.random.default_rng(7)
    for n, d in NORM_SIZES:
        x, x64 = put(rng.standard_normal((n, d)) * 2 + 0.5, xdt)
        dy, dy64 = put(rng.standard_normal((n, d)), xdt)
        w, w64 = put(1 + 0.3 * rng.standard_normal(d), wdt) if wdt else (None, None)
        b, b64 = put(0.3 * rng.standard_normal(d), wdt) if wdt else (None, None)
        y, mean, rstd = mm.muon_layernorm_forward(strided(x, pad), w, b, eps=1e-5)
        ry, rmean, rrstd = ref.layernorm_forward(x64, w64, b64, 1e-5)
        gam = (d / 32 + 32) * U
        one = BF if xdt == "bf16" else 0.0
        aw = np.abs(w64) if wdt else 1.0
        emean = gam * np.abs(x64).mean(1) + U * np.abs(rmean)
        within(num(mean), rmean, emean, ("mean", n, d))
        # rstd = v^-1/2: relative error half of v's; v sums squares of x - mean, each off by emean
        cen = np.abs(x64 - rmean[:, None])
        ev = (2 * (emean[:, None] + U * cen) * cen).mean(1) + emean ** 2 + gam * (cen ** 2).mean(1)
        er = rrstd * (0.5 * ev * rrstd ** 2 + 8 * U)
        within(num(rstd), rrstd, er, ("rstd", n, d))
        exh = (emean[:, None] + U * cen) * rrstd[:, None] + cen * er[:, None]
        ey = exh * aw + 4 * U * (np.abs(ry) + cen * rrstd[:, None] * aw) + one * np.abs(ry)
        within(num(y), ry, ey * 1.01 + 1e-30, ("y", n, d))

        # backward, from the kernel's own statistics
        ws = mm.alloc_layernorm_workspace(n, d)
        dx, dw, db = mm.muon_layernorm_backward(strided(dy, pad), strided(x, pad), w, mean, rstd, ws)
        m64, r64 = num(mean), num(rstd)
        rdx, rdw, rdb = ref.layernorm_backward(dy64, x64, w64, m64, r64)
        xh = (x64 - m64[:, None]) * r64[:, None]
        g = dy64 * (w64 if wdt else 1.0)
        eg, exh = 2 * U * np.abs(g), 3 * U * np.abs(xh)
        c1, c2 = np.abs(g).mean(1, keepdims=True), np.abs(g * xh).mean(1, keepdims=True)
        edx = r64[:, None] * (eg + (gam + 4 * U) * c1 + np.abs(xh) * (gam + 8 * U) * c2 + exh * c2 +
                              4 * U * (np.abs(g) + c1 + np.abs(xh) * c2)) + one * np.abs(rdx)
        within(num(dx), rdx, edx * 1.01 + 1e-30, ("dx", n, d))
        wone = BF if (wdt or xdt) == "bf16" else 0.0
        if wdt:
            within(num(dw), rdw, (n + 8) * U * np.abs(dy64 * xh).sum(0) + wone * np.abs(rdw) + 1e-30, ("dw", n, d))
        else:
            assert dw is None
        within(num(db), rdb, (n + 8) * U * np.abs(dy64).sum(0) + wone * np.abs(rdb) + 1e-30, ("db", n, d))


def test_layernorm_many_rows_and_repeatability():
    """More rows than CTAs fit at once; the same inputs give the same bits."""
    rng = np.random.default_rng(8)
    n, d = 20011, 192
    x, x64 = put(rng.standard_normal((n, d)), "bf16")
    dy, dy64 = put(rng.standard_normal((n, d)), "bf16")
    w, w64 = put(1 + 0.3 * rng.standard_normal(d), "f32")
    y, mean, rstd = mm.muon_layernorm_forward(x, w, w)
    ws = mm.alloc_layernorm_workspace(n, d)
    a = mm.muon_layernorm_backward(dy, x, w, mean, rstd, ws)
    ws.fill_(255)
    b = mm.muon_layernorm_backward(dy, x, w, mean, rstd, ws)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    _, rdw, rdb = ref.layernorm_backward(dy64, x64, w64, num(mean), num(rstd))
    xh = (x64 - num(mean)[:, None]) * num(rstd)[:, None]
    within(num(a[1]), rdw, (n + 8) * U * np.abs(dy64 * xh).sum(0), "dw")
    within(num(a[2]), rdb, (n + 8) * U * np.abs(dy64).sum(0), "db")


def test_layernorm_constant_rows_empty_batches_and_nonfinite():
    w = torch.full((40,), 2.0, device=dev())
    y, mean, rstd = mm.muon_layernorm_forward(torch.full((3, 40), 5.0, device=dev()), w, w, eps=1e-5)
    assert torch.equal(y, torch.full_like(y, 2.0)) and torch.equal(mean, torch.full_like(mean, 5.0))
    # no rows: no outputs to write, and the gradients' sums are zero
    x = torch.empty(0, 40, device=dev())
    y, mean, rstd = mm.muon_layernorm_forward(x, w)
    assert y.shape == (0, 40)
    dx, dw, db = mm.muon_layernorm_backward(x, x, w, mean, rstd, mm.alloc_layernorm_workspace(0, 40))
    assert dx.shape == (0, 40) and not dw.any() and not db.any()
    # a NaN stays in its row (and reaches the column sums)
    x = torch.randn(5, 40, device=dev())
    x[2, 3] = float("nan")
    y, mean, rstd = mm.muon_layernorm_forward(x, w)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3, 4]]).all()


def test_layernorm_without_weight_gradients_needs_no_workspace():
    x = torch.randn(6, 300, device=dev())
    _, mean, rstd = mm.muon_layernorm_forward(x)
    dx, dw, db = mm.muon_layernorm_backward(x, x, None, mean, rstd, None, bias=False)
    assert dw is None and db is None and torch.isfinite(dx).all()
    with pytest.raises(mm.MuonError):
        mm.muon_layernorm_backward(x, x, None, mean, rstd, None, bias=True)
    small = mm.alloc_layernorm_workspace(6, 300)[:256]
    with pytest.raises(mm.MuonError):
        mm.muon_layernorm_backward(x, x, None, mean, rstd, small, bias=True)


def test_layernorm_unaligned_views():
    """Rows and vectors that start off every vector boundary."""
    rng = np.random.default_rng(9)
    for xdt in ("bf16", "f32"):
        for off in (1, 2, 3, 5):
            n, d = 6, 1536
            flat, _ = put(rng.standard_normal(off + n * d), xdt)
            wf, _ = put(rng.standard_normal(off + d), "f32")
            x, w = flat[off:].view(n, d), wf[off:]
            y, mean, rstd = mm.muon_layernorm_forward(x, w, w)
            yc, mc, rc = mm.muon_layernorm_forward(x.clone(), w.clone(), w.clone())
            assert np.max(np.abs(num(y) - num(yc))) <= 2 * BF * np.max(np.abs(num(yc)))
            ws = mm.alloc_layernorm_workspace(n, d)
            a = mm.muon_layernorm_backward(x, x, w, mean, rstd, ws)
            b = mm.muon_layernorm_backward(x.clone(), x.clone(), w.clone(), mean, rstd, ws)
            for p, q in zip(a, b):
                assert np.max(np.abs(num(p) - num(q))) <= (2 * BF if xdt == "bf16" else 1e-4) * np.max(np.abs(num(q)))


# ------------------------------------------------------------------ linear cross entropy
def ce_case(n, v, d, dt, seed, sharp=1.0):
    rng = np.random.default_rng(seed)
    w, w64 = put(rng.standard_normal((v, d)) * 2 / np.sqrt(d), dt)
    labels = rng.integers(0, v, n)
    h, h64 = put(rng.standard_normal((n, d)) * sharp + w64[labels], dt)
    labels[rng.random(n) < 0.2] = -100
    return h, h64, w, w64, torch.from_numpy(labels).to(dev()), labels


def ce_tolerances(h64, w64, dt):
    """(error of a logit, by row: the largest over the vocabulary)"""
    d = h64.shape[1]
    steps = d / 16 + 16
    # 32-bit operands are cut into three bf16 parts each; what is dropped is below 2^-23 of a product
    parts = 1 if dt == "bf16" else 4
    return (parts * steps * 2 * U) * (np.abs(h64) @ np.abs(w64).T).max(1)


CE_SIZES = [(1, 1, 1), (1, 5, 8), (3, 2, 16), (2, 7, 3), (5, 100, 65), (8, 1000, 64), (16, 257, 72), (129, 255, 128),
            (128, 256, 64), (127, 300, 200), (257, 513, 96), (300, 1111, 321), (1, 5000, 256), (1000, 40, 40),
            (64, 9000, 130)]


@pytest.mark.parametrize("size", CE_SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_ce(dt, size):
    n, v, d = size
    h, h64, w, w64, labels, lab = ce_case(n, v, d, dt, n + v + d)
    ws = mm.alloc_linear_ce_workspace(n, v, d, TYPES[dt])
    loss, lse, stats = mm.muon_linear_ce_forward(h, w, labels, ws)
    assert mm.muon_check_status(ws) == mm.MUON_OK
    rloss, rlse, rmean, count = ref.linear_ce_forward(h64, w64, lab)
    ez = ce_tolerances(h64, w64, dt)
    # exponentials within 4 ulp and the argument's rounding, their sum within (v/32 + 32) u
    spread = np.abs(h64 @ w64.T).max(1) + 1
    elog = ez + (v / 32 + 64 + 4 * spread) * U + 4 * U * np.abs(rlse)
    within(num(lse), rlse, elog, "lse")
    within(num(loss), rloss, elog + ez + 2 * U * np.abs(rlse), "loss")
    assert np.all(num(loss)[lab == -100] == 0)
    eloss = (elog + ez)[lab != -100].sum() + 64 * U * np.abs(rloss).sum()
    assert stats[1].item() == count
    within(num(stats[0]), rmean, eloss / max(count, 1) + 1e-30, "mean")

    lse64 = num(lse)
    for how in ("mean", "rows"):
        rng = np.random.default_rng(3)
        rg, rg64 = put(rng.random(n), "f32")
        if how == "mean":
            dh, dw = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats, grad_scale=3.0)
            coef = np.full(n, 3.0 / max(count, 1))
        else:
            dh, dw = mm.muon_linear_ce_backward(h, w, labels, lse, ws, row_grad=rg)
            coef = rg64
        assert mm.muon_check_status(ws) == mm.MUON_OK
        g = ref.linear_ce_logit_grad(h64, w64, lab, lse64, coef)
        z = h64 @ w64.T
        counted = (lab != -100) * coef
        eg = counted[:, None] * np.exp(z - lse64[:, None]) * (ez + (16 + 4 * spread) * U)[:, None] + 8 * U * np.abs(g) + \
            4 * U * counted[:, None]
        parts = 1 if dt == "bf16" else 4
        if dt == "bf16":
            eg = eg + BF * (np.abs(g) + eg)
        one = BF if dt == "bf16" else 0.0
        edh = eg @ np.abs(w64) + parts * (v / 16 + 64) * 2 * U * (np.abs(g) @ np.abs(w64))
        edw = eg.T @ np.abs(h64) + parts * (n / 16 + 64) * 2 * U * (np.abs(g).T @ np.abs(h64))
        within(num(dh), g @ w64, edh + one * (np.abs(g @ w64) + edh) + 1e-30, "dh " + how)
        within(num(dw), g.T @ h64, edw + one * (np.abs(g.T @ h64) + edw) + 1e-30, "dw " + how)
        assert not dh[labels == -100].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_ce_gradient_matches_differences(dt):
    """The loss moves along a direction as the gradient says (central differences of the
    oracle's loss around the kernel's gradient)."""
    n, v, d = 40, 333, 48
    h, h64, w, w64, labels, lab = ce_case(n, v, d, dt, 5)
    ws = mm.alloc_linear_ce_workspace(n, v, d, TYPES[dt])
    _, lse, stats = mm.muon_linear_ce_forward(h, w, labels, ws)
    dh, dw = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats)
    rng = np.random.default_rng(1)
    for arg, grad, which in ((h64, num(dh), 0), (w64, num(dw), 1)):
        e = rng.standard_normal(arg.shape)
        step = 1e-4
        f = [ref.linear_ce_forward(*((arg + s * step * e, w64) if which == 0 else (h64, arg + s * step * e)), lab)[2] for s in (1, -1)]
        slope = (f[0] - f[1]) / (2 * step)
        # each entry is off by at most the rounding of g and of the result (two of 2^-8 in bf16)
        tol = (3 * BF if dt == "bf16" else 1e-5) * np.linalg.norm(grad) * np.linalg.norm(e) / np.sqrt(e.size) * 6 + 1e-6
        assert abs(slope - (grad * e).sum()) < tol


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_ce_strides_and_alignment(dt):
    """Rows cut out of wider buffers, odd offsets: the same numbers as packed inputs."""
    for n, v, d, pad, off in ((33, 200, 64, 8, 0), (33, 200, 64, 5, 0), (20, 77, 50, 3, 1), (9, 130, 128, 0, 1)):
        h, h64, w, w64, labels, lab = ce_case(n, v, d, dt, n)
        hb = torch.full((off + n * (d + pad) + 8,), float("nan"), dtype=h.dtype, device=h.device)
        wb = torch.full((off + v * (d + pad) + 8,), float("nan"), dtype=h.dtype, device=h.device)
        hv = hb[off:off + n * (d + pad)].view(n, d + pad)[:, :d]
        wv = wb[off:off + v * (d + pad)].view(v, d + pad)[:, :d]
        hv.copy_(h)
        wv.copy_(w)
        ws = mm.linear_ce_workspace_for(hv, wv, labels)
        packed = mm.alloc_linear_ce_workspace(n, v, d, TYPES[dt])
        a, b = mm.muon_linear_ce_forward(hv, wv, labels, ws), mm.muon_linear_ce_forward(h, w, labels, packed)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        a = mm.muon_linear_ce_backward(hv, wv, labels, b[1], ws, stats=b[2])
        b = mm.muon_linear_ce_backward(h, w, labels, b[1], packed, stats=b[2])
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_linear_ce_labels():
    """All ignored; out of range; an ignore_index inside the vocabulary; the last column."""
    n, v, d = 20, 300, 64
    h, h64, w, w64, labels, lab = ce_case(n, v, d, "bf16", 11)
    ws = mm.alloc_linear_ce_workspace(n, v, d)
    none = torch.full_like(labels, -100)
    loss, lse, stats = mm.muon_linear_ce_forward(h, w, none, ws)
    assert not loss.any() and stats.tolist() == [0.0, 0.0] and torch.isfinite(lse).all()
    nan = torch.full((n,), float("nan"), device=dev())
    dh, dw = mm.muon_linear_ce_backward(h, w, none, lse, ws, row_grad=nan, stats=stats)
    assert not dh.any() and not dw.any()
    odd = labels.clone()
    odd[3], odd[4], odd[5] = v, -1, v - 1
    loss, lse, stats = mm.muon_linear_ce_forward(h, w, odd, ws)
    assert torch.isnan(loss[3]) and torch.isnan(loss[4]) and torch.isfinite(loss[5]) and torch.isnan(stats[0])
    dh, dw = mm.muon_linear_ce_backward(h, w, odd, lse, ws, row_grad=torch.ones(n, device=dev()))
    assert not dh[3].any() and not dh[4].any() and dh[5].any() and torch.isfinite(dw).all()
    zero = torch.where(labels == -100, 0, labels)
    loss, lse, stats = mm.muon_linear_ce_forward(h, w, zero, ws, ignore_index=0)
    assert not loss[zero == 0].any() and stats[1].item() == (zero != 0).sum().item()


@pytest.mark.parametrize("dt,d,pad", [("bf16", 64, 0), ("bf16", 72, 24), ("bf16", 61, 0), ("bf16", 64, 3), ("f32", 64, 0),
                                      ("f32", 61, 2)])
def test_linear_ce_rows_without_gradient_may_hold_anything(dt, d, pad):
    """NaN and infinities in rows whose label is ignored or out of range change nothing: the
    gradients are bit for bit those with zeros there."""
    n, v = 140, 300
    h, h64, w, w64, labels, lab = ce_case(n, v, d, dt, 12)
    labels = labels.clone()
    labels[::3], labels[7] = -100, v + 5
    dead = (labels < 0) | (labels >= v)
    big = torch.zeros(n, d + pad, dtype=h.dtype, device=dev())
    clean = torch.where(dead[:, None], 0.0, h.float()).to(h.dtype)
    junk = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38], device=dev()).repeat(n * d // 4 + 1)[:n * d]
    big[:, :d] = torch.where(dead[:, None], junk.view(n, d), h.float()).to(h.dtype)
    big = big[:, :d]
    ws = mm.linear_ce_workspace_for(big, w, labels)
    loss, lse, _ = mm.muon_linear_ce_forward(big, w, labels, ws)
    want, lsew, _ = mm.muon_linear_ce_forward(clean, w, labels, ws)
    ok = ~dead
    assert torch.equal(loss[ok], want[ok]) and torch.equal(lse[ok], lsew[ok]) and not loss[labels == -100].any()
    got = mm.muon_linear_ce_backward(big, w, labels, lse, ws)
    ref_ = mm.muon_linear_ce_backward(clean, w, labels, lsew, ws)
    assert all(torch.equal(p, q) and bool(torch.isfinite(p).all()) for p, q in zip(got, ref_))
    assert not got[0][dead].any() and bool(got[1].any())


def test_linear_ce_extremes():
    """Logits far apart, all equal, and not finite."""
    v, d = 500, 32
    w = torch.zeros(v, d, device=dev())
    w[:, 0] = torch.linspace(-300, 300, v, device=dev())
    h = torch.zeros(5, d, device=dev())
    h[0, 0], h[1, 0], h[3, 0], h[4, 0] = 10.0, -10.0, float("inf"), float("nan")
    labels = torch.tensor([0, 0, 7, 1, 1], device=dev())
    ws = mm.alloc_linear_ce_workspace(5, v, d, torch.float32)
    loss, lse, stats = mm.muon_linear_ce_forward(h, w, labels, ws)
    want = ref.linear_ce_forward(num(h[:3]), num(w), labels[:3].cpu().numpy())
    assert np.allclose(num(loss[:3]), want[0], rtol=1e-5, atol=1e-3)      # 3000 in fp32 has spacing 2.4e-4
    assert abs(loss[2].item() - np.log(v)) < 1e-5
    assert torch.isnan(loss[3]) and torch.isnan(loss[4])
    dh, dw = mm.muon_linear_ce_backward(h[:3], w, labels[:3], lse[:3].contiguous(), ws, row_grad=torch.ones(3, device=dev()))
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()
    # no rows
    e = torch.empty(0, d, device=dev())
    none = torch.empty(0, dtype=torch.int64, device=dev())
    loss, lse, stats = mm.muon_linear_ce_forward(e, w, none, ws)
    assert stats.tolist() == [0.0, 0.0]
    dh, dw = mm.muon_linear_ce_backward(e, w, none, lse, ws, stats=stats)
    assert dh.shape == (0, d) and not dw.any() and dw.shape == w.shape


def test_linear_ce_large_repeats_and_other_stream():
    """Several pieces of the vocabulary; the same bits twice and on another stream; one
    gradient at a time gives what both do."""
    n, v, d = 700, 20001, 256
    h, h64, w, w64, labels, lab = ce_case(n, v, d, "bf16", 21)
    ws = mm.alloc_linear_ce_workspace(n, v, d)
    loss, lse, stats = mm.muon_linear_ce_forward(h, w, labels, ws)
    rloss, rlse, rmean, count = ref.linear_ce_forward(h64, w64, lab)
    assert np.max(np.abs(num(lse) - rlse)) < 1e-4 and abs(stats[0].item() - rmean) < 1e-4
    a = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats)
    rdh, rdw = ref.linear_ce_backward(h64, w64, lab, num(lse), np.full(n, 1.0 / count))
    for p, q in zip(a, (rdh, rdw)):
        assert np.linalg.norm(num(p) - q) < 2 * BF * np.linalg.norm(q)
    ws.view(torch.uint8)[256:].fill_(255)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = mm.muon_linear_ce_forward(h, w, labels, ws, stream=s)
    c = mm.muon_linear_ce_backward(h, w, labels, b[1], ws, stats=b[2], stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((loss, lse, stats), b)) and all(torch.equal(p, q) for p, q in zip(a, c))
    dh, none = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats, need_dw=False)
    assert none is None and torch.equal(dh, a[0])
    none, dw = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats, need_dh=False)
    assert none is None and torch.equal(dw, a[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_ce_upstream_factor(dt):
    """A factor on the device multiplies both gradients once, whichever way dH is summed
    (few rows: ranges of K; more: none), and the rounding of g does not depend on it."""
    for n, v, d in ((24, 3000, 64), (600, 700, 96)):
        h, h64, w, w64, labels, lab = ce_case(n, v, d, dt, 77)
        ws = mm.alloc_linear_ce_workspace(n, v, d, TYPES[dt])
        _, lse, stats = mm.muon_linear_ce_forward(h, w, labels, ws)
        one = mm.muon_linear_ce_backward(h, w, labels, lse, ws)
        up = torch.tensor(0.125, device=dev())
        a = mm.muon_linear_ce_backward(h, w, labels, lse, ws, upstream=up, grad_scale=4.0)
        assert all(torch.equal(p * 0.5, q) for p, q in zip(one, a))
        count = stats[1].item()
        b = mm.muon_linear_ce_backward(h, w, labels, lse, ws, stats=stats)
        for p, q in zip(one, b):
            tol = (2 * BF if dt == "bf16" else 4 * U) * np.abs(num(p)) / count
            within(num(q), num(p) / count, tol, "mean")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_ce_back_to_back(dt):
    """Hundreds of calls queued without a wait between them, with tiles that fill only part of
    a CTA pair: no wait in a kernel expires, every call gives the first one's bits."""
    mm.muon_debug_set(0, 200)
    try:
        for n, v, d in ((300, 10007, 130), (70, 1300, 300), (8, 9000, 257)):
            h, h64, w, w64, labels, lab = ce_case(n, v, d, dt, 5)
            ws = mm.alloc_linear_ce_workspace(n, v, d, TYPES[dt])
            first = mm.muon_linear_ce_forward(h, w, labels, ws)
            first += mm.muon_linear_ce_backward(h, w, labels, first[1], ws, stats=first[2])
            for _ in range(150):
                out = mm.muon_linear_ce_forward(h, w, labels, ws)
                out += mm.muon_linear_ce_backward(h, w, labels, out[1], ws, stats=out[2])
            assert mm.muon_check_status(ws) == mm.MUON_OK
            assert all(torch.equal(p, q) for p, q in zip(first, out))
    finally:
        mm.muon_debug_set(0, 0)


def test_linear_ce_expired_wait_is_reported():
    """A producer that issues no loads (test flag): the waits run out, the call returns, the
    status says so, and the next call is right again."""
    n, v, d = 40, 600, 64
    h, h64, w, w64, labels, lab = ce_case(n, v, d, "bf16", 6)
    ws = mm.alloc_linear_ce_workspace(n, v, d)
    want = mm.muon_linear_ce_forward(h, w, labels, ws)
    mm.muon_debug_set(mm.MUON_DEBUG_STALL_PRODUCER, 50)
    try:
        mm.muon_linear_ce_forward(h, w, labels, ws)
        assert mm.muon_check_status(ws) == mm.MUON_ERR_TIMEOUT
    finally:
        mm.muon_debug_set(0, 0)
    got = mm.muon_linear_ce_forward(h, w, labels, ws)
    assert mm.muon_check_status(ws) == mm.MUON_OK
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_linear_ce_in_a_cuda_graph():
    n, v, d = 130, 1000, 64
    h, h64, w, w64, labels, lab = ce_case(n, v, d, "bf16", 31)
    ws = mm.alloc_linear_ce_workspace(n, v, d)
    want = mm.muon_linear_ce_forward(h, w, labels, ws)
    wantg = mm.muon_linear_ce_backward(h, w, labels, want[1], ws, stats=want[2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mm.muon_linear_ce_forward(h, w, labels, ws)
        grads = mm.muon_linear_ce_backward(h, w, labels, out[1], ws, stats=out[2])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out + grads, want + wantg))


# ------------------------------------------------------------------ AdamW, 8-bit moments
def padded(a):
    return np.concatenate([a, np.zeros(-len(a) % 128)])


def compare_codes(got_codes, got_scale, exact, bits, top, binades, err, what):
    """Codes equal the oracle's, but where the fp32 value's error can cross a rounding edge
    (then they are neighbours).  err: relative error of the fp32 moment."""
    code, scale, value, slack = ref.quantise(exact, bits, top, binades)
    got = np.asarray(got_codes, np.int64)
    mag = got & 127 if top == 127 else got
    assert np.array_equal(np.asarray(got_scale, np.int64), scale.astype(np.int64)), what
    off = mag - code
    # eight places a binade: a relative error e moves a place by at most 8*log2(e)*e < 12 e
    assert np.all(np.abs(off) <= 1) and np.all((off == 0) | (slack <= 16 * err)), what
    if top == 127:
        assert np.all((got < 128) | (exact < 0)), what
        assert np.all(got != 128), what


@pytest.mark.parametrize("gdt", ["bf16", "f32"])
@pytest.mark.parametrize("pdt", ["bf16", "f32"])
def test_adamw8_against_the_oracle(pdt, gdt):
    sizes = [1, 7, 16, 127, 128, 129, 1536, 4095, 4096, 4097, 100003]
    rng = np.random.default_rng(30)
    P0 = [put(rng.standard_normal(k) * 0.02, pdt) for k in sizes]
    P = [p for p, _ in P0]
    opt = mm.AdamW8(P, lr=1e-3, betas=(0.9, 0.99), weight_decay=0.05, seed=77)
    ref_p = [q for _, q in P0]
    for t in range(1, 5):
        before = opt.state_dict()
        # magnitudes across blocks and inside them, exact zeros among them
        G = [put(rng.standard_normal(k) * 10.0 ** rng.uniform(-6, -1) * 10.0 ** rng.uniform(-3, 0, k) * (rng.random(k) > 0.1), gdt)
             for k in sizes]
        opt.step([g for g, _ in G])
        torch.cuda.synchronize()
        for i, k in enumerate(sizes):
            a, n = opt.starts[i], opt.starts[i + 1] - opt.starts[i]
            codes = {q: before[q][a:a + n].cpu().numpy() for q in "mv"}
            scales = {q: before[q + "_scale"][a // 128:(a + n) // 128].cpu().numpy() for q in "mv"}
            m0, v0 = ref.decode(codes["m"], scales["m"], True)[:k], ref.decode(codes["v"], scales["v"], False)[:k]
            p, m, v = ref.adamw8_update(ref_p[i], G[i][1], m0, v0, t, 1e-3, 0.9, 0.99, 1e-8, 0.05)
            got = num(P[i])
            # m sums two terms that may cancel: its error is relative to their magnitudes
            terms = np.abs(ref_p[i]) + 1e-3 * ((0.9 * np.abs(m0) + 0.1 * np.abs(G[i][1])) / (1 - 0.9 ** t) /
                                               (np.sqrt(v / (1 - 0.99 ** t)) + 1e-8))
            within(got, p, 16 * U * terms + (BF * (np.abs(p) + 1e-30) * 1.01 if pdt == "bf16" else 0) + 1e-37, ("p", k, t))
            bits = ref.random_bits(77, t, a + np.arange(n)).astype(np.int64)
            cancel = padded((0.9 * np.abs(m0) + 0.1 * np.abs(G[i][1])) / np.maximum(np.abs(m), 1e-300))
            sl = slice(a, a + n), slice(a // 128, (a + n) // 128)
            compare_codes(opt.m[sl[0]].cpu().numpy(), opt.m_scale[sl[1]].cpu().numpy(), padded(m), bits & 0xFFFF, 127, 16,
                          4 * U * np.maximum(cancel, 1), ("m", k, t))
            compare_codes(opt.v[sl[0]].cpu().numpy(), opt.v_scale[sl[1]].cpu().numpy(), padded(v), bits >> 16, 255, 32,
                          8 * U, ("v", k, t))
            ref_p[i] = got
    m, v = opt.moments()
    assert np.array_equal(num(m), ref.decode(opt.m.cpu().numpy(), opt.m_scale.cpu().numpy(), True))
    assert np.array_equal(num(v), ref.decode(opt.v.cpu().numpy(), opt.v_scale.cpu().numpy(), False))


def test_adamw8_many_tensors_resume_and_repeat():
    """More parameters than one launch takes; a checkpoint continues bit for bit; another
    seed rounds otherwise; parameters and gradients off every vector boundary."""
    rng = np.random.default_rng(4)
    sizes = [int(k) for k in rng.integers(0, 700, 300)] + [0, 5000]
    flat, _ = put(rng.standard_normal(sum(sizes) + 3) * 0.02, "bf16")
    gflat = [put(rng.standard_normal(sum(sizes) + 5) * 1e-3, "bf16")[0] for _ in range(4)]

    def cut(f, off):
        out, at = [], off
        for k in sizes:
            out.append(f[at:at + k])
            at += k
        return out

    def run(seed, resume_at=None):
        P = cut(flat.clone(), 3)
        opt = mm.AdamW8(P, lr=1e-2, seed=seed)
        for t in range(4):
            if t == resume_at:
                sd = opt.state_dict()
                opt = mm.AdamW8(P, lr=1e-2, seed=1234)
                opt.load_state_dict(sd)
            opt.step(cut(gflat[t], 5))
        return P, opt

    (pa, a), (pb, b), (pc, c) = run(9), run(9, resume_at=2), run(10)
    assert all(torch.equal(x, y) for x, y in zip(pa, pb))
    for q in ("m", "v", "m_scale", "v_scale"):
        assert torch.equal(getattr(a, q), getattr(b, q))
    assert not torch.equal(a.m, c.m)
    # aligned copies of the same tensors give the same bits
    P = [p.clone() for p in cut(flat, 3)]
    opt = mm.AdamW8(P, lr=1e-2, seed=9)
    for t in range(4):
        opt.step([g.clone() for g in cut(gflat[t], 5)])
    assert all(torch.equal(x, y) for x, y in zip(pa, P)) and torch.equal(a.m, opt.m) and torch.equal(a.v, opt.v)


def test_adamw8_parameters_cast_or_moved_after_construction():
    """A parameter whose data was replaced is taken as it is now, or refused, with the state
    and the parameters unchanged."""
    p, q = torch.zeros(300, device=dev()), torch.zeros(40, device=dev())
    g = [torch.full((300,), 1e-3, device=dev()), torch.full((40,), 1e-3, device=dev())]
    opt = mm.AdamW8([p, q], lr=1e-3)
    opt.step(g)
    guard = torch.full((900,), 7.0, dtype=torch.bfloat16, device=dev())
    p.data = guard[300:600]                      # narrower than what the optimizer was made with
    with pytest.raises(ValueError):              # two dtypes
        opt.step(g)
    q.data = q.data.bfloat16()
    opt.step(g)
    assert opt.step_count == 2
    # a step of 1e-3 is below half of bf16's spacing at 7, so p's values show nothing; q's do
    assert bool((guard == 7).all()) and bool((q < -1.5e-3).all()) and bool((q > -2.5e-3).all())
    for bad in (p.data[:299], p.data.cpu(), torch.zeros(600, dtype=torch.bfloat16, device=dev())[::2]):
        p.data = bad
        with pytest.raises(ValueError):
            opt.step(g)
    p.data = guard[300:600]
    for bad in ([g[0]], [g[0], g[1][:39]], [g[0].cpu(), g[1]], [g[0], g[1].bfloat16()]):
        with pytest.raises(ValueError):
            opt.step(bad)
    assert opt.step_count == 2


def test_adamw8_nonfinite_and_extreme_gradients():
    k = 300
    p = torch.zeros(k, device=dev())
    opt = mm.AdamW8([p], lr=1e-3)
    g = torch.full((k,), 1e-3, device=dev())
    g[5], g[6], g[7], g[8], g[200] = float("nan"), float("inf"), 1e30, 0.0, 1e-25
    clean = torch.zeros(k, device=dev())
    ref_opt = mm.AdamW8([clean], lr=1e-3)
    ok = torch.full((k,), 1e-3, device=dev())
    ref_opt.step([ok])
    opt.step([g])
    m, v = opt.moments()
    assert torch.isnan(p[5:7]).all() and torch.isnan(m[5:7]).all() and torch.isfinite(v).all()
    assert torch.isfinite(p[7]) and p[8] == 0 and m[8] == 0 and v[8] == 0
    rest = torch.ones(k, dtype=torch.bool, device=dev())
    rest[[5, 6, 7, 8, 200]] = False
    assert torch.equal(p[rest], clean[rest])
    opt.step([ok])
    assert torch.isnan(p[5:7]).all() and torch.isfinite(p[rest]).all()
    # tiny next to large: the second moment of the small one stays above zero, its update bounded
    q = torch.zeros(128, device=dev())
    o = mm.AdamW8([q], lr=1e-3)
    h = torch.full((128,), 1e-12, device=dev())
    h[0] = 1e6
    for _ in range(3):
        o.step([h])
    m, v = o.moments()
    assert (v > 0).all() and torch.isfinite(q).all() and (q.abs() <= 1e-2).all()


def test_adamw8_rounding_is_unbiased():
    """Over many elements the moments' mean moves as the exact one's."""
    k, steps = 1 << 18, 20
    p = torch.zeros(k, device=dev())
    opt = mm.AdamW8([p], lr=0.0, betas=(0.9, 0.999), seed=5)
    g = torch.full((k,), 1.0, device=dev())
    opt.step([g])
    g2 = torch.full((k,), 0.9, device=dev())
    for _ in range(steps):
        opt.step([g2])
    m, v = (num(x).mean() for x in opt.moments())
    em, ev = 0.1, 0.001
    for _ in range(steps):
        em, ev = 0.9 * em + 0.1 * 0.9, 0.999 * ev + 0.001 * 0.81
    # a step's rounding has spread below half the spacing (1/16), held at most 20 steps: 5 standard errors
    assert abs(m / em - 1) < 5 * np.sqrt(20) / 16 / np.sqrt(k)
    assert abs(v / ev - 1) < 5 * np.sqrt(20) / 16 / np.sqrt(k)


def test_periodic_muon_with_eight_bit_moments_resumes():
    rng = np.random.default_rng(6)
    W0 = torch.from_numpy(rng.standard_normal((96, 160)).astype(np.float32) * 0.02).to(dev(), torch.bfloat16)
    A0 = [torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev(), torch.bfloat16) for s in ((77,), (30, 50))]
    G = [[torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32) * 1e-2).to(dev(), torch.bfloat16) for t in (W0, *A0)]
         for _ in range(4)]

    def run(resume_at=None):
        W, A = W0.clone(), [a.clone() for a in A0]
        opt = mm.PeriodicMuon([W], aux_params=A, aux_bits=8, aux_seed=3)
        for t in range(4):
            if t == resume_at:
                sd = opt.state_dict()
                opt = mm.PeriodicMuon([W], aux_params=A, aux_bits=8)
                opt.load_state_dict(sd)
            opt.step(G[t][:1], G[t][1:])
        return [W, *A]

    assert all(torch.equal(a, b) for a, b in zip(run(), run(2)))
    wide = mm.PeriodicMuon([W0.clone()], aux_params=[a.clone() for a in A0])
    with pytest.raises(ValueError):
        wide.load_state_dict(mm.PeriodicMuon([W0.clone()], aux_params=[a.clone() for a in A0], aux_bits=8).state_dict())


# ------------------------------------------------------------------ differentiable forms
def test_functional_forms_match_torch():
    """layer_norm and linear_cross_entropy under autograd, with broadcast and transposed
    inputs, against torch's own in fp64."""
    rng = np.random.default_rng(2)
    x0, w0, b0 = rng.standard_normal((2, 9, 40)), 1 + 0.1 * rng.standard_normal(40), 0.1 * rng.standard_normal(40)
    v0, lab = rng.standard_normal((111, 40)) * 0.3, rng.integers(0, 111, (2, 9))
    lab[1, 3:] = -100
    labels = torch.from_numpy(lab).to(dev())
    t = [torch.from_numpy(a).to(dev(), torch.float32).requires_grad_() for a in (x0, w0, b0, v0)]
    loss = mm.linear_cross_entropy(mm.layer_norm(t[0], t[1], t[2]), t[3], labels)
    (2.5 * loss).backward()
    r = [torch.from_numpy(a).float().double().requires_grad_() for a in (x0, w0, b0, v0)]
    y = torch.nn.functional.layer_norm(r[0], (40,), r[1], r[2])
    want = torch.nn.functional.cross_entropy((y @ r[3].T).view(-1, 111), torch.from_numpy(lab).view(-1))
    (2.5 * want).backward()
    assert abs(loss.item() - want.item()) < 1e-5
    for a, b in zip(t, r):
        assert np.linalg.norm(num(a.grad) - b.grad.numpy()) < 1e-5 * np.linalg.norm(b.grad.numpy())
    # a broadcast upstream gradient, and an input whose columns are not contiguous
    x = torch.from_numpy(x0[0].T.copy()).to(dev(), torch.float32).T.requires_grad_()
    mm.layer_norm(x, t[1].detach()).sum().backward()
    q = torch.from_numpy(x0[0]).float().double().requires_grad_()
    torch.nn.functional.layer_norm(q, (40,), r[1].detach()).sum().backward()
    assert np.max(np.abs(num(x.grad) - q.grad.numpy())) < 1e-5


def test_example_learns():
    """The head's operators and Muon together: examples/lm_head_step.py's loss falls."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "lm_head_step.py")
    spec = importlib.util.spec_from_file_location("lm_head_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(steps=60, verbose=False)
    assert abs(losses[0] - np.log(mod.VOCAB)) < 0.5 and losses[-1] < losses[0] - 2.0
