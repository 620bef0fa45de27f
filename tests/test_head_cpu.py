"""The head's operators without a GPU: the fp64 oracle against independent facts
(differences, torch's AdamW, the format's definition), the C entry points' refusals and
workspace sizes."""
import ctypes
import os

import numpy as np
import pytest

from oracle import head_ref as ref


@pytest.fixture(scope="session")
def lib():
    from matrix_aware_optimizer_muon_gb300 import _lib
    from matrix_aware_optimizer_muon_gb300 import build as b
    if not os.path.exists(_lib.LIB_PATH):
        b.build()
    return _lib.load_library()


def test_layernorm_gradient_matches_differences():
    rng = np.random.default_rng(0)
    x, dy, w, b = rng.standard_normal((3, 7)), rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal(7)

    def f(x, w, b):
        return (ref.layernorm_forward(x, w, b)[0] * dy).sum()

    _, mean, rstd = ref.layernorm_forward(x, w, b)
    dx, dw, db = ref.layernorm_backward(dy, x, w, mean, rstd)
    for arg, grad in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(arg.shape):
            old = arg[i]
            arg[i] = old + 1e-6
            hi = f(x, w, b)
            arg[i] = old - 1e-6
            lo = f(x, w, b)
            arg[i] = old
            assert abs((hi - lo) / 2e-6 - grad[i]) < 1e-7


def test_linear_ce_gradient_matches_differences():
    rng = np.random.default_rng(1)
    h, w = rng.standard_normal((4, 5)), rng.standard_normal((6, 5))
    labels, coef = np.array([2, -100, 5, 0]), np.array([0.3, 0.9, 1.2, 0.5])

    def f(h, w):
        return (ref.linear_ce_forward(h, w, labels)[0] * coef).sum()

    lse = ref.linear_ce_forward(h, w, labels)[1]
    dh, dw = ref.linear_ce_backward(h, w, labels, lse, coef)
    for arg, grad in ((h, dh), (w, dw)):
        for i in np.ndindex(arg.shape):
            old = arg[i]
            arg[i] = old + 1e-6
            hi = f(h, w)
            arg[i] = old - 1e-6
            lo = f(h, w)
            arg[i] = old
            assert abs((hi - lo) / 2e-6 - grad[i]) < 1e-7
    assert np.all(dh[1] == 0)


def test_grid_is_the_top_bits_of_fp32():
    """value(q) has the fp32 bits q << 20, and place() is its inverse, subnormals included."""
    q = np.arange(0, 2040)
    bits = (q.astype(np.uint32) << 20).view(np.float32).astype(np.float64)
    assert np.array_equal(ref.grid_value(q), bits)
    assert np.array_equal(ref.grid_place(bits), q)


def test_codes_hold_the_largest_value_and_round_to_neighbours():
    rng = np.random.default_rng(2)
    for k in range(40):
        x = rng.standard_normal(ref.BLOCK) * 10.0 ** rng.uniform(-30, 30) * 10.0 ** rng.uniform(-6, 0, ref.BLOCK)
        bits = rng.integers(0, 65536, ref.BLOCK)
        for top, binades, y in ((127, 16, x), (255, 32, np.abs(x))):
            code, scale, value, _ = ref.quantise(y, bits, top, binades)
            base = 8 * max(scale[0] - binades, 0)
            place = ref.grid_place(np.abs(y))
            ok = place >= base + 1
            assert ok[np.argmax(np.abs(y))] and 0 < code[np.argmax(np.abs(y))] <= top
            assert np.all((code + base - np.floor(place))[ok] >= 0) and np.all((code + base - np.floor(place))[ok] <= 1)
            signed = code + 128 * ((value < 0)) if top == 127 else code
            assert np.array_equal(ref.decode(signed, scale, top == 127), value)


def test_rounding_bits_are_uniform_and_independent():
    """Mean, pair correlation of neighbours, steps and halves: within 5 standard errors."""
    n = 1 << 18
    a = ref.random_bits(3, 10, np.arange(n)).astype(np.float64)
    b = ref.random_bits(3, 11, np.arange(n)).astype(np.float64)
    c = ref.random_bits(4, 10, np.arange(n)).astype(np.float64)
    hi, lo = np.floor(a / 65536) / 65536 - 0.5, (a % 65536) / 65536 - 0.5
    for u in (hi, lo):
        assert abs(u.mean()) < 5 / np.sqrt(12 * n)
        assert abs((u ** 2).mean() - 1 / 12) < 5 * np.sqrt(1 / 180 / n)
        for v in (np.roll(u, 1), np.roll(u, 128), np.floor(b / 65536) / 65536 - 0.5, (b % 65536) / 65536 - 0.5,
                  np.floor(c / 65536) / 65536 - 0.5, (c % 65536) / 65536 - 0.5):
            assert abs((u * v).mean() * 12) < 5 / np.sqrt(n)
    assert abs((hi * lo).mean() * 12) < 5 / np.sqrt(n)
    for k in range(32):
        share = ((a.astype(np.int64) >> k) & 1).mean()
        assert abs(share - 0.5) < 2.5 / np.sqrt(n)


def test_adamw8_update_is_torch_adamw():
    import torch
    rng = np.random.default_rng(5)
    p0 = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([p], lr=1e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    q, m, v = p0.copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g)
        opt.step()
        q, m, v = ref.adamw8_update(q, g, m, v, t, 1e-3, 0.9, 0.99, 1e-8, 0.1)
    assert np.allclose(p.detach().numpy(), q, rtol=1e-12, atol=1e-14)


def test_eight_bit_second_moment_follows_its_mean():
    """With beta2 = 0.999 a step moves v by far less than the grid's spacing; rounded
    stochastically it still decays with the exact one, on average over a block's elements."""
    n, t1 = 128 * 64, 1500
    v = np.ones(n)
    for t in range(1, t1 + 1):
        r = ref.random_bits(0, t, np.arange(n)).astype(np.int64) >> 16
        _, _, v, _ = ref.quantise(0.999 * v, r, 255, 32)
    exact = 0.999 ** t1
    # each element's walk has a relative spread below 0.25: the mean of 8192 within 5 of its errors
    assert abs(v.mean() / exact - 1) < 5 * 0.25 / np.sqrt(n)


# ------------------------------------------------------------------- refusals
FAKE = 1 << 20


def test_layernorm_refusals(lib):
    def fwd(x=FAKE, ldx=8, w=None, rows=2, dim=8, xdt=1, wdt=0, eps=1e-5, y=FAKE, ldy=8):
        return lib.muon_layernorm_forward(x, ldx, w, None, rows, dim, xdt, wdt, eps, y, ldy, None, None, None)

    assert fwd(rows=0, x=None, y=None) == 0
    for bad in (dict(x=None), dict(y=None), dict(ldx=7), dict(ldy=7), dict(rows=-1), dict(dim=0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=FAKE + 1), dict(rows=1 << 31), dict(dim=1 << 31), dict(w=FAKE + 2)):
        assert fwd(**bad) == -1, bad
    assert fwd(xdt=2) == -2 and fwd(wdt=7) == -2
    assert lib.muon_layernorm_workspace_size(-1, 8) == ctypes.c_size_t(-1).value
    assert lib.muon_layernorm_workspace_size(3, 0) == ctypes.c_size_t(-1).value
    assert lib.muon_layernorm_workspace_size(3, 8) > 0

    def bwd(dy=FAKE, x=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, rows=2, dim=8, dw=None, ws=None, nws=0, ld=8, xdt=1):
        return lib.muon_layernorm_backward(dy, ld, x, 8, None, mean, rstd, rows, dim, xdt, 0, dx, 8, dw, None, ws, nws,
                                           None)

    assert bwd(rows=0) == 0
    for bad in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(ld=7), dict(dim=0)):
        assert bwd(**bad) == -1, bad
    assert bwd(xdt=3) == -2
    assert bwd(dw=FAKE) == -3
    assert bwd(dw=FAKE, ws=FAKE + 64, nws=1 << 30) == -3
    assert bwd(dw=FAKE, ws=FAKE, nws=8) == -3


def _ce(**kw):
    from matrix_aware_optimizer_muon_gb300 import MuonLinearCe
    d = dict(H=FAKE, W=FAKE, labels=FAKE, rows=4, vocab=16, dim=8, ldh=8, ldw=8, dtype=1, ignore_index=-100)
    d.update(kw)
    return MuonLinearCe(*[d[f[0]] for f in MuonLinearCe._fields_])


def test_linear_ce_refusals(lib):
    big = ctypes.c_size_t(-1).value
    size = lambda a, b: lib.muon_linear_ce_workspace_size(ctypes.byref(a), b)  # noqa: E731
    assert 0 < size(_ce(), 0) <= size(_ce(), 1) < big
    assert lib.muon_linear_ce_workspace_size(None, 0) == big

    def fwd(a, loss=FAKE, lse=FAKE, stats=FAKE, ws=FAKE, n=1 << 40):
        return lib.muon_linear_ce_forward(ctypes.byref(a), loss, lse, stats, ws, n, None)

    def bwd(a, lse=FAKE, dH=FAKE, dW=FAKE, ws=FAKE, n=1 << 40):
        return lib.muon_linear_ce_backward(ctypes.byref(a), lse, None, None, None, 1.0, dH, dW, ws, n, None)

    for bad in (dict(rows=-1), dict(vocab=0), dict(dim=0), dict(ldh=7), dict(ldw=7), dict(rows=1 << 31)):
        assert size(_ce(**bad), 1) == big and fwd(_ce(**bad)) == -1 and bwd(_ce(**bad)) == -1, bad
    for bad in (dict(H=None), dict(W=None), dict(labels=None), dict(H=FAKE + 1), dict(W=FAKE + 1), dict(labels=FAKE + 4)):
        assert fwd(_ce(**bad)) == -1 and bwd(_ce(**bad)) == -1, bad
    assert fwd(_ce(dtype=9)) == -2 and bwd(_ce(dtype=9)) == -2 and size(_ce(dtype=9), 0) == big
    assert fwd(_ce(), loss=None) == -1 and fwd(_ce(), lse=None) == -1 and bwd(_ce(), lse=None) == -1
    assert fwd(_ce(), lse=FAKE + 2) == -1 and bwd(_ce(), dW=FAKE + 1) == -1
    for ws, n in ((None, 1 << 40), (FAKE + 16, 1 << 40), (FAKE, 255)):
        assert fwd(_ce(), ws=ws, n=n) == -3 and bwd(_ce(), ws=ws, n=n) == -3
    assert fwd(_ce(), n=size(_ce(), 0) - 1) == -3 and bwd(_ce(), n=size(_ce(), 1) - 1) == -3


def test_sizes_whose_padding_would_pass_31_bits_are_refused(lib):
    big, top = ctypes.c_size_t(-1).value, 1 << 30
    for k in ("rows", "vocab"):
        a = _ce(**{k: top + 1})
        assert lib.muon_linear_ce_workspace_size(ctypes.byref(a), 0) == big, k
        a = _ce(**{k: top})
        assert lib.muon_linear_ce_workspace_size(ctypes.byref(a), 0) < big, k
    a = _ce(dim=top + 1, ldh=top + 8, ldw=top + 8)
    assert lib.muon_linear_ce_workspace_size(ctypes.byref(a), 0) == big
    assert lib.muon_layernorm_workspace_size(3, top + 1) == big and lib.muon_layernorm_workspace_size(3, top) < big
    assert lib.muon_layernorm_workspace_size(top + 1, 3) == big and lib.muon_layernorm_workspace_size(top, 3) < big


def _p8(**kw):
    from matrix_aware_optimizer_muon_gb300.head import _PARAM8
    d = dict(P=FAKE, G=FAKE, m=FAKE, v=FAKE, m_scale=FAKE, v_scale=FAKE, numel=300, first=0, p_dtype=1, g_dtype=1)
    d.update(kw)
    a = np.zeros(1, dtype=_PARAM8)
    for k, v in d.items():
        a[k] = v
    return a


def test_adamw8_refusals(lib):
    def step(arr, n=1, t=1, b1=0.9, b2=0.999, eps=1e-8):
        return lib.muon_adamw8_step(None if arr is None else arr.ctypes.data, n, t, 1e-4, b1, b2, eps, 0.0, 0, None)

    assert step(_p8(), n=0) == 0 and step(None, n=0) == 0
    assert step(None) == -1 and step(_p8(), n=-1) == -1 and step(_p8(), t=0) == -1
    for bad in (dict(P=0), dict(G=0), dict(m=0), dict(v=0), dict(m_scale=0), dict(v_scale=0), dict(numel=-1), dict(first=64),
                dict(first=-128), dict(P=FAKE + 1), dict(m=FAKE + 8), dict(v=FAKE + 1)):
        assert step(_p8(**bad)) == -1, bad
    assert step(_p8(p_dtype=2)) == -2 and step(_p8(g_dtype=5)) == -2
    assert step(np.concatenate([_p8(), _p8(p_dtype=0)]), n=2) == -2
    for kw in (dict(b1=1.0), dict(b2=-0.1), dict(eps=-1.0), dict(b1=float("nan"))):
        assert step(_p8(), **kw) == -1, kw

    def unpack(m=FAKE, ms=FAKE, v=FAKE, vs=FAKE, n=256, mo=FAKE, vo=FAKE):
        return lib.muon_adamw8_unpack(m, ms, v, vs, n, mo, vo, None)

    assert unpack(n=0) == 0
    for bad in (dict(n=100), dict(n=-128), dict(ms=None), dict(vs=None), dict(mo=None), dict(v=None), dict(mo=FAKE + 16),
                dict(m=FAKE + 4)):
        assert unpack(**bad) == -1, bad


def test_python_refusals():
    import torch

    import matrix_aware_optimizer_muon_gb300 as mm
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        mm.muon_layernorm_forward(x)
    with pytest.raises(ValueError):
        mm.muon_linear_ce_forward(x, x, torch.zeros(4, dtype=torch.int64), x)
    with pytest.raises(ValueError):
        mm.AdamW8([])
    with pytest.raises(ValueError):
        mm.AdamW8([x])
    with pytest.raises(ValueError):
        mm.PeriodicMuon([x], aux_params=[x], aux_bits=16)
