"""The 8-bit output of RMS norm to the last bit: given y, a scale is the fp32 number nearest to
max|y|/448 (2^-100 at least), and a code the e4m3 number nearest to the fp32 quotient y/s, ties
to even."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm
from matrix_aware_optimizer_muon_gb300 import head
from oracle import head_ref as ref

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


def codes_of(y):
    """(codes' values, scales) of fp32 rows."""
    n, d = y.shape
    k = -(-d // 128)
    p = np.zeros((n, k * 128))
    p[:, :d] = y
    scale = np.maximum((np.abs(p.reshape(n, k, 128)).max(2) / 448.0).astype(np.float32), np.float32(2.0 ** -100)).astype(np.float64)
    q = p.astype(np.float32) / np.repeat(scale, 128, 1).astype(np.float32)
    return ref.e4m3(q)[:, :d], scale


def next_to_midpoints(n, d, rng):
    """Rows whose groups hold numbers at and next to all the quotients where a code changes."""
    k = -(-d // 128)
    y = np.zeros((n, k * 128), np.float32)
    grid = np.unique(ref.e4m3(np.arange(0, 448 * 1024 + 1) / 1024.0))
    mid = (grid[1:] + grid[:-1]) / 2
    for r in range(n):
        for g in range(k):
            most = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-3, 4))
            s = np.float32(np.float64(most) / 448.0)
            near = (rng.choice(mid, 127) * np.float64(s)).astype(np.float32)
            for _ in range(2):
                near = np.where(rng.random(127) < 0.4, np.nextafter(near, np.float32(rng.choice([0, 1e3]))), near).astype(np.float32)
            y[r, 128 * g: 128 * (g + 1)] = np.append(near * rng.choice([-1, 1], 127), most).astype(np.float32)
    y = y[:, :d]
    y[:, ::128] = np.abs(y).max(1, keepdims=True)          # (a short last group has its largest, too)
    return y


# rows in a warp, a CTA, element by element, in a loop over the row
SHAPES = [(6, 256), (5, 1024), (3, 2048), (3, 4096), (2, 16384), (7, 1023), (4, 1537), (2, 9001), (2, 20001)]


@pytest.mark.parametrize("n, d", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_codes_are_the_nearest(n, d, residual):
    rng = np.random.default_rng(d)
    # y is the weights where every t is 1 or -1 (up to rstd's rounding, which y shows)
    t = torch.from_numpy(np.where(rng.random((n, d)) < 0.5, -1.0, 1.0).astype(np.float32)).to(dev())
    for trial in range(3):
        w = torch.from_numpy(next_to_midpoints(1, d, rng)[0]).to(dev())
        x, r = (t * 0.25, t * 0.75) if residual else (t, None)
        y, codes, scales, _, _ = head._rms_forward(x, w, r, 0.0, True, True, True, None)
        want, scale = codes_of(y.cpu().numpy())
        assert np.array_equal(scales.cpu().numpy().astype(np.float64), scale)
        got = codes.float().cpu().numpy().astype(np.float64)
        assert np.array_equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("n, d", SHAPES)
def test_codes_of_any_rows(n, d):
    """Rows of a wide range of sizes, tiny and huge scales among them."""
    rng = np.random.default_rng(n * d)
    x = torch.from_numpy((rng.standard_normal((n, d)) * 2.0 ** rng.integers(-20, 20, (n, d))).astype(np.float32)).to(dev())
    for power in (0, -90, 100):
        w = torch.from_numpy((rng.standard_normal(d) * 2.0 ** power).astype(np.float32)).to(dev())
        y, codes, scales, _, _ = head._rms_forward(x, w, None, 1e-6, True, True, True, None)
        want, scale = codes_of(y.cpu().numpy())
        assert np.array_equal(scales.cpu().numpy().astype(np.float64), scale)
        assert np.array_equal(codes.float().cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("n, d", [(5, 1024), (3, 4096)])
def test_codes_of_bf16_rows(n, d):
    """t of 1 and -1 and a power of two of columns: rstd is 1 and y is the weights, to the bit."""
    rng = np.random.default_rng(d)
    sign = np.where(rng.random((n, d)) < 0.5, -1.0, 1.0)
    x = torch.from_numpy(sign).to(dev(), torch.bfloat16)
    for trial in range(3):
        w = next_to_midpoints(1, d, rng)[0]
        codes, scales, rstd, _ = mm.muon_rmsnorm_forward_fp8(x, torch.from_numpy(w).to(dev()), eps=0.0)
        assert bool((rstd == 1).all())
        want, scale = codes_of(sign * w)
        assert np.array_equal(scales.cpu().numpy().astype(np.float64), scale)
        assert np.array_equal(codes.float().cpu().numpy().astype(np.float64), want)
