"""Alternatives where their order is hard to keep: rows of W that are copies of one another, large
terms that cancel, entries far below the others.

The logits that rank them are exact to 2^-45 of their largest partial sum; the cases' other
logits lie much farther apart than that, so that the order in 64 bits is the order."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev():
    return torch.device("cuda:0")


def put(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype])
    return t.to(dev()), t.double().numpy()


def ranked(z, top):
    """The largest of each row, equal ones by the lower index."""
    return np.stack([np.lexsort((np.arange(len(r)), -r))[:top] for r in z])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [12, 150, 300])
@pytest.mark.parametrize("d", [136, 1001])
def test_copies_of_a_row_go_by_their_ids(dt, n, d):
    """Equal rows of W have equal logits, whichever lanes and warps add them."""
    rng = np.random.default_rng(n + d)
    v, distinct = 600, 75
    base, base64 = put(rng.standard_normal((distinct, d)), dt)
    which = rng.permutation(np.arange(v) % distinct)
    w = base[torch.from_numpy(which).to(dev())].contiguous()
    ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=20, backward=False)
    for _ in range(4):
        h, h64 = put(rng.standard_normal((n, d)), dt)
        z = (h64 @ base64.T)[:, which]
        for top in (5, 20):
            ids = mm.muon_linear_logprob_forward(h, w, None, ws, top=top)[3].cpu().numpy()
            assert np.array_equal(ids, ranked(z, top)), (top, int((ids != ranked(z, top)).any(1).sum()))


def cancelling(v, d, dt, size, rows, rng):
    """W whose rows (those of the share `rows`) hold a pair of channels, far apart, that cancel
    exactly for the h that has one number in both; `size` is the product of one of them."""
    w = rng.standard_normal((v, d)) * 2 / np.sqrt(d)
    w[:, [3, d - 5]] = 0.0
    b = 2.0 ** rng.integers(-1, 2, v) * (1 + rng.integers(0, 64, v) / 64.0) * (rng.random(v) < rows)
    w[:, 3], w[:, d - 5] = b * np.sqrt(size), -b * np.sqrt(size)
    return put(w, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [2, 8, 40, 200])
@pytest.mark.parametrize("rows", [1.0, 0.02])
def test_terms_that_cancel(dt, n, rows):
    """Partial sums far above the logits: the first sums' error passes the distance between
    neighbours, in every row of W or in some of them."""
    v, d, top = 4096, 520, 8
    for power in (8, 14, 20):
        rng = np.random.default_rng(n + power)
        w, w64 = cancelling(v, d, dt, 4.0 ** (power // 2), rows, rng)
        h = rng.standard_normal((n, d))
        h[:, 3] = h[:, d - 5] = 2.0 ** (power // 2)
        h, h64 = put(h, dt)
        z = h64 @ w64.T
        best = -np.sort(-z, 1)[:, :top + 1]
        partial = (np.abs(h64[:, 3])[:, None] * np.abs(w64[:, 3])).max()
        assert (best[:, :-1] - best[:, 1:]).min() > 2.0 ** -43 * partial          # (the case is one that can be ranked)
        ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=top, backward=False)
        _, _, lse, ids, alt = mm.muon_linear_logprob_forward(h, w, None, ws, top=top)
        assert np.array_equal(ids.cpu().numpy(), ranked(z, top)), (power, int((ids.cpu().numpy() != ranked(z, top)).any(1).sum()))
        # an alternative is its exact logit less lse, rounded once (the exact one to 2^-43 here)
        off = np.abs(alt.double().cpu().numpy() + lse.double().cpu().numpy()[:, None] - best[:, :top])
        assert np.all(off <= 2.0 ** -24 * np.abs(alt.double().cpu().numpy()) + 2.0 ** -42 * partial)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 8, 200])
@pytest.mark.parametrize("low", [-1e4, -1e9, -1e30])
def test_bias_columns_far_below(dt, n, low):
    """Entries shut by a large finite number in their row of W, longer by far than the other rows."""
    v, d, top = 5000, 264, 10
    rng = np.random.default_rng(n)
    h = rng.standard_normal((n, d))
    h[:, -1] = 1.0
    w = rng.standard_normal((v, d)) * 2 / np.sqrt(d)
    w[:, -1] = np.where(np.arange(v) % 5 == 2, low, 0.0)
    (w, w64), (h, h64) = put(w, dt), put(h, dt)
    ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=top, backward=False)
    ids = mm.muon_linear_logprob_forward(h, w, None, ws, top=top)[3].cpu().numpy()
    assert np.array_equal(ids, ranked(h64 @ w64.T, top))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n, v, d", [(160, 70001, 40), (20, 270000, 24), (3, 270000, 24), (153, 33, 8), (200, 481, 72), (5, 481, 72)])
def test_vocabularies_of_all_sizes(dt, n, v, d):
    """More groups of columns than a CTA's threads hold, and fewer than it has threads; long rows, rows of
    zeros and a padded end among W's."""
    rng = np.random.default_rng(v + n)
    w = rng.standard_normal((v, d)) * 2 / np.sqrt(d)
    w[rng.integers(0, v, max(1, v // 50))] *= 30.0
    w[rng.integers(0, v, max(1, v // 50))] = 0.0
    w[v - v // 10:] *= 0.1
    (w, w64), (h, h64) = put(w, dt), put(rng.standard_normal((n, d)), dt)
    z = h64 @ w64.T
    for top in (1, 8, 32):
        ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=top, backward=False)
        ids = mm.muon_linear_logprob_forward(h, w, None, ws, top=top)[3].cpu().numpy()
        part = np.argpartition(-z, min(4 * top + 8, v - 1), 1)[:, :4 * top + 8]
        part.sort(1)
        at = ranked(np.take_along_axis(z, part, 1), top)
        assert np.array_equal(ids, np.take_along_axis(part, at, 1))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [4, 170])
@pytest.mark.parametrize("scale_h, scale_w", [(1e-12, 1.0), (1e12, 1e-12), (1e-9, 1e-9), (1e15, 1e10), (1.0, 1e-20)])
def test_rows_of_all_lengths(dt, n, scale_h, scale_w):
    v, d, top = 3000, 200, 6
    rng = np.random.default_rng(n)
    (w, w64), (h, h64) = put(rng.standard_normal((v, d)) * scale_w, dt), put(rng.standard_normal((n, d)) * scale_h, dt)
    ws = mm.alloc_linear_logprob_workspace(n, v, d, TYPES[dt], top=top, backward=False)
    _, _, lse, ids, _ = mm.muon_linear_logprob_forward(h, w, None, ws, top=top)
    assert torch.isfinite(lse).all() and np.array_equal(ids.cpu().numpy(), ranked(h64 @ w64.T, top))
