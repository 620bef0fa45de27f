"""Alternatives where their order is hard to keep: rows of W that are copies of one another.

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
