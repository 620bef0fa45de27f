"""Edges of the head's operators on the GPU: extreme values, failures that have to show, long
sums, several pieces of the vocabulary, many rows.

Tolerances are derived as in test_gpu_head.py."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_muon_gb300 as mm
from oracle import head_ref as ref
from test_gpu_head import BF, TYPES, U, ce_case, ce_tolerances, dev, num, put, strided, within

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
