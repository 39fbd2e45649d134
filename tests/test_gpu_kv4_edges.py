"""GPU tests of the 4-bit cache and of the key mass where test_gpu_kv4.py has none: rows
without a log-sum-exp whose queries are not finite. Tolerances are those derived there."""
import math

import numpy as np
import pytest
import torch

import chunked_causal_attention_gb300 as cca

from test_gpu_kv4 import MASS_PLANS, bf16, built, check_mass

pytestmark = pytest.mark.gpu

NOT_FINITE = (float("nan"), float("inf"), -float("inf"))


def unset_rows(q, rows):
    """A copy of q [B, H, T, D] whose given rows hold NaN, infinities or the largest values."""
    q = q.clone()
    for i, t in enumerate(rows):
        q[:, i % q.shape[1], t] = (NOT_FINITE + (3e38, -3e38))[i % 5]
        q[:, i % q.shape[1], t, i % 8] = NOT_FINITE[i % 3]
    return q


# ------------------------------------------------------------------ key mass: rows without a log-sum-exp

@pytest.mark.parametrize("plan", ["whole", "cut", "docs", "late context"])
@pytest.mark.parametrize("D,H,Hkv", [(128, 4, 4), (64, 6, 2), (80, 4, 1), (256, 2, 1)])
def test_key_mass_of_rows_without_lse_that_are_not_finite(plan, D, H, Hkv):
    """Such rows count for nothing, as if their queries were any others: the same bits."""
    rng = np.random.default_rng(D + H)
    L, chunks = 700, MASS_PLANS[plan]
    q, k = 2 * bf16(rng, 2, H, L, D), bf16(rng, 2, Hkv, L, D)
    _, lse = cca.forward(q, k, k, chunks)
    rows = [3, 127, 128, 130, 255, 300, 301, 444, 445, 446, 511, 512, 640, 699]
    for i, t in enumerate(rows):
        lse[:, i % H, t] = -math.inf
    ws = cca.key_mass_workspace(q, k, chunks)
    want = cca.key_mass(q, k, lse, chunks, ws=ws)
    check_mass(q, k, lse, chunks, want, D ** -0.5)
    got = cca.key_mass(unset_rows(q, rows), k, lse, chunks, ws=ws)
    assert cca.attn_status(ws) == 0 and torch.equal(got, want)


def test_key_mass_after_a_forward_over_a_nan_query():
    """The forward gives a NaN query row the log-sum-exp -inf; the other rows' weights stand."""
    rng = np.random.default_rng(7)
    q, k = 2 * bf16(rng, 1, 2, 900, 128), bf16(rng, 1, 1, 900, 128)
    chunks = cca.attn_plan(900, 2, cca.PLAN_FLOPS)
    bad = q.clone()
    bad[0, 0, 650] = float("nan")
    _, lse = cca.forward(bad, k, k, chunks)
    assert lse[0, 0, 650] == -math.inf and int(lse.isfinite().sum()) == 2 * 900 - 1
    check_mass(q, k, lse, chunks, cca.key_mass(bad, k, lse, chunks), 128 ** -0.5)
