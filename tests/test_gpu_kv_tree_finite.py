"""Queries of a tree that are not finite: each makes its own result NaN and no other, however the keys are split."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
from draft_helpers import reference, run_tree
from gpu_helpers import BQ_DT
from test_gpu_kv_tree_rows import BOUND, dev, make

pytestmark = pytest.mark.gpu

# Sequences, heads, heads of keys and values, bound on the lengths, and the numbers of splits that the plan may have.  The kernel for many
# rows takes the last four.
PLANS = {
    "few rows, whole": ([(1, 130)], 8, 2, None, (1, 1)),
    "few rows, few splits": ([(5, 3000)], 8, 2, None, (2, 16)),
    "few rows, several sequences": ([(12, 4000), (3, 90), (9, 2500)], 8, 2, None, (2, 16)),
    "few rows, many splits": ([(12, 30000)], 8, 2, None, (17, 64)),
    "many rows, whole": ([(250, 256), (256, 256)] + [(2, 40)] * 14, 64, 16, None, (1, 1)),
    "many rows, few splits": ([(256, 6200)], 32, 8, None, (2, 16)),
    "many rows, several sequences": ([(64, 1500), (40, 700)] + [(2, 50)] * 14, 64, 16, 2048, (2, 16)),
    "many rows, many splits": ([(40, 900), (33, 300)], 8, 2, BOUND, (17, 64)),
}


def check(dev, plan, dim, block, bits, dtype, bad):
    lens, heads, kv_heads, bound, splits = PLANS[plan]
    rng = np.random.default_rng(dim + bits)
    pool, batch, parents, q = make(dev, rng, lens, heads, kv_heads, dim, block, bits, 16, dtype, bound=bound)
    if dim == 128:
        size = bq.bq_kv_tree_attention_workspace_bytes(pool.cache, batch.batch, BQ_DT[dtype], heads)
        per = batch.tokens * heads * (dim + 3) * 4
        assert splits[0] <= max(size // per, 1) <= splits[1], size // per
    want, want_lse, tol, tol_lse = reference(pool, batch, parents, q, dtype, dim ** -0.5)
    rows = [(batch.tokens - 1, heads - 1), (0, heads - 2)]
    for token, head in rows:
        q[token, head, 5 + head] = float(bad)
    out, lse = run_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5)
    torch.cuda.synchronize()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for token, head in rows:
        assert np.isnan(out[token, head]).all(), (token, head, out[token, head][:4], lse[token, head])
        assert bad != "nan" or np.isnan(lse[token, head]), (token, head, lse[token, head])
        out[token, head], lse[token, head] = want[token, head], want_lse[token, head]
    assert (np.abs(out - want) <= tol).all() and (np.abs(lse - want_lse) <= tol_lse).all()


@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("dtype,bits", [("bfloat16", 4), ("float16", 8)])
@pytest.mark.parametrize("plan", PLANS)
def test_queries_that_are_not_finite(dev, plan, dtype, bits, bad):
    check(dev, plan, 128, 64, bits, dtype, bad)


@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("dim,block,bits,dtype", [(64, 32, 8, "float16"), (64, 64, 4, "bfloat16"), (256, 128, 8, "bfloat16"),
                                                  (256, 32, 4, "float16")])
@pytest.mark.parametrize("plan", [p for p in PLANS if p.startswith("few")])
def test_other_widths(dev, plan, dim, block, bits, dtype, bad):
    check(dev, plan, dim, block, bits, dtype, bad)


def test_a_query_of_an_unused_place_may_hold_anything(dev):
    """Its row is zeros, whatever its query; the others' are their own."""
    for plan in ("few rows, few splits", "many rows, many splits"):
        lens, heads, kv_heads, bound, _ = PLANS[plan]
        rng = np.random.default_rng(3)
        pool, batch, parents, q = make(dev, rng, lens, heads, kv_heads, 128, 64, 4, 16, "bfloat16", bound=bound)
        parents[2] = -7
        want, want_lse, tol, tol_lse = reference(pool, batch, parents, q, "bfloat16", 0.088)
        q[2] = float("nan")
        out, lse = run_tree(dev, pool, batch, parents, q, "bfloat16", 0.088)
        torch.cuda.synchronize()
        assert not out[2].any() and torch.isneginf(lse[2]).all()
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (np.abs(out - want) <= tol).all()
        seen = ~np.isneginf(want_lse)
        assert np.array_equal(~np.isneginf(lse), seen) and (np.abs(lse[seen] - want_lse[seen]) <= tol_lse[seen]).all()
