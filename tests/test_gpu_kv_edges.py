"""bq_kv_attention at the edges of its arguments: no keys, rows of no sequence, row numbers out of range, scales of
either sign and zero, the largest joins."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
import synth
from kv_helpers import Batch, Pool, check_attention, hide_unused, queries, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("lens", [[(1, 0)], [(1, 0), (1, 0), (3, 0)], [(600, 0), (0, 0), (2, 0)]],
                         ids=["one", "few", "many"])
@pytest.mark.parametrize("by", ["length", "table"])
def test_no_sequence_has_a_key(dev, lens, dtype, by):
    """Zeros, and -infinity in lse, for every row."""
    rng = np.random.default_rng(1)
    pool = Pool(dev, synth.table16(), 2, 16, 2, 64, 64)
    batch = Batch(dev, pool, lens, rng)
    if by == "table":  # room for keys, but no table to find them by
        batch.dev[1].fill_(40)
        batch.batch = bq.kv_batch(*batch.dev, batch.tokens, batch.max_q, 40, table_stride=0)
    q = queries(dev, rng, batch.tokens, 4, 64, dtype)
    out, lse = run_attention(dev, pool, batch, q, dtype, 0.125)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("lens", [[(2, 40), (3, 30), (1, 20)], [(500, 600), (3, 30), (1, 20)]], ids=["few", "many"])
def test_row_numbers_out_of_range(dev, lens):
    """Entries of q_start below zero count as zero and those past the last row as its end, however far
    out: what lies between two of them is never taken for rows."""
    rng = np.random.default_rng(2)
    pool = Pool(dev, synth.table16(), 60, 16, 2, 64, 64)
    pool.fill(rng)
    batch = Batch(dev, pool, lens, rng)
    q = queries(dev, rng, batch.tokens, 4, 64, "bfloat16")
    want, want_lse = run_attention(dev, pool, batch, q, "bfloat16", 0.125)
    n = lens[0][0]
    for starts, kept in (([-2 ** 31, n, -2 ** 31, -2 ** 31], n), ([-7, n, -2 ** 31, -1], n), ([0, n, -5, -9], n),
                         ([0, n, n + 3, 2 ** 31 - 1], n + 4), ([2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, -1], 0)):
        batch.dev[0].copy_(torch.tensor(starts, dtype=torch.int32))
        out, lse = run_attention(dev, pool, batch, q, "bfloat16", 0.125)
        torch.cuda.synchronize()
        assert torch.equal(out[:kept], want[:kept]) and torch.equal(lse[:kept], want_lse[:kept]), starts
        assert bool((out[kept:] == 77.0).all()) and bool((lse[kept:] == 77.0).all()), starts


@pytest.mark.parametrize("tokens", [4095, 4096])
def test_many_splits_of_two_to_the_24_rows(dev, tokens):
    """4096 tokens of 4096 heads, all but two of them in no sequence, over room for more than 16 splits: the
    joining kernel for many splits ends one row short of this."""
    heads, kv_heads, dim, page = 4096, 64, 64, 16
    rng = np.random.default_rng(3)
    pool = Pool(dev, synth.table16(), 12, page, kv_heads, dim, 64)
    pool.fill(rng)
    small = Batch(dev, pool, [(1, 70), (1, 55)], rng)
    q = queries(dev, rng, 2, heads, dim, "bfloat16")
    want, want_lse = run_attention(dev, pool, small, q, "bfloat16", 0.125)

    wide = torch.full((2, 17 * 8192 // page), -1, dtype=torch.int32, device=dev)
    wide[:, :small.dev[2].shape[1]] = small.dev[2]
    b = bq.kv_batch(small.dev[0], small.dev[1], wide, tokens, 1, 17 * 8192)
    size = bq.bq_kv_attention_workspace_bytes(pool.cache, b, bq.BQ_BF16, heads)
    assert size >= 17 * tokens * heads * (dim + 3) * 4
    if torch.cuda.mem_get_info()[0] < size + (8 << 30):
        pytest.skip("not enough memory free")
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    long_q = torch.zeros(tokens, heads, dim, dtype=torch.bfloat16, device=dev)
    long_q[:2] = q
    out = torch.full((tokens, heads, dim), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((tokens, heads), 7.0, device=dev)
    bq.check(bq.bq_kv_attention(pool.cache, b, bq.BQ_BF16, long_q, heads * dim, heads, 0.125, 1, 0, out, heads * dim,
                                lse, ws, size), "attention")
    torch.cuda.synchronize()
    assert bool((out[2:] == 7.0).all()) and bool((lse[2:] == 7.0).all())
    # other splits of the same keys: both within one rounding of the weights (2^-11 of sum p |v|) and of the result
    most = float(np.nanmax(np.abs(pool.values(1))))
    assert bool(((out[:2].float() - want.float()).abs() <= 2 * (2.0 ** -8 * want.float().abs() + 2.0 ** -11 * most)).all())
    assert bool(((lse[:2] - want_lse).abs() <= 2.0 ** -19 * (1 + want_lse.abs())).all())
    del ws
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("scale", [-0.09, 0.0, -0.0, 1e-40, -1e-30])
@pytest.mark.parametrize("lens", [[(1, 5), (1, 300), (2, 130)], [(40, 300)], [(50, 60), (200, 450), (3, 3)]],
                         ids=["few", "many", "chunk"])
@pytest.mark.parametrize("causal,window", [(1, 0), (1, 40), (0, 0)])
def test_scales_of_either_sign_and_zero(dev, causal, window, lens, scale, dtype):
    """A negative scale turns the order of the keys round; with zero every key that a row sees weighs the same, and
    the hidden ones nothing."""
    rng = np.random.default_rng(4)
    pool = Pool(dev, synth.table256(), sum(-(-kv // 16) for _, kv in lens) + 2, 16, 2, 128, 64)
    pool.fill(rng)
    batch = Batch(dev, pool, lens, rng)
    hide_unused(pool, batch)
    batch.table[0, 0] = -1  # a page that is not there
    batch.dev[2].copy_(torch.from_numpy(batch.table))
    q = queries(dev, rng, batch.tokens, 6, 128, dtype)
    check_attention(dev, pool, batch, q, dtype, scale, causal, window)
