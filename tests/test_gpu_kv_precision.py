"""How exact bq_kv_attention is as a whole where a sequence brings many rows: the 2-norm of its error against
binary64 sums, in units of what rounding the exact result to the type costs.

With q and out in binary16 the cached values are rounded once to binary16, independently of the result's own
rounding and as much: sqrt(2) units.  What keys and weights add is a small part of such a rounding, times
scores of a few: 1.75 in all.  With q in bfloat16, whose unit is 8 times as large, keys (times scores of a few:
5/8), values, weights and the table's entries (1/8 each) are rounded to binary16 once: 1.2 units; the
same bound."""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import TORCH_DT
from kv_helpers import Batch, Pool, hide_unused, queries, reference, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


SHAPES = [(64, 32, 4), (64, 64, 8), (128, 64, 4), (128, 128, 8), (128, 32, 8), (256, 64, 4), (256, 256, 8)]
LENS = {"piece": [(400, 1200)], "whole prompt": [(300, 300)], "both": [(400, 900), (40, 800), (1, 700), (6, 650)]}


@pytest.mark.parametrize("dim,B,bits", SHAPES)
@pytest.mark.parametrize("name", LENS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_error_in_units_of_the_results_rounding(dev, dtype, name, dim, B, bits):
    lens = LENS[name]
    rng = np.random.default_rng(dim + B + bits)
    pool = Pool(dev, synth.table16() if bits == 4 else synth.table256(), sum(-(-kv // 32) for _, kv in lens) + 1, 32, 2, dim, B)
    pool.fill(rng)
    batch = Batch(dev, pool, lens, rng)
    hide_unused(pool, batch)
    q = queries(dev, rng, batch.tokens, 8, dim, dtype, 2.0)
    want = torch.from_numpy(reference(pool, batch, q, dtype, dim ** -0.5)[0])
    rounding = want.to(TORCH_DT[dtype]).double() - want
    out, _ = run_attention(dev, pool, batch, q, dtype, dim ** -0.5)
    error = out.double().cpu() - want
    for s, (n, _) in enumerate(lens):  # each sequence by itself, whatever stands beside it
        if n < 40:
            continue  # single rows: what one key holds is not averaged
        rows = slice(batch.starts[s], batch.starts[s] + n)
        assert error[rows].norm() <= 1.75 * rounding[rows].norm(), (s, float(error[rows].norm() / rounding[rows].norm()))


@pytest.mark.parametrize("dim,B,bits,lens", [(64, 32, 4, [(6, 3000), (5, 900)]), (64, 32, 8, [(6, 3000), (5, 900)]),
                                             (128, 64, 8, [(1, 3000), (1, 900)]), (128, 64, 8, [(6, 3000), (5, 900)]),
                                             (64, 64, 4, [(6, 3000), (1, 900)])])
def test_few_rows_with_weights_in_two_parts(dev, dim, B, bits, lens):
    """binary16, forms whose registers hold the weights' rests: table entries and weights in two parts (2^-22), so that
    the result's own rounding is nearly all: 1.2 units."""
    rng = np.random.default_rng(dim + B + bits)
    pool = Pool(dev, synth.table16() if bits == 4 else synth.table256(), sum(-(-kv // 32) for _, kv in lens) + 1, 32, 2, dim, B)
    pool.fill(rng)
    batch = Batch(dev, pool, lens, rng)
    q = queries(dev, rng, batch.tokens, 8, dim, "float16", 2.0)
    want = torch.from_numpy(reference(pool, batch, q, "float16", dim ** -0.5)[0])
    out, _ = run_attention(dev, pool, batch, q, "float16", dim ** -0.5)
    assert (out.double().cpu() - want).norm() <= 1.2 * (want.half().double() - want).norm()
