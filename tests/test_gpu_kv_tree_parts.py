"""Ragged batches of drafts with few rows to a key/value head, whose parts every workgroup finds from the lengths: up to 64 sequences, one for
each lane; past that the keys of each are split alike."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
from draft_helpers import check_tree
from gpu_helpers import BQ_DT
from test_gpu_kv_tree_rows import dev, make

pytestmark = pytest.mark.gpu


def lengths(rng, seqs, most):
    """Drafts of up to 16 tokens; some sequences bring none, some have no context, one is far longer than the others."""
    lens = []
    for s in range(seqs):
        n = int(rng.integers(1, 17)) if s % 6 else 0
        lens.append((n, n + int(rng.integers(0, most)) if s % 5 else n))
    lens[seqs // 3] = (16, 4 * most)
    lens[-1] = (3, most + 3)
    return lens


@pytest.mark.parametrize("seqs", [2, 31, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("dim,block,bits,dtype", [(128, 64, 4, "bfloat16"), (128, 128, 8, "float16"), (64, 32, 8, "float16"),
                                                  (256, 128, 8, "bfloat16")])
def test_ragged_batches(dev, seqs, dim, block, bits, dtype):
    rng = np.random.default_rng(seqs + dim)
    pool, batch, parents, q = make(dev, rng, lengths(rng, seqs, 700), 4, 1, dim, block, bits, 16, dtype, unused=0.05, bound=None)
    if dim < 256 or seqs < 63:  # split: wide heads fill the device with so many sequences
        assert bq.bq_kv_tree_attention_workspace_bytes(pool.cache, batch.batch, BQ_DT[dtype], 4) > 0
    check_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5, tag=(seqs, dim))
    check_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5, window=500, tag=(seqs, dim, "window"))


@pytest.mark.parametrize("seqs", [5, 33, 64])
def test_equal_lengths(dev, seqs):
    rng = np.random.default_rng(seqs)
    pool, batch, parents, q = make(dev, rng, [(8, 1000)] * seqs, 8, 2, 128, 64, 4, 16, "bfloat16", bound=None)
    assert bq.bq_kv_tree_attention_workspace_bytes(pool.cache, batch.batch, bq.BQ_BF16, 8) > 0
    check_tree(dev, pool, batch, parents, q, "bfloat16", 0.088, tag=seqs)


@pytest.mark.parametrize("seqs", [3, 64])
def test_one_sequence_with_all_the_keys(dev, seqs):
    """The others bring nothing: every part there is belongs to one sequence, first or last."""
    rng = np.random.default_rng(seqs)
    for at in (0, seqs - 1):
        lens = [(0, 0)] * seqs
        lens[at] = (16, 9000)
        pool, batch, parents, q = make(dev, rng, lens, 8, 2, 128, 64, 4, 16, "bfloat16", bound=None)
        check_tree(dev, pool, batch, parents, q, "bfloat16", 0.088, tag=at)


@pytest.mark.parametrize("bound", [None, 300])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_a_short_window_in_a_large_batch(dev, dtype, bound):
    """Which kernel a call takes may depend on its window: the workspace that is asked for without one is enough."""
    rng = np.random.default_rng(70)
    most = bound or 700
    lens = [(int(rng.integers(12, 21)), int(rng.integers(40, most))) for _ in range(70)]
    lens[3] = (20, most)
    pool, batch, parents, q = make(dev, rng, lens, 32, 8, 128, 64, 4, 16, dtype, unused=0.05, bound=None)
    for window in (0, 9, 120):
        check_tree(dev, pool, batch, parents, q, dtype, 0.088, window=window, tag=window)
