"""CPU test of which kernel a call of bq_kv_tree_attention takes, by what it asks for: 4 drafts of 64 tokens over 2048 keys (64 blocks of 128
rows) are one round of the kernel for few rows, without splits; where there are 256 blocks the kernel for many rows takes shorter
contexts and splits them."""
import pytest

import dequantization_block_absmax_amd as bq
from test_kv_boundary import batch, cache


def need(seqs, nodes, keys, dtype=bq.BQ_BF16, heads=32):
    c = cache(kv_heads=8, num_pages=1 << 14, page_size=64)
    b = batch(num_seqs=seqs, tokens=seqs * nodes, max_q_len=nodes, max_kv_len=keys, table_stride=-(-keys // 64))
    return bq.bq_kv_tree_attention_workspace_bytes(c, b, dtype, heads)


def splits(seqs, nodes, keys, **kw):
    return need(seqs, nodes, keys, **kw) / (seqs * nodes * 32 * (128 + 3) * 4)


@pytest.mark.parametrize("seqs,nodes,keys", [(4, 64, 2048), (8, 32, 2048), (2, 128, 2048)])
def test_few_blocks_take_the_kernel_for_few_rows(seqs, nodes, keys):
    assert splits(seqs, nodes, keys) == 0


@pytest.mark.parametrize("seqs,nodes,keys", [(16, 64, 512), (4, 256, 512), (8, 128, 512), (32, 32, 512)])
def test_many_blocks_take_the_kernel_for_many_rows(seqs, nodes, keys):
    assert splits(seqs, nodes, keys) == 2



def test_blocks_that_few_rows_leave_part_empty():
    """128 drafts of 17 tokens are 1024 blocks of 68 rows: the kernel for few rows, without splits.  128 of 26 are the other's."""
    assert splits(128, 17, 8192) == 0
    assert splits(128, 26, 8192) > 0
