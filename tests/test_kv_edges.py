"""CPU tests of the plan of bq_kv_attention at the edges of its sizes: what it asks for and refuses
before any HIP call."""
import pytest
import torch

import dequantization_block_absmax_amd as bq
from test_kv_boundary import attend, batch, cache


@pytest.mark.parametrize("kw", [dict(max_kv_len=0), dict(table_stride=0), dict(max_kv_len=0, max_q_len=3),
                                dict(max_kv_len=0, num_seqs=1, tokens=1), dict(table_stride=0, num_seqs=65535)],
                         ids=str)
@pytest.mark.parametrize("heads", [4, 16])
def test_a_batch_without_keys_is_planned(kw, heads):
    """A call whose sequences have no key is planned like another: nothing to split or to join."""
    assert bq.bq_kv_attention_workspace_bytes(cache(), batch(**kw), bq.BQ_BF16, heads) == 0


@pytest.mark.parametrize("dim,over", [(256, 1 << 26), (128, 1 << 27), (64, 1 << 28)])
def test_a_join_that_is_too_large_is_refused_before_any_work(dim, over):
    """Splits of the keys are joined by a launch of their own, 256 threads for 1024 / dim rows; where that counts
    more than 2^32 - 1 threads nothing at all is enqueued."""
    c = cache(head_dim=dim, blocksize=64, kv_heads=64)
    b = batch(num_seqs=2, tokens=over // 4096 + 1, max_q_len=1, max_kv_len=20000, table_stride=2000)
    assert bq.bq_kv_attention_workspace_bytes(c, b, bq.BQ_BF16, 4096) > 2 * over * dim * 4
    row = 4096 * dim
    assert attend(c, b, heads=4096, q_stride=row, out_stride=row) == bq.BQ_ERR_SIZE


@pytest.mark.parametrize("dtype", [bq.BQ_F16, bq.BQ_BF16])
def test_the_expanded_copy_may_take_four_gib(dtype):
    """64 sequences of up to 16384 keys, 8 heads of 128, one of them long: 4 GiB of expanded keys and values, in either
    type; twice as many keys are left to the other kernel, whose workspace is partial sums."""
    c = cache(kv_heads=8, num_pages=1 << 14, page_size=64)
    def need(keys):
        b = batch(num_seqs=64, tokens=2111, max_q_len=2048, max_kv_len=keys, table_stride=keys // 64)
        return bq.bq_kv_attention_workspace_bytes(c, b, dtype, 32)
    assert 4 << 30 < need(16384) < (4 << 30) * 5 // 4 + (1 << 29)
    assert 0 < need(32768) < 1 << 30


def test_page_tables_that_no_stride_describes():
    """kv_batch reads the stride off the table: a transposed or an expanded one has none, and was read wrongly, or as
    if it were empty."""
    t = torch.zeros(3, 7, dtype=torch.int32)
    lens = torch.zeros(3, dtype=torch.int32)

    def stride(table, **kw):
        return bq.kv_batch(lens, lens, table, 3, 1, 16, **kw).table_stride

    assert stride(t) == 7 and stride(t[:, :4]) == 7 and stride(t[:, 2:]) == 7 and stride(t[::2]) == 14
    assert stride(t[:1, :4]) == 4 and stride(t[:, :1]) == 7 and stride(t.t().contiguous().t()[:1, :1]) == 1
    assert stride(t.t(), table_stride=5) == 5
    for bad in (t.t(), t[:1].expand(3, 7), t[:, ::2]):
        with pytest.raises(ValueError):
            stride(bad)
