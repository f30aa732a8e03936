"""CPU tests of the plan of bq_kv_attention at the edges of its sizes: what it asks for and refuses
before any HIP call."""
import pytest

import dequantization_block_absmax_amd as bq
from test_kv_boundary import batch, cache


@pytest.mark.parametrize("kw", [dict(max_kv_len=0), dict(table_stride=0), dict(max_kv_len=0, max_q_len=3),
                                dict(max_kv_len=0, num_seqs=1, tokens=1), dict(table_stride=0, num_seqs=65535)],
                         ids=str)
@pytest.mark.parametrize("heads", [4, 16])
def test_a_batch_without_keys_is_planned(kw, heads):
    """A call whose sequences have no key is planned like another: nothing to split or to join."""
    assert bq.bq_kv_attention_workspace_bytes(cache(), batch(**kw), bq.BQ_BF16, heads) == 0
