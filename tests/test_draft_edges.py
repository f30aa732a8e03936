"""CPU tests of what bq_kv_append refuses at the edge of its sizes, before any HIP call."""
import dequantization_block_absmax_amd as bq
from test_draft_boundary import append
from test_kv_boundary import FAKE, cache


def test_a_launch_that_is_too_large_is_refused_before_any_work():
    """Keys, values and queries stand side by side in one launch, which counts at most 2^32 - 1 threads."""
    c = cache(num_pages=1 << 20, blocksize=128)
    assert append(c, tokens=2 ** 25 - 1, q=None) == bq.BQ_ERR_SIZE
    heads, row = 512, 512 * 128
    assert append(c, tokens=2 ** 18 - 1, q_stride=row, heads=heads, k_stride=1 << 16, v_stride=1 << 16, q_out=2 * FAKE,
                  q_out_stride=row, positions=None) == bq.BQ_ERR_NULL  # 2^34 - 2^16 elements of queries pass the check of sizes
    c = cache(kv_heads=512, num_pages=1 << 12, blocksize=128)
    assert append(c, tokens=2 ** 18 - 1, k_stride=row, v_stride=row, heads=heads, q_stride=row, q_out_stride=row) == bq.BQ_ERR_SIZE
