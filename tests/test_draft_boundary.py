"""CPU tests of what bq_kv_append, bq_kv_tree_attention and bq_kv_tree_accept refuse, each before any HIP call, and of the
host's helpers."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
from draft_helpers import chains, seen_by
from test_kv_boundary import BAD_CACHES, FAKE, batch, cache


def rotation(**kw):
    args = dict(cos=FAKE, sin=FAKE, rotary_dim=128, interleaved=False, max_positions=100, stride=64)
    args.update(kw)
    return bq.rotation(**args)


def append(c=None, r=None, **kw):
    args = dict(dtype=bq.BQ_BF16, k=FAKE, v=FAKE, tokens=5, k_stride=512, v_stride=512, positions=FAKE, slots=FAKE, q=FAKE,
                q_stride=2048, heads=16, q_out=FAKE, q_out_stride=2048, stream=0)
    args.update(kw)
    return bq.bq_kv_append(cache() if c is None else c, rotation() if r is None else r, **args)


def tree(c=None, b=None, **kw):
    args = dict(parents=FAKE, dtype=bq.BQ_BF16, q=FAKE, q_stride=2048, heads=16, scale=0.1, window=0, out=FAKE,
                out_stride=2048, lse=None, workspace=FAKE, workspace_bytes=1 << 60, stream=0)
    args.update(kw)
    return bq.bq_kv_tree_attention(cache() if c is None else c, batch() if b is None else b, **args)


def accept(c=None, b=None, **kw):
    args = dict(path=FAKE, path_stride=4, path_len=FAKE, stream=0)
    args.update(kw)
    return bq.bq_kv_tree_accept(cache() if c is None else c, batch() if b is None else b, **args)


@pytest.mark.parametrize("fn", [append, tree, accept])
@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=lambda x: str(x)[:40])
def test_bad_caches(fn, kw, status):
    assert fn(cache(**kw)) == status


def test_null_structs():
    assert bq.bq_kv_append(None, rotation(), bq.BQ_BF16, FAKE, FAKE, 5, 512, 512, FAKE, FAKE, stream=0) == bq.BQ_ERR_NULL
    assert bq.bq_kv_append(cache(), None, bq.BQ_BF16, FAKE, FAKE, 5, 512, 512, FAKE, FAKE, stream=0) == bq.BQ_ERR_NULL
    for c, b in ((None, batch()), (cache(), None)):
        assert bq.bq_kv_tree_attention(c, b, FAKE, bq.BQ_BF16, FAKE, 2048, 16, 0.1, 0, FAKE, 2048, stream=0) == bq.BQ_ERR_NULL
        assert bq.bq_kv_tree_accept(c, b, FAKE, 4, FAKE, stream=0) == bq.BQ_ERR_NULL


def test_append_rows():
    assert append(dtype=3) == bq.BQ_ERR_DTYPE
    for kw in (dict(tokens=-1), dict(tokens=2 ** 34 // 512), dict(k_stride=511), dict(v_stride=0), dict(v_stride=-512),
               dict(k_stride=2 ** 62), dict(heads=0), dict(heads=-3), dict(q_stride=2047), dict(q_out_stride=2047),
               dict(q_out_stride=2 ** 61), dict(q_stride=-2048), dict(tokens=2 ** 34 // 2048), dict(heads=2 ** 31 - 1),
               dict(q_stride=2056)):  # in place with another stride
        assert append(**kw) == bq.BQ_ERR_SIZE, kw
    for name in ("k", "v", "slots", "positions", "q_out"):
        assert append(**{name: None}) == bq.BQ_ERR_NULL, name
    for kw in (dict(k=FAKE + 8), dict(v=FAKE + 2), dict(slots=FAKE + 4), dict(positions=FAKE + 4), dict(q=FAKE + 8),
               dict(q_out=FAKE + 4), dict(k_stride=516), dict(v_stride=513), dict(q_stride=2052, q_out_stride=2052),
               dict(q_out=2 * FAKE, q_out_stride=2052), dict(dtype=bq.BQ_F32, k_stride=514)):
        assert append(**kw) == bq.BQ_ERR_ALIGNMENT, kw
    assert append(tokens=0) == bq.BQ_OK  # nothing enqueued
    assert append(tokens=0, k=None, v=None, slots=None, positions=None, q=None, q_out=None) == bq.BQ_OK
    # without queries theirs are not looked at
    assert append(tokens=0, q=None, heads=-1, q_stride=-5, q_out_stride=3) == bq.BQ_OK


def test_rotations():
    for kw in (dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=-16)):
        assert append(r=rotation(**kw)) == bq.BQ_ERR_FORMAT, kw
    for kw in (dict(max_positions=0), dict(max_positions=-1), dict(stride=60), dict(stride=-64), dict(stride=2 ** 60)):
        assert append(r=rotation(**kw)) == bq.BQ_ERR_SIZE, kw
    for kw in (dict(cos=FAKE + 8), dict(sin=FAKE + 4), dict(stride=66)):
        assert append(r=rotation(**kw)) == bq.BQ_ERR_ALIGNMENT, kw
    for kw in (dict(cos=None), dict(sin=None)):
        assert append(r=rotation(**kw)) == bq.BQ_ERR_NULL, kw


def test_rotation_reads_tables():
    t = torch.zeros(10, 32)
    r = bq.rotation(t, t, 64)
    assert (r.stride, r.max_positions, r.rotary_dim, r.interleaved) == (32, 10, 64, 0)
    assert bq.rotation(t[:, :16], t[:, 16:], 32, True).stride == 32
    assert bq.rotation(t[:1], t[1:2], 64).max_positions == 1 and bq.rotation(t[::2], t[::2], 64).stride == 64
    for c, s, dim in ((t, t, 66), (t.t(), t.t(), 16), (t, t[:5], 64), (t.double(), t.double(), 64), (t[0], t[0], 64),
                      (t, torch.zeros(10, 36)[:, :32], 64), (t[:1].expand(10, 32), t[:1].expand(10, 32), 64), (t.int(), t.int(), 64)):
        with pytest.raises(ValueError):
            bq.rotation(c, s, dim)


def test_tree_validation():
    assert tree(dtype=bq.BQ_F32) == bq.BQ_ERR_DTYPE
    for dim in (32, 96, 160, 192, 224):
        assert tree(cache(head_dim=dim, blocksize=32)) == bq.BQ_ERR_FORMAT
    for kw in (dict(heads=0), dict(heads=15), dict(heads=1 << 21), dict(q_stride=2047), dict(out_stride=0), dict(window=-1),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert tree(**kw) == bq.BQ_ERR_SIZE, kw
    for kw in (dict(num_seqs=-1), dict(num_seqs=65536), dict(tokens=-1), dict(max_q_len=-1), dict(max_q_len=257, tokens=300),
               dict(max_q_len=2 ** 31 - 1), dict(max_kv_len=-1), dict(table_stride=-1), dict(tokens=1 << 31)):
        assert tree(b=batch(**kw)) == bq.BQ_ERR_SIZE, kw
        assert bq.bq_kv_tree_attention_workspace_bytes(cache(), batch(**kw), bq.BQ_BF16, 16) == 0
    for kw in (dict(num_seqs=0), dict(tokens=0), dict(max_q_len=0)):
        assert tree(b=batch(**kw)) == bq.BQ_OK, kw
        assert tree(b=batch(q_start=None, kv_len=None, page_table=None, **kw), q=None, out=None, parents=None) == bq.BQ_OK
    for kw in (dict(q_start=None), dict(kv_len=None), dict(page_table=None)):
        assert tree(b=batch(**kw)) == bq.BQ_ERR_NULL, kw
    for kw in (dict(q=None), dict(out=None), dict(parents=None)):
        assert tree(**kw) == bq.BQ_ERR_NULL, kw
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 4), dict(q_stride=2052), dict(lse=FAKE + 2), dict(parents=FAKE + 2)):
        assert tree(**kw) == bq.BQ_ERR_ALIGNMENT, kw
    long = batch(num_seqs=1, tokens=20, max_q_len=20, max_kv_len=100000, table_stride=7000)
    need = bq.bq_kv_tree_attention_workspace_bytes(cache(), long, bq.BQ_BF16, 16)
    assert need > 0
    assert tree(b=long, workspace_bytes=need - 1) == bq.BQ_ERR_WORKSPACE
    assert tree(b=long, workspace=None) == bq.BQ_ERR_WORKSPACE
    assert tree(b=long, workspace=FAKE + 128) == bq.BQ_ERR_ALIGNMENT


def test_accept_validation():
    for kw in (dict(num_seqs=-1), dict(num_seqs=65536), dict(tokens=-1), dict(max_q_len=-1), dict(max_kv_len=-1),
               dict(table_stride=-1)):
        assert accept(b=batch(**kw)) == bq.BQ_ERR_SIZE, kw
    assert accept(path_stride=-1) == bq.BQ_ERR_SIZE
    assert accept(cache(kv_heads=(1 << 20) + 1, num_pages=1)) == bq.BQ_ERR_SIZE
    for kw in (dict(num_seqs=0), dict(tokens=0)):
        assert accept(b=batch(**kw)) == bq.BQ_OK
        assert accept(b=batch(q_start=None, kv_len=None, page_table=None, **kw), path=None, path_len=None) == bq.BQ_OK
    for kw in (dict(q_start=None), dict(kv_len=None), dict(page_table=None)):
        assert accept(b=batch(**kw)) == bq.BQ_ERR_NULL
    for kw in (dict(path=None), dict(path_len=None)):
        assert accept(**kw) == bq.BQ_ERR_NULL
    for kw in (dict(path=FAKE + 2), dict(path_len=FAKE + 1)):
        assert accept(**kw) == bq.BQ_ERR_ALIGNMENT


def test_the_definition_of_a_tree():
    """The reference itself, by hand: two roots, a branch, an unused place and what follows it."""
    parents = [-1, 0, 0, -1, 2, 9, 5, 4]
    assert chains(parents) == [[0], [1, 0], [2, 0], [3], [4, 2, 0], None, None, [7, 4, 2, 0]]
    seen = seen_by(parents, 12, 0)
    assert seen[4].nonzero()[0].tolist() == [0, 1, 2, 3, 4, 6, 8] and not seen[5].any() and not seen[6].any()
    seen = seen_by(parents, 12, 3)  # token 7 stands at position 7 and sees positions 5, 6 and 7: tokens 2, 4 and 7
    assert seen[7].nonzero()[0].tolist() == [6, 8, 11] and seen[1].nonzero()[0].tolist() == [3, 4, 5]
    assert seen_by([-1, 0, 1], 2, 0).tolist() == [[False, False], [True, False], [True, True]]  # no room for the first
