"""CPU tests of what bq_kv_write, bq_kv_read and bq_kv_attention refuse, each before any HIP call."""
import numpy as np
import pytest

import dequantization_block_absmax_amd as bq
import synth

FAKE = 1 << 20  # an aligned non-null address; never dereferenced by a rejected call
T16 = synth.table16()
T256 = synth.table256()


def cache(**kw):
    args = dict(k_packed=FAKE, k_absmax=FAKE, v_packed=FAKE, v_absmax=FAKE, table=T16, num_pages=8, page_size=16,
                kv_heads=4, head_dim=128, blocksize=64)
    args.update(kw)
    return bq.kv_cache(**args)


def write(c=None, **kw):
    args = dict(dtype=bq.BQ_BF16, k=FAKE, v=FAKE, tokens=5, k_stride=512, v_stride=512, slots=FAKE, stream=0)
    args.update(kw)
    return bq.bq_kv_write(cache() if c is None else c, **args)


def read(c=None, **kw):
    args = dict(dtype=bq.BQ_BF16, k=FAKE, v=FAKE, tokens=5, k_stride=512, v_stride=512, slots=FAKE, stream=0)
    args.update(kw)
    return bq.bq_kv_read(cache() if c is None else c, **args)


def batch(**kw):
    args = dict(q_start=FAKE, kv_len=FAKE, page_table=FAKE, tokens=3, max_q_len=1, max_kv_len=100, num_seqs=3,
                table_stride=7)
    args.update(kw)
    return bq.kv_batch(**args)


def attend(c=None, b=None, **kw):
    args = dict(dtype=bq.BQ_BF16, q=FAKE, q_stride=2048, heads=16, scale=0.1, causal=1, window=0, out=FAKE,
                out_stride=2048, lse=None, workspace=FAKE, workspace_bytes=1 << 60, stream=0)
    args.update(kw)
    return bq.bq_kv_attention(cache() if c is None else c, batch() if b is None else b, **args)


BAD_CACHES = [
    (dict(num_pages=0), bq.BQ_ERR_SIZE), (dict(num_pages=-1), bq.BQ_ERR_SIZE), (dict(kv_heads=0), bq.BQ_ERR_SIZE),
    (dict(kv_heads=-4), bq.BQ_ERR_SIZE), (dict(page_size=8), bq.BQ_ERR_FORMAT), (dict(page_size=0), bq.BQ_ERR_FORMAT),
    (dict(page_size=48), bq.BQ_ERR_FORMAT), (dict(page_size=8192), bq.BQ_ERR_FORMAT),
    (dict(page_size=-16), bq.BQ_ERR_FORMAT), (dict(head_dim=0), bq.BQ_ERR_FORMAT),
    (dict(head_dim=80), bq.BQ_ERR_FORMAT), (dict(head_dim=288), bq.BQ_ERR_FORMAT),
    (dict(blocksize=16), bq.BQ_ERR_BLOCKSIZE), (dict(blocksize=256), bq.BQ_ERR_BLOCKSIZE),
    (dict(blocksize=96), bq.BQ_ERR_BLOCKSIZE), (dict(head_dim=192, blocksize=128), bq.BQ_ERR_BLOCKSIZE),
    (dict(num_pages=2 ** 31 - 1, page_size=4096, blocksize=32), bq.BQ_ERR_SIZE),  # more than INT32_MAX blocks
    (dict(table=None), bq.BQ_ERR_NULL), (dict(table=T16[::-1].copy()), bq.BQ_ERR_TABLE),
    (dict(table=np.float32(np.linspace(-1, 1, 100))), bq.BQ_ERR_TABLE),
    (dict(k_packed=None), bq.BQ_ERR_NULL), (dict(k_absmax=None), bq.BQ_ERR_NULL),
    (dict(v_packed=None), bq.BQ_ERR_NULL), (dict(v_absmax=None), bq.BQ_ERR_NULL),
    (dict(k_packed=FAKE + 8), bq.BQ_ERR_ALIGNMENT), (dict(k_absmax=FAKE + 4), bq.BQ_ERR_ALIGNMENT),
    (dict(v_packed=FAKE + 1), bq.BQ_ERR_ALIGNMENT), (dict(v_absmax=FAKE + 8), bq.BQ_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("fn", [write, read, attend])
@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=lambda x: str(x)[:40])
def test_bad_caches(fn, kw, status):
    assert fn(cache(**kw)) == status


@pytest.mark.parametrize("entry", [bq.bq_kv_write, bq.bq_kv_read])
def test_null_cache(entry):
    assert entry(None, bq.BQ_BF16, FAKE, FAKE, 5, 512, 512, FAKE, 0) == bq.BQ_ERR_NULL


@pytest.mark.parametrize("fn", [write, read])
def test_rows_validation(fn):
    assert fn(dtype=3) == bq.BQ_ERR_DTYPE
    assert fn(tokens=-1) == bq.BQ_ERR_SIZE
    assert fn(tokens=2 ** 34 // 512) == bq.BQ_ERR_SIZE
    assert fn(k_stride=511) == bq.BQ_ERR_SIZE
    assert fn(v_stride=0) == bq.BQ_ERR_SIZE
    assert fn(v_stride=-512) == bq.BQ_ERR_SIZE
    assert fn(k_stride=2 ** 62) == bq.BQ_ERR_SIZE
    assert fn(tokens=0) == bq.BQ_OK  # nothing enqueued
    assert fn(tokens=0, k=None, v=None, slots=None) == bq.BQ_OK
    for name in ("k", "v", "slots"):
        assert fn(**{name: None}) == bq.BQ_ERR_NULL, name
    assert fn(k=FAKE + 8) == bq.BQ_ERR_ALIGNMENT
    assert fn(v=FAKE + 2) == bq.BQ_ERR_ALIGNMENT
    assert fn(slots=FAKE + 4) == bq.BQ_ERR_ALIGNMENT
    assert fn(k_stride=516) == bq.BQ_ERR_ALIGNMENT
    assert fn(v_stride=513) == bq.BQ_ERR_ALIGNMENT
    assert fn(dtype=bq.BQ_F32, k_stride=514) == bq.BQ_ERR_ALIGNMENT


def test_attention_validation():
    assert attend(dtype=bq.BQ_F32) == bq.BQ_ERR_DTYPE
    assert attend(dtype=7) == bq.BQ_ERR_DTYPE
    for dim in (32, 96, 160, 192, 224):
        assert attend(cache(head_dim=dim, blocksize=32)) == bq.BQ_ERR_FORMAT
    assert bq.bq_kv_attention(None, batch(), bq.BQ_BF16, FAKE, 2048, 16, 0.1, 1, 0, FAKE, 2048, None, FAKE, 1 << 40,
                              0) == bq.BQ_ERR_NULL
    assert bq.bq_kv_attention(cache(), None, bq.BQ_BF16, FAKE, 2048, 16, 0.1, 1, 0, FAKE, 2048, None, FAKE, 1 << 40,
                              0) == bq.BQ_ERR_NULL
    for kw in (dict(heads=0), dict(heads=-4), dict(heads=15), dict(heads=1 << 21), dict(q_stride=2047),
               dict(out_stride=0), dict(q_stride=1 << 40), dict(window=-1), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert attend(**kw) == bq.BQ_ERR_SIZE, kw
    for kw in (dict(num_seqs=-1), dict(num_seqs=65536), dict(tokens=-1), dict(max_q_len=-1), dict(max_kv_len=-1),
               dict(table_stride=-1), dict(tokens=1 << 31)):
        assert attend(b=batch(**kw)) == bq.BQ_ERR_SIZE, kw
    for kw in (dict(num_seqs=0), dict(tokens=0), dict(max_q_len=0)):
        assert attend(b=batch(**kw)) == bq.BQ_OK, kw
        assert attend(b=batch(q_start=None, kv_len=None, page_table=None, **kw), q=None, out=None) == bq.BQ_OK
    for kw in (dict(q_start=None), dict(kv_len=None), dict(page_table=None)):
        assert attend(b=batch(**kw)) == bq.BQ_ERR_NULL, kw
    for kw in (dict(q=None), dict(out=None)):
        assert attend(**kw) == bq.BQ_ERR_NULL, kw
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 4), dict(q_stride=2052), dict(out_stride=2049), dict(lse=FAKE + 2)):
        assert attend(**kw) == bq.BQ_ERR_ALIGNMENT, kw
    for kw in (dict(q_start=FAKE + 2), dict(kv_len=FAKE + 1), dict(page_table=FAKE + 3)):
        assert attend(b=batch(**kw)) == bq.BQ_ERR_ALIGNMENT, kw


def test_attention_workspace():
    """A long context over few rows is split, which needs a workspace; invalid or empty calls need none."""
    def size(c=None, b=None, dtype=bq.BQ_BF16, heads=16):
        return bq.bq_kv_attention_workspace_bytes(cache() if c is None else c, batch() if b is None else b, dtype, heads)

    assert size(dtype=bq.BQ_F32) == 0 and size(heads=3) == 0 and size(cache(page_size=7)) == 0
    assert size(b=batch(num_seqs=0)) == 0
    long = batch(num_seqs=1, tokens=1, max_kv_len=100000, table_stride=7000)
    need = size(b=long)
    assert need > 0 and need == size(b=long)
    assert attend(b=long, workspace_bytes=need - 1) == bq.BQ_ERR_WORKSPACE
    assert attend(b=long, workspace=None) == bq.BQ_ERR_WORKSPACE
    assert attend(b=long, workspace=FAKE + 128) == bq.BQ_ERR_ALIGNMENT


def test_attention_sizes_beyond_int32():
    """Counts whose products leave 32 or 64 bits are refused, or planned without overflow."""
    for kw in (dict(tokens=(1 << 31) // 16), dict(tokens=1 << 30, max_q_len=1 << 30)):
        assert attend(b=batch(**kw)) == bq.BQ_ERR_SIZE, kw
    wide = dict(max_kv_len=2 ** 31 - 1, table_stride=2 ** 31 - 1)
    assert attend(b=batch(**wide)) == bq.BQ_ERR_SIZE
    assert bq.bq_kv_attention_workspace_bytes(cache(), batch(**wide), bq.BQ_BF16, 16) == 0
    # an expanded copy of 2^77 bytes is not taken for a small one
    c = cache(kv_heads=1 << 19, num_pages=1, page_size=16, head_dim=128, blocksize=128)
    b = batch(num_seqs=65535, tokens=2047, max_q_len=2047, max_kv_len=1 << 30, table_stride=1 << 26)
    need = bq.bq_kv_attention_workspace_bytes(c, b, bq.BQ_BF16, 1 << 20)
    assert need <= (2047 << 20) * 64 * (128 + 3) * 4 + 256
