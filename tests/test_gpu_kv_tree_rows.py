"""bq_kv_tree_attention with many rows and keys to a call, where a kernel of its own takes it: the batch's bound on the lengths
decides, so short sequences under a large bound reach every edge of it."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
import synth
from draft_helpers import check_tree, compare, random_tree, reference, run_tree
from gpu_helpers import BQ_DT
from kv_helpers import Batch, Pool, hide_unused, queries

pytestmark = pytest.mark.gpu
BOUND = 1 << 19  # keys


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


def widen(dev, pool, batch, bound=BOUND):
    """The same sequences under a larger bound: the page table has a column for every page that it allows."""
    width = -(-bound // pool.page_size)
    table = np.full((len(batch.lens), width), -1, np.int32)
    table[:, :batch.table.shape[1]] = batch.table
    batch.dev[2] = torch.from_numpy(table).to(dev)
    batch.max_kv = bound
    batch.batch = bq.kv_batch(*batch.dev, batch.tokens, batch.max_q, bound)


def make(dev, rng, lens, heads, kv_heads, dim, block, bits, page, dtype, unused=0.0, bound=BOUND, **kw):
    pages = sum(-(-kv // page) for _, kv in lens) + 2
    pool = Pool(dev, synth.table16() if bits == 4 else synth.table256(), pages, page, kv_heads, dim, block)
    pool.fill(rng)
    batch = Batch(dev, pool, lens, rng, **kw)
    hide_unused(pool, batch)
    if bound:
        widen(dev, pool, batch, bound)
    parents = [p for n, _ in lens for p in random_tree(rng, n, unused)]
    return pool, batch, parents, queries(dev, rng, batch.tokens, heads, dim, dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_forms(dev, block, bits, dtype):
    rng = np.random.default_rng(block + bits)
    lens = [(26, 300), (1, 1), (40, 40), (0, 0), (7, 95), (33, 161), (0, 50), (2, 640), (256, 1500)]
    for heads, kv_heads, page in ((2, 2, 16), (8, 2, 64), (7, 1, 32), (12, 3, 128)):
        pool, batch, parents, q = make(dev, rng, lens, heads, kv_heads, 128, block, bits, page, dtype, unused=0.1)
        check_tree(dev, pool, batch, parents, q, dtype, 128 ** -0.5, tag=(block, bits, heads))


@pytest.mark.parametrize("nodes", [5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256])
@pytest.mark.parametrize("heads", [1, 3, 16])
def test_sizes_of_a_tree(dev, nodes, heads):
    rng = np.random.default_rng(nodes)
    lens = [(nodes, nodes + c) for c in (0, 1, 31, 33, 480)]
    pool, batch, parents, q = make(dev, rng, lens, heads, 1, 128, 64, 4, 32, "bfloat16", unused=0.05)
    check_tree(dev, pool, batch, parents, q, "bfloat16", 0.088, tag=(nodes, heads))


@pytest.mark.parametrize("window", [1, 2, 3, 16, 31, 64, 100, 333, 5000])
@pytest.mark.parametrize("bits,dtype", [(8, "float16"), (4, "bfloat16")])
def test_windows(dev, window, bits, dtype):
    """The kernel for few rows takes those with short windows, in the workspace that was asked for without one."""
    rng = np.random.default_rng(window)
    lens = [(60, 700), (9, 9), (30, 35), (64, 164), (5, 4000), (1, 40)]
    for bound in (BOUND, 30000):
        pool, batch, parents, q = make(dev, rng, lens, 12, 2, 128, 64, bits, 64, dtype, unused=0.05, bound=bound)
        n = batch.starts[1]
        parents[:n] = [i - 1 if i % 7 else int(rng.integers(-1, max(1, i))) if i else -1 for i in range(n)]  # long paths
        check_tree(dev, pool, batch, parents, q, dtype, 128 ** -0.5, window=window)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_unused_places_hold_anything(dev, dtype):
    rng = np.random.default_rng(9)
    lens = [(20, 90), (20, 90), (33, 33), (5, 64), (48, 500)]
    pool, batch, parents, q = make(dev, rng, lens, 8, 2, 128, 64, 4, 16, dtype)
    parents = [-1, 0, 0, 1] + [-2] * 16 + [-2] * 20 + [-1, -5, 0, 2, 3] + [-1] * 28 + [-2, -1, -2, 1, 3] + random_tree(rng, 48, 0.4)
    for s, (n, kv) in enumerate(lens):
        bad = [i for i in range(n) if not -1 <= parents[batch.starts[s] + i] < i]
        if len(bad) == n:  # no token at all sees the context
            bad = range(-(kv - n), n)
        for i in bad:
            j = kv - n + i
            for side in range(2):
                a = pool.absmax[side].view(pool.num_pages, pool.kv_heads, pool.page_size, -1)
                a[int(batch.table[s, j // 16]), :, j % 16] = float("nan")
    check_tree(dev, pool, batch, parents, q, dtype, 0.1)
    check_tree(dev, pool, batch, parents, q, dtype, 0.1, window=17)


@pytest.mark.parametrize("bound", [None, BOUND])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_maxima_far_apart(dev, dim, dtype, bound):
    """Keys and values of very different sizes side by side, runs of far smaller and far larger values, and maxima of zero."""
    rng = np.random.default_rng(dim)
    lens = [(40, 900), (24, 400)]
    pool, batch, parents, q = make(dev, rng, lens, 6, 2, dim, 32, 4, 16, dtype, unused=0.05, bound=bound)
    size = [np.ones((pool.num_pages, pool.page_size), np.float32) for _ in range(2)]
    for s, (_, kv) in enumerate(lens):
        j = np.arange(kv)
        page, slot = batch.table[s, j // 16], j % 16
        size[0][page, slot] = np.exp2(-rng.integers(0, 30, kv) * (rng.random(kv) < 0.3)).astype(np.float32)
        step = np.array([0, 0, -70, -70, 0, 20, 20, -70, 0])[np.minimum(j // 100, 8)]
        size[1][page, slot] = np.exp2(step - rng.integers(0, 25, kv) * (rng.random(kv) < 0.1)).astype(np.float32)
        for side in range(2):
            none = rng.random(kv) < 0.05
            size[side][page[none], slot[none]] = 0.0
    for side in range(2):
        a = pool.absmax[side].view(pool.num_pages, pool.kv_heads, pool.page_size, -1)
        a.mul_(torch.from_numpy(size[side]).to(dev)[:, None, :, None])
    check_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5, tag=(dim, bound))
    check_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5, window=150, tag=(dim, bound))
    for side in range(2):  # nothing but zeros: every weight the same
        pool.absmax[side].nan_to_num_(0.0).mul_(0.0)
        check_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5, tag=(dim, bound, "zeros", side))


@pytest.mark.parametrize("seqs", [63, 64, 65, 129, 300, 1024, 1025])
def test_many_sequences(dev, seqs):
    """More sequences than lanes find their parts; some bring no token, some no key."""
    rng = np.random.default_rng(seqs)
    lens = []
    for s in range(seqs):
        n = int(rng.integers(0, 9)) if s % 5 else 0
        lens.append((n, n + int(rng.integers(0, 120)) if s % 7 else n))
    lens[seqs // 2] = (70, 600)
    lens[-1] = (20, 333)
    pool, batch, parents, q = make(dev, rng, lens, 8, 2, 128, 64, 4, 16, "bfloat16", unused=0.1, bound=1 << 15)
    check_tree(dev, pool, batch, parents, q, "bfloat16", 0.088, tag=seqs)


def test_long_contexts_are_split(dev):
    rng = np.random.default_rng(11)
    for lens, heads, kv_heads, dtype, bits in (([(40, 60000)], 16, 4, "float16", 8), ([(33, 30000), (5, 64), (20, 41003)], 8, 2, "bfloat16", 4)):
        pool, batch, parents, q = make(dev, rng, lens, heads, kv_heads, 128, 64, bits, 128, dtype, unused=0.1, bound=None)
        assert bq.bq_kv_tree_attention_workspace_bytes(pool.cache, batch.batch, BQ_DT[dtype], heads) > 0
        check_tree(dev, pool, batch, parents, q, dtype, 0.088, tag=bits)
        check_tree(dev, pool, batch, parents, q, dtype, 0.088, window=2000, tag=bits)


def test_rows_and_limits(dev):
    """Strided rows; rows of no sequence and past max_q_len stay; pages outside the pool, drafts longer than their sequence."""
    rng = np.random.default_rng(13)
    lens = [(10, 100), (6, 4), (24, 200), (3, 60)]
    pool, batch, parents, q = make(dev, rng, lens, 8, 2, 128, 32, 8, 16, "float16", max_q_len=20)
    batch.table[2, 3] = pool.num_pages
    batch.table[3, 0] = -1
    tokens = batch.tokens
    batch.tokens += 5
    widen(dev, pool, batch)
    wide = torch.zeros(tokens + 5, 9, 128, dtype=torch.float16, device=dev)
    wide[:tokens, :8] = q
    out, lse = check_tree(dev, pool, batch, parents + [-1] * 5, wide[:, :8], "float16", 0.088)
    assert (out[tokens:] == 77.0).all() and (out[batch.starts[2] + 20:batch.starts[3]] == 77.0).all()
    assert (lse[tokens:] == 77.0).all()


def test_large_scores(dev):
    rng = np.random.default_rng(15)
    lens = [(40, 300), (17, 80)]
    pool, batch, parents, q = make(dev, rng, lens, 4, 2, 128, 64, 4, 16, "bfloat16", unused=0.1)
    q[3] = 0.0
    q[5] *= 2.0 ** -120
    for scale in (0.0, -0.09, 0.088):
        check_tree(dev, pool, batch, parents, q, "bfloat16", scale, tag=scale)
    out, lse = run_tree(dev, pool, batch, parents, q * 2.0 ** 100, "bfloat16", 1.0)
    torch.cuda.synchronize()
    vmax = np.abs(np.nan_to_num(pool.values(1))).max()
    assert torch.isfinite(out).all() and float(out.abs().max()) <= vmax * (1 + 2.0 ** -7)


def test_replays_and_streams(dev):
    """Two captured calls in one workspace, replayed one after the other with other lengths, trees and queries; and the same
    bits on another stream, at the same time as a call in another workspace."""
    rng = np.random.default_rng(17)
    lens = [(30, 2000), (25, 1500)]
    pool, batch, parents, q = make(dev, rng, lens, 8, 2, 128, 64, 4, 16, "bfloat16", unused=0.1)
    par = torch.tensor(parents, dtype=torch.int64).to(torch.int32).to(dev)
    size = bq.bq_kv_tree_attention_workspace_bytes(pool.cache, batch.batch, bq.BQ_BF16, 8)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)
    outs = [torch.zeros_like(q) for _ in range(2)]

    def one(i, scale):
        bq.check(bq.bq_kv_tree_attention(pool.cache, batch.batch, par, bq.BQ_BF16, q, q.stride(0), 8, scale, 0, outs[i],
                                         outs[i].stride(0), None, ws, size))

    torch.cuda.synchronize()
    graphs = []
    for i, scale in enumerate((0.088, 0.05)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            one(i, scale)
    side = torch.cuda.Stream()
    for k in range(3):
        now = [p for n, _ in lens for p in random_tree(rng, n, 0.1)]
        par.copy_(torch.tensor(now, dtype=torch.int64).to(torch.int32))
        q.copy_(queries(dev, rng, batch.tokens, 8, 128, "bfloat16"))
        batch.lens = [(30, 2000 - 100 * k), (25, 1500 - 77 * k)]
        batch.dev[1].copy_(torch.tensor([kv for _, kv in batch.lens], dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other, _ = run_tree(dev, pool, batch, now, q, "bfloat16", 0.05, with_lse=False)
        eager, eager_lse = run_tree(dev, pool, batch, now, q, "bfloat16", 0.088)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], other)
        compare(eager, eager_lse, *reference(pool, batch, now, q, "bfloat16", 0.088), k)


@pytest.mark.parametrize("bound", [None, BOUND])
@pytest.mark.parametrize("dim", [64, 128])
def test_no_keys_and_rows_elsewhere(dev, dim, bound):
    """Drafts of sequences without a key; rows before the first sequence and between its rows of out stay as they were."""
    rng = np.random.default_rng(dim)
    lens = [(5, 0), (70, 0), (0, 0), (33, 20), (40, 40), (12, 500)]
    pool, batch, parents, q = make(dev, rng, lens, 8, 2, dim, 64, 4, 16, "bfloat16", unused=0.1, bound=bound)
    check_tree(dev, pool, batch, parents, q, "bfloat16", 0.1)
    want, _ = run_tree(dev, pool, batch, parents, q, "bfloat16", 0.1)
    shift = 7
    wide_q = torch.zeros(batch.tokens + shift, 10, dim, dtype=q.dtype, device=dev)
    wide_q[shift:, 1:9] = q
    wide = torch.full((batch.tokens + shift, 11, dim), 77.0, dtype=q.dtype, device=dev)
    lse = torch.full((batch.tokens + shift, 8), 77.0, device=dev)
    starts = batch.dev[0] + shift
    moved = bq.kv_batch(starts, batch.dev[1], batch.dev[2], batch.tokens + shift, batch.max_q, batch.max_kv)
    size = bq.bq_kv_tree_attention_workspace_bytes(pool.cache, moved, bq.BQ_BF16, 8)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device=dev)
    par = torch.tensor([0] * shift + parents, dtype=torch.int64).to(torch.int32).to(dev)
    bq.check(bq.bq_kv_tree_attention(pool.cache, moved, par, bq.BQ_BF16, wide_q[:, 1:9], wide_q.stride(0), 8, 0.1, 0, wide[:, 2:10],
                                     wide.stride(0), lse, ws, size))
    torch.cuda.synchronize()
    assert torch.equal(wide[shift:, 2:10], want)
    assert (wide[:shift] == 77.0).all() and (wide[:, :2] == 77.0).all() and (wide[:, 10] == 77.0).all() and (lse[:shift] == 77.0).all()


@pytest.mark.parametrize("heads,kv_heads,dim", [(128, 1, 128), (64, 64, 128), (128, 1, 64), (96, 3, 256)])
def test_many_heads(dev, heads, kv_heads, dim):
    rng = np.random.default_rng(heads)
    pool, batch, parents, q = make(dev, rng, [(256, 300), (3, 77)], heads, kv_heads, dim, 64, 4, 32, "bfloat16", unused=0.02)
    check_tree(dev, pool, batch, parents, q, "bfloat16", dim ** -0.5)
