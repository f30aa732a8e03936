"""bq_kv_tree_attention on the GPU against binary64, from the definition."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
import synth
from draft_helpers import check_tree, compare, random_tree, reference, run_tree
from gpu_helpers import BQ_DT, TORCH_DT
from kv_helpers import Batch, Pool, hide_unused, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


def make(dev, rng, lens, heads, kv_heads, dim, block, bits, page, dtype, unused=0.0, **kw):
    pages = sum(-(-kv // page) for _, kv in lens) + 2
    pool = Pool(dev, synth.table16() if bits == 4 else synth.table256(), pages, page, kv_heads, dim, block)
    pool.fill(rng)
    batch = Batch(dev, pool, lens, rng, **kw)
    hide_unused(pool, batch)
    parents = [p for n, _ in lens for p in random_tree(rng, n, unused)]
    return pool, batch, parents, queries(dev, rng, batch.tokens, heads, dim, dtype)


FORMS = [  # head_dim, block, bits: every form of the kernels
    (d, b, bits) for d in (64, 128, 256) for b in (32, 64, 128, 256) if b <= d for bits in (4, 8)
]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_forms(dev, form, dtype):
    dim, block, bits = form
    rng = np.random.default_rng(dim + block + bits)
    lens = [(26, 300), (1, 1), (40, 40), (0, 0), (7, 95), (33, 161), (0, 50), (2, 640)]
    for heads, kv_heads in ((2, 2), (8, 2), (7, 1)):
        pool, batch, parents, q = make(dev, rng, lens, heads, kv_heads, dim, block, bits, 16, dtype, unused=0.1)
        check_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5, tag=(form, heads))


@pytest.mark.parametrize("nodes", [1, 2, 3, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256])
@pytest.mark.parametrize("heads", [1, 3, 16])
def test_sizes_of_a_tree(dev, nodes, heads):
    """Tiles that begin and end inside the tree's words; contexts that end anywhere in a group of keys."""
    rng = np.random.default_rng(nodes)
    lens = [(nodes, nodes + c) for c in (0, 1, 31, 33, 480)]
    pool, batch, parents, q = make(dev, rng, lens, heads, 1, 64, 64, 4, 32, "bfloat16", unused=0.05)
    check_tree(dev, pool, batch, parents, q, "bfloat16", 0.125, tag=(nodes, heads))


@pytest.mark.parametrize("window", [1, 2, 3, 16, 31, 64, 100, 333, 5000])
@pytest.mark.parametrize("dim,dtype", [(64, "float16"), (128, "bfloat16"), (256, "bfloat16")])
def test_windows(dev, window, dim, dtype):
    """A window counts positions: a deep token sees less of the context, and not all of its ancestors."""
    rng = np.random.default_rng(window)
    lens = [(60, 700), (9, 9), (30, 35), (64, 164), (5, 4000), (1, 40)]
    pool, batch, parents, q = make(dev, rng, lens, 6, 2, dim, 64, 4, 64, dtype, unused=0.05)
    n = batch.starts[1]
    parents[:n] = [i - 1 if i % 7 else int(rng.integers(-1, max(1, i))) if i else -1 for i in range(n)]  # long paths
    check_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5, window=window)


def test_chains_and_stars(dev):
    """A chain is causal attention; in a star every token sees the context and itself; one root above all others."""
    rng = np.random.default_rng(7)
    lens = [(256, 400), (256, 256), (64, 1000), (200, 333)]
    pool, batch, parents, q = make(dev, rng, lens, 4, 2, 128, 128, 8, 64, "bfloat16")
    shapes = [list(range(-1, 255)), [-1] * 256, [-1] + [0] * 63, [(i - 1) // 2 if i else -1 for i in range(200)]]
    parents = [p for s in shapes for p in s]
    out, _ = check_tree(dev, pool, batch, parents, q, "bfloat16", 0.088)
    check_tree(dev, pool, batch, parents, q, "bfloat16", 0.088, window=90)
    causal = torch.zeros_like(out)
    need = bq.bq_kv_attention_workspace_bytes(pool.cache, batch.batch, bq.BQ_BF16, 4)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    bq.check(bq.bq_kv_attention(pool.cache, batch.batch, bq.BQ_BF16, q, q.stride(0), 4, 0.088, 1, 0, causal,
                                causal.stride(0), None, ws, need))
    torch.cuda.synchronize()
    want, _, tol, _ = reference(pool, batch, parents, q, "bfloat16", 0.088)
    assert (np.abs(causal[:256].double().cpu().numpy() - want[:256]) <= tol[:256]).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_unused_places_hold_anything(dev, dtype):
    """NaN maxima and codes in unused places, at the tree's end, in its middle and everywhere."""
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


def test_long_contexts_are_split(dev):
    rng = np.random.default_rng(11)
    lens = [(12, 30000), (30, 9000)]
    for dim, dtype, bits, heads in ((128, "float16", 8, 4), (64, "bfloat16", 4, 16)):
        pool, batch, parents, q = make(dev, rng, lens, heads, 1, dim, 64, bits, 128, dtype, unused=0.1)
        assert bq.bq_kv_tree_attention_workspace_bytes(pool.cache, batch.batch, BQ_DT[dtype], heads) > 0
        check_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5, tag=dim)
        check_tree(dev, pool, batch, parents, q, dtype, dim ** -0.5, window=2000, tag=dim)


def test_rows_and_limits(dev):
    """Strided rows; rows of no sequence and past max_q_len stay; lengths past max_kv_len, pages outside the pool, drafts
    longer than their sequence."""
    rng = np.random.default_rng(13)
    lens = [(10, 100), (6, 4), (24, 200), (3, 60)]
    pool, batch, parents, q = make(dev, rng, lens, 4, 2, 64, 32, 8, 16, "float16", max_q_len=20)
    batch.table[2, 3] = pool.num_pages
    batch.table[3, 0] = -1
    batch.dev[2].copy_(torch.from_numpy(batch.table))
    tokens = batch.tokens
    batch.batch = bq.kv_batch(*batch.dev, tokens + 5, 20, 200)
    wide = torch.zeros(tokens + 5, 5, 64, dtype=torch.float16, device=dev)
    wide[:tokens, :4] = q
    out, lse = check_tree(dev, pool, batch, parents + [-1] * 5, wide[:, :4], "float16", 0.125)
    assert (out[tokens:] == 77.0).all() and (out[batch.starts[2] + 20:batch.starts[3]] == 77.0).all()
    assert (lse[tokens:] == 77.0).all()


def test_large_and_masked_scores(dev):
    """Logits of thousands, negative and zero scales, queries of zeros and of the type's largest values."""
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
    """A captured call replayed with other lengths, trees and queries, two in one workspace, one after the other, with eager
    calls between; and the same bits on another stream."""
    rng = np.random.default_rng(17)
    lens = [(30, 2000), (25, 1500)]
    pool, batch, parents, q = make(dev, rng, lens, 8, 2, 128, 64, 4, 16, "bfloat16", unused=0.1)
    par = torch.tensor(parents, dtype=torch.int64).to(torch.int32).to(dev)
    size = bq.bq_kv_tree_attention_workspace_bytes(pool.cache, batch.batch, bq.BQ_BF16, 8)
    assert size > 0
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
    for k in range(3):
        now = [p for n, _ in lens for p in random_tree(rng, n, 0.1)]
        par.copy_(torch.tensor(now, dtype=torch.int64).to(torch.int32))
        q.copy_(queries(dev, rng, batch.tokens, 8, 128, "bfloat16"))
        batch.lens = [(30, 2000 - 100 * k), (25, 1500 - 77 * k)]
        batch.dev[1].copy_(torch.tensor([kv for _, kv in batch.lens], dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        eager, _ = run_tree(dev, pool, batch, now, q, "bfloat16", 0.088, with_lse=False)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other, _ = run_tree(dev, pool, batch, now, q, "bfloat16", 0.05, with_lse=False)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], other)
        want, want_lse, tol, tol_lse = reference(pool, batch, now, q, "bfloat16", 0.088)
        assert (np.abs(eager.double().cpu().numpy() - want) <= tol).all(), k


def test_a_cache_past_four_gib(dev):
    """Pages whose codes lie past 2^32 bytes."""
    rng = np.random.default_rng(19)
    page, kv_heads, dim = 128, 8, 128
    pages = (5 << 30) // (page * kv_heads * dim)  # 5 GiB of 8-bit codes
    packed = [torch.zeros(pages * page * kv_heads * dim, dtype=torch.uint8, device=dev) for _ in range(2)]
    absmax = [torch.zeros(pages * page * kv_heads, device=dev) for _ in range(2)]
    small = Pool(dev, synth.table256(), 8, page, kv_heads, dim, dim)
    small.fill(rng)
    batch = Batch(dev, small, [(20, 900)], rng)
    far = torch.from_numpy(rng.permutation(pages - (pages * 9 // 10))[:8] + pages * 9 // 10).to(dev)
    for i in range(2):
        packed[i].view(pages, -1)[far] = small.packed[i].view(8, -1)
        absmax[i].view(pages, -1)[far] = small.absmax[i].view(8, -1)
    big = bq.kv_cache(packed[0], absmax[0], packed[1], absmax[1], small.table, pages, page, kv_heads, dim, dim)
    parents = random_tree(rng, 20)
    q = queries(dev, rng, 20, 16, dim, "bfloat16")
    want, _ = run_tree(dev, small, batch, parents, q, "bfloat16", 0.088)
    table = torch.where(batch.dev[2] >= 0, far.to(torch.int32)[batch.dev[2].clamp(min=0).long()], -1).contiguous()
    moved = bq.kv_batch(batch.dev[0], batch.dev[1], table, 20, 20, 900)
    small.cache, batch.batch = big, moved
    got, _ = run_tree(dev, small, batch, parents, q, "bfloat16", 0.088)
    assert torch.equal(got, want)
    path = torch.tensor([[2, 5, 11, 19]], dtype=torch.int32, device=dev)
    before = [t.view(pages, -1)[far].clone() for t in packed]
    bq.check(bq.bq_kv_tree_accept(big, moved, path, 4, torch.tensor([4], dtype=torch.int32, device=dev)))
    torch.cuda.synchronize()
    for side in range(2):
        now = packed[side].view(pages, kv_heads, page, dim)
        old = before[side].view(8, kv_heads, page, dim)
        for i, p in enumerate((2, 5, 11, 19)):
            a, b = 880 + p, 880 + i
            assert torch.equal(now[int(table[0, b // page]), :, b % page], old[int(batch.dev[2][0, a // page]), :, a % page])
