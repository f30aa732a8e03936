"""bq_kv_tree_accept on the GPU: every byte of the pool against moves one by one on the host."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
import synth
from kv_helpers import Batch, Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


def expected(pool, batch, paths):
    """The pool's arrays after the moves."""
    h, d, ps = pool.kv_heads, pool.head_dim, pool.page_size
    parts = [pool.packed[i].cpu().numpy().reshape(pool.num_pages, h, ps, -1).copy() for i in range(2)]
    parts += [pool.absmax[i].cpu().numpy().reshape(pool.num_pages, h, ps, -1).copy() for i in range(2)]
    for s, (n, kv) in enumerate(batch.lens):
        before = -1
        for i, p in enumerate(paths[s][:n]):
            if not before < p < n:
                break
            before = p
            at = [kv - n + p, kv - n + i]
            if min(at) < 0:
                continue
            page = [batch.table[s, a // ps] for a in at]
            if any(g < 0 or g >= pool.num_pages for g in page):
                continue
            for x in parts:
                x[page[1], :, at[1] % ps] = x[page[0], :, at[0] % ps]
    return parts


def move(dev, pool, batch, paths, stride=None, stream=None):
    width = max(1, max(len(p) for p in paths))
    t = torch.full((len(paths), stride or width), 1 << 30, dtype=torch.int32)
    for s, p in enumerate(paths):
        t[s, :len(p)] = torch.tensor(p, dtype=torch.int64).to(torch.int32)
    lens = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)
    t = t.to(dev)
    bq.check(bq.bq_kv_tree_accept(pool.cache, batch.batch, t, t.stride(0), lens, stream), "accept")
    torch.cuda.synchronize()


def check(dev, pool, batch, paths, **kw):
    want = expected(pool, batch, paths)
    move(dev, pool, batch, paths, **kw)
    got = [pool.packed[0], pool.packed[1], pool.absmax[0], pool.absmax[1]]
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy().view(np.uint8), w.reshape(-1).view(np.uint8))


def filled(dev, rng, pages, page, kv_heads, dim, block, bits):
    pool = Pool(dev, synth.table16() if bits == 4 else synth.table256(), pages, page, kv_heads, dim, block)
    pool.fill(rng)
    return pool


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim,block", [(32, 32), (64, 32), (96, 32), (128, 128), (160, 32), (256, 32), (256, 256)])
def test_paths(dev, dim, block, bits):
    """Chains that overlap their own sources, gaps, whole drafts, single tokens, nothing; ragged contexts."""
    rng = np.random.default_rng(dim + bits)
    pool = filled(dev, rng, 60, 16, 3, dim, block, bits)
    lens = [(10, 10), (40, 75), (5, 33), (0, 0), (1, 17), (23, 100), (64, 64), (12, 31), (0, 9)]
    batch = Batch(dev, pool, lens, rng)
    paths = [[1, 2, 3, 4, 5, 6, 7, 8, 9], list(range(1, 40, 2)), [4], [], [0], [0, 1, 9, 10, 22], list(range(64)),
             [2, 3, 5, 7, 11], []]
    check(dev, pool, batch, paths)


def test_long_paths_overlap(dev):
    """More tokens than a wave takes at a time, each source another's destination."""
    rng = np.random.default_rng(1)
    pool = filled(dev, rng, 80, 16, 2, 128, 64, 4)
    batch = Batch(dev, pool, [(256, 300), (200, 200), (256, 256)], rng)
    check(dev, pool, batch, [list(range(1, 256)), sorted(rng.choice(200, 130, replace=False).tolist()), list(range(0, 256, 2))])


@pytest.mark.parametrize("seed", range(4))
def test_random_paths(dev, seed):
    rng = np.random.default_rng(100 + seed)
    pool = filled(dev, rng, 400, [16, 32, 64, 128][seed], 1 + seed, 64, 32, 4)
    lens = []
    for _ in range(40):
        n = int(rng.integers(0, 50))
        lens.append((n, n + int(rng.integers(0, 60))))
    batch = Batch(dev, pool, lens, rng)
    paths = [sorted(rng.choice(n, int(rng.integers(0, n + 1)), replace=False).tolist()) if n else [] for n, _ in lens]
    check(dev, pool, batch, paths, stride=60)


def test_rows_that_do_not_ascend_end(dev):
    rng = np.random.default_rng(2)
    pool = filled(dev, rng, 40, 16, 2, 64, 64, 8)
    batch = Batch(dev, pool, [(20, 30)] * 8, rng)
    paths = [[3, 3, 5], [-1, 4], [5, 2, 9], [19, 20], [2, 2 ** 31 - 1], [1, -2 ** 31, 7], list(range(1, 20)) + [19, 20, 21],
             [0, 2, 3, 20, 5]]
    check(dev, pool, batch, paths)


def test_lengths_and_pages_out_of_range(dev):
    """Path lengths above the draft or negative, drafts longer than the sequence, pages outside the pool."""
    rng = np.random.default_rng(3)
    pool = filled(dev, rng, 40, 16, 2, 64, 32, 4)
    batch = Batch(dev, pool, [(8, 40), (30, 20), (20, 40), (6, 6)], rng)
    batch.table[0, 2] = 40
    batch.table[2, 1] = -5
    batch.dev[2].copy_(torch.from_numpy(batch.table))
    check(dev, pool, batch, [[1, 3, 7], list(range(1, 30)), [2, 6, 9, 18], [1, 5]])
    want = expected(pool, batch, [[], [], [], list(range(6))])
    t = torch.arange(12, dtype=torch.int32, device=dev)
    lens = torch.tensor([-3, -2 ** 31, 0, 2 ** 31 - 1], dtype=torch.int32, device=dev)  # a row for all
    bq.check(bq.bq_kv_tree_accept(pool.cache, batch.batch, t, 0, lens))
    torch.cuda.synchronize()
    for g, w in zip([pool.packed[0], pool.absmax[1]], [want[0], want[3]]):
        assert np.array_equal(g.cpu().numpy().view(np.uint8), w.reshape(-1).view(np.uint8))


def test_captured(dev):
    rng = np.random.default_rng(4)
    pool = filled(dev, rng, 40, 16, 2, 128, 64, 4)
    batch = Batch(dev, pool, [(20, 60), (17, 17)], rng)
    path = torch.zeros(2, 20, dtype=torch.int32, device=dev)
    count = torch.zeros(2, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bq.check(bq.bq_kv_tree_accept(pool.cache, batch.batch, path, 20, count))
    for _ in range(3):
        paths = [sorted(rng.choice(n, int(rng.integers(1, n + 1)), replace=False).tolist()) for n in (20, 17)]
        pool.fill(rng)
        want = expected(pool, batch, paths)
        for s, p in enumerate(paths):
            path[s, :len(p)] = torch.tensor(p, dtype=torch.int32)
        count.copy_(torch.tensor([len(p) for p in paths], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip([pool.packed[0], pool.packed[1], pool.absmax[0], pool.absmax[1]], want):
            assert np.array_equal(g.cpu().numpy().view(np.uint8), w.reshape(-1).view(np.uint8))
