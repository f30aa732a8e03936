"""Drafting as a server does it: prompts and drafts appended with rotation, the tree's attention, the accepted path moved to
the front, and the next draft behind it."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
import synth
from draft_helpers import angles, check_tree, random_tree
from gpu_helpers import BQ_DT, TORCH_DT
from kv_helpers import Batch, Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


def slots_of(batch, page, s, at):
    return batch.table[s, at // page].astype(np.int64) * page + at % page


def append(dev, pool, rot, dtype, x, heads, positions, slots, q_out):
    """x: (tokens, heads + 2 kv_heads, dim), the fused projection's output."""
    q, k, v = x[:, :heads], x[:, heads:heads + pool.kv_heads], x[:, heads + pool.kv_heads:]
    bq.check(bq.bq_kv_append(pool.cache, rot, BQ_DT[dtype], k, v, len(positions), k.stride(0), v.stride(0),
                             torch.from_numpy(np.asarray(positions, np.int64)).to(dev),
                             torch.from_numpy(np.asarray(slots, np.int64)).to(dev), q, q.stride(0), heads, q_out,
                             q_out.stride(0)), "append")


@pytest.mark.parametrize("heads,kv_heads,dim,block,bits,page,dtype,nodes", [
    (8, 2, 128, 64, 4, 16, "bfloat16", 24),
    (4, 2, 64, 32, 8, 32, "float16", 9),
    (4, 1, 256, 128, 4, 64, "bfloat16", 5),
    (32, 1, 128, 128, 8, 64, "float16", 70),
])
def test_drafts_one_after_the_other(dev, heads, kv_heads, dim, block, bits, page, dtype, nodes):
    rng = np.random.default_rng(heads * dim + nodes)
    prompts = [37, 1, 300, 0]
    steps, longest = 4, 300 + 5 * nodes
    table = synth.table16() if bits == 4 else synth.table256()
    pool, plain = (Pool(dev, table, 4 * -(-longest // page), page, kv_heads, dim, block) for _ in range(2))
    room = Batch(dev, pool, [(1, longest)] * 4, rng)  # pages of each sequence
    cos, sin = angles(longest, dim)
    cos, sin = torch.from_numpy(cos).to(dev), torch.from_numpy(sin).to(dev)
    rot = bq.rotation(cos, sin, dim, False)

    def project(n):
        return torch.from_numpy(rng.standard_normal((n, heads + 2 * kv_heads, dim)).astype(np.float32)).to(TORCH_DT[dtype]).to(dev)

    # the prompts, in one call into both pools
    at = [np.arange(n) for n in prompts]
    x = project(sum(prompts))
    q_out = torch.empty(len(x), heads, dim, dtype=x.dtype, device=dev)
    slots = np.concatenate([slots_of(room, page, s, a) for s, a in enumerate(at)])
    for p in (pool, plain):
        append(dev, p, rot, dtype, x, heads, np.concatenate(at), slots, q_out)
    have = list(prompts)
    for step in range(steps):
        draft = [int(rng.integers(1, nodes + 1)) for _ in have]
        if step == 1:
            draft[2] = 0  # a sequence that drafts nothing this time
        trees = [random_tree(rng, n) for n in draft]
        depth = []
        for tree in trees:
            d = []
            for parent in tree:
                d.append(d[parent] + 1 if parent >= 0 else 0)
            depth.append(np.array(d, np.int64))
        batch = Batch(dev, pool, [(n, h + n) for n, h in zip(draft, have)], rng)
        batch.table = room.table
        batch.dev[2] = torch.from_numpy(room.table).to(dev)
        batch.batch = bq.kv_batch(*batch.dev, batch.tokens, batch.max_q, batch.max_kv)
        x = project(batch.tokens)
        q_out = torch.empty(len(x), heads, dim, dtype=x.dtype, device=dev)
        places = [h + np.arange(n) for n, h in zip(draft, have)]
        append(dev, pool, rot, dtype, x, heads, np.concatenate([h + d for h, d in zip(have, depth)]),
               np.concatenate([slots_of(room, page, s, a) for s, a in enumerate(places)]), q_out)
        parents = [p for tree in trees for p in tree]
        check_tree(dev, pool, batch, parents, q_out, dtype, dim ** -0.5, tag=step)
        # a path from a root down, as far as it is taken
        paths = []
        for tree in trees:
            path, last = [], -1
            while True:
                below = [i for i, p in enumerate(tree) if p == last]
                if not below or rng.random() < 0.2:
                    break
                last = int(rng.choice(below))
                path.append(last)
            paths.append(path)
        width = max(1, max(len(p) for p in paths))
        path = torch.full((4, width), -1, dtype=torch.int32)
        for s, p in enumerate(paths):
            path[s, :len(p)] = torch.tensor(p, dtype=torch.int32)
        path = path.to(dev)
        bq.check(bq.bq_kv_tree_accept(pool.cache, batch.batch, path, width,
                                      torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)))
        # the same tokens as if nothing had been drafted
        rows = np.concatenate([batch.starts[s] + np.array(p, np.int64) for s, p in enumerate(paths)])
        taken = [h + np.arange(len(p)) for h, p in zip(have, paths)]
        if len(rows):
            append(dev, plain, rot, dtype, x[torch.from_numpy(rows).to(dev)], heads, np.concatenate(taken),
                   np.concatenate([slots_of(room, page, s, a) for s, a in enumerate(taken)]),
                   torch.empty(len(rows), heads, dim, dtype=x.dtype, device=dev))
        have = [h + len(p) for h, p in zip(have, paths)]
        torch.cuda.synchronize()
        for s, h in enumerate(have):
            j = np.arange(h)
            where = (torch.from_numpy(room.table[s, j // page].astype(np.int64)).to(dev), slice(None), torch.from_numpy(j % page).to(dev))
            for a, b in ((pool.packed, plain.packed), (pool.absmax, plain.absmax)):
                for side in range(2):
                    shape = (pool.num_pages, kv_heads, page, -1)
                    now, want = a[side].view(shape)[where], b[side].view(shape)[where]
                    assert torch.equal(now, want), (step, s, side)


def test_a_step_in_a_graph(dev):
    """Append, attention and accept of one draft in one graph, replayed with other drafts; replays and eager steps leave the
    same bits."""
    rng = np.random.default_rng(3)
    heads, kv_heads, dim, page, dtype = 8, 2, 128, 16, "bfloat16"
    lens = [(20, 120), (20, 400)]
    pool, other = (Pool(dev, synth.table16(), 80, page, kv_heads, dim, 64) for _ in range(2))
    pool.fill(rng)
    batch = Batch(dev, pool, lens, rng)
    cos, sin = (torch.from_numpy(t).to(dev) for t in angles(512, dim))
    rot = bq.rotation(cos, sin, dim, True)
    x = torch.zeros(40, heads + 2 * kv_heads, dim, dtype=torch.bfloat16, device=dev)
    q, out = (torch.zeros(40, heads, dim, dtype=torch.bfloat16, device=dev) for _ in range(2))
    positions = torch.zeros(40, dtype=torch.int64, device=dev)
    slots = torch.from_numpy(np.concatenate([slots_of(batch, page, s, kv - n + np.arange(n)) for s, (n, kv) in enumerate(lens)])).to(dev)
    parents = torch.zeros(40, dtype=torch.int32, device=dev)
    path = torch.zeros(2, 4, dtype=torch.int32, device=dev)
    count = torch.zeros(2, dtype=torch.int32, device=dev)
    size = bq.bq_kv_tree_attention_workspace_bytes(pool.cache, batch.batch, bq.BQ_BF16, heads)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device=dev)

    def one(cache, result):
        k, v = x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
        bq.check(bq.bq_kv_append(cache, rot, bq.BQ_BF16, k, v, 40, k.stride(0), v.stride(0), positions, slots, x, x.stride(0),
                                 heads, q, q.stride(0)))
        bq.check(bq.bq_kv_tree_attention(cache, batch.batch, parents, bq.BQ_BF16, q, q.stride(0), heads, 0.088, 0, result,
                                         result.stride(0), None, ws, size))
        bq.check(bq.bq_kv_tree_accept(cache, batch.batch, path, 4, count))

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one(pool.cache, out)
    for k in range(4):
        now = [p for n, _ in lens for p in random_tree(rng, n)]
        parents.copy_(torch.tensor(now, dtype=torch.int32))
        x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32)))
        positions.copy_(torch.from_numpy(rng.integers(0, 512, 40)))
        path.copy_(torch.from_numpy(np.sort(rng.permutation(20)[:8].reshape(2, 4), 1).astype(np.int32)))
        count.copy_(torch.tensor([k, 4 - k], dtype=torch.int32))
        for a, b in zip(other.packed + other.absmax, pool.packed + pool.absmax):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        replayed, queries = out.clone(), q.clone()
        eager = torch.zeros_like(out)
        one(other.cache, eager)
        torch.cuda.synchronize()
        assert torch.equal(replayed, eager) and torch.equal(q, queries), k
        for a, b in zip(other.packed + other.absmax, pool.packed + pool.absmax):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k
