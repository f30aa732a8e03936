"""bq_kv_append on the GPU: codes, maxima and rotated queries bit for bit against binary32 arithmetic on the host and the
oracle's quantization."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
import oracle
import synth
from draft_helpers import angles, rotated
from gpu_helpers import BQ_DT, TORCH_DT, host_bits
from kv_helpers import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def orc():
    return oracle.Oracle()


class Tokens:
    """New tokens as parts of a fused projection's output, with specials among them."""

    def __init__(self, dev, rng, tokens, heads, kv_heads, dim, dtype, specials=True):
        n = heads + 2 * kv_heads
        x = rng.standard_normal((tokens, n, dim)).astype(np.float32)
        x *= np.exp(2 * rng.standard_normal((1, n, 1))).astype(np.float32)
        if specials and tokens > 2:
            x[0, heads:, :] = 0.0
            x[1, :, 3] = np.nan
            x[1, :, dim - 1] = np.inf
            x[2, :, 1] = -np.inf
            x[-1, :, 0] *= 1e-30 if dtype != "float16" else 1e-5
        self.x = torch.from_numpy(x).to(TORCH_DT[dtype]).to(dev)
        self.q, self.k, self.v = self.x[:, :heads], self.x[:, heads:heads + kv_heads], self.x[:, heads + kv_heads:]

    def host(self, t):
        return t.float().cpu().numpy()


def call(pool, rot, dtype, t, positions, slots, q_out=None, stream=None):
    q = t.q if q_out is not None else None
    bq.check(bq.bq_kv_append(pool.cache, rot, BQ_DT[dtype], t.k, t.v, len(positions), t.k.stride(0), t.v.stride(0),
                             positions, slots, q, t.q.stride(0), t.q.shape[1], q_out,
                             q_out.stride(0) if q_out is not None else 0, stream), "append")


def check_pool(orc, pool, keys, values, slots, positions, max_positions):
    """Every byte of the pool: written ones as the oracle quantizes binary32 keys and values, others untouched."""
    h, d, ps, b = pool.kv_heads, pool.head_dim, pool.page_size, pool.blocksize
    for side, x in enumerate((keys, values)):
        packed = np.full((pool.num_pages, h, ps, d * pool.bits // 8), 0xA5, np.uint8)
        absmax = np.full((pool.num_pages, h, ps, d // b), np.nan, np.float32)
        for i, s in enumerate(slots):
            if not (0 <= s < pool.num_pages * ps and 0 <= positions[i] < max_positions):
                continue
            a, p = orc.quantize_blockwise(np.ascontiguousarray(x[i]).reshape(-1), oracle.F32, b, pool.table)
            packed[s // ps, :, s % ps] = p[:h * d * pool.bits // 8].reshape(h, -1)
            absmax[s // ps, :, s % ps] = a.reshape(h, -1)
        got = pool.absmax[side].cpu().numpy().reshape(absmax.shape)
        assert np.array_equal(np.isnan(got), np.isnan(absmax)), side
        assert np.array_equal(got.view(np.uint32)[~np.isnan(got)], absmax.view(np.uint32)[~np.isnan(got)]), side
        assert np.array_equal(pool.packed[side].cpu().numpy().reshape(packed.shape), packed), side


def check_queries(got, want, dtype):
    """want in binary32, rounded once; a NaN is any NaN."""
    w = torch.from_numpy(want).to(TORCH_DT[dtype])
    g = got.cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    keep = ~torch.isnan(w)
    assert np.array_equal(host_bits(g[keep]), host_bits(w[keep]))


def places(rng, pool, tokens, max_positions, bad=True):
    slots = rng.permutation(pool.num_pages * pool.page_size)[:tokens].astype(np.int64)
    positions = rng.integers(0, max_positions, tokens).astype(np.int64)
    if bad and tokens > 8:
        slots[3], slots[4], slots[5] = -1, pool.num_pages * pool.page_size, -2 ** 63
        positions[6], positions[7], positions[8] = -1, max_positions, 2 ** 62
        positions[0], positions[1] = 0, max_positions - 1
    return slots, positions


SHAPES = [  # tokens, heads, kv_heads, dim, rotary, block, page, bits
    (1, 4, 1, 128, 128, 128, 16, 4), (33, 8, 2, 128, 128, 64, 16, 4), (70, 6, 3, 64, 32, 32, 32, 8), (19, 5, 5, 96, 48, 32, 16, 4),
    (9, 7, 1, 256, 256, 256, 64, 8), (40, 3, 3, 32, 16, 32, 16, 8), (25, 12, 4, 192, 16, 64, 16, 4), (12, 2, 1, 160, 160, 32, 16, 8),
    (11, 1, 1, 32, 32, 32, 16, 4),
]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_matches_binary32(dev, orc, shape, interleaved, dtype):
    tokens, heads, kv_heads, dim, rotary, block, page, bits = shape
    rng = np.random.default_rng(tokens * 31 + dim)
    table = synth.table16() if bits == 4 else synth.table256()
    pool = Pool(dev, table, -(-tokens // page) + 2, page, kv_heads, dim, block)
    t = Tokens(dev, rng, tokens, heads, kv_heads, dim, dtype)
    cos, sin = angles(50, rotary)
    slots, positions = places(rng, pool, tokens, 50)
    c, s = torch.from_numpy(cos).to(dev), torch.from_numpy(sin).to(dev)
    rot = bq.rotation(c, s, rotary, interleaved)
    out = torch.full((tokens, heads + 1, dim), 5.0, dtype=TORCH_DT[dtype], device=dev)
    call(pool, rot, dtype, t, torch.from_numpy(positions).to(dev), torch.from_numpy(slots).to(dev), out[:, :heads])
    torch.cuda.synchronize()
    safe = np.where((positions >= 0) & (positions < 50), positions, 0)
    keys = rotated(t.host(t.k), cos, sin, safe, rotary, interleaved)
    check_pool(orc, pool, keys, t.host(t.v), slots, positions, 50)
    want = rotated(t.host(t.q), cos, sin, safe, rotary, interleaved)
    want[safe != positions] = 5.0  # left out altogether
    check_queries(out[:, :heads], want, dtype)
    assert (out[:, heads] == 5.0).all()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("rotary,interleaved", [(128, False), (128, True), (64, False), (16, True), (16, False)])
@pytest.mark.parametrize("tokens", [7, 4100])  # one head to a lane, and four
def test_queries_in_place(dev, dtype, rotary, interleaved, tokens):
    heads, dim = 10, 128
    rng = np.random.default_rng(rotary + tokens)
    pool = Pool(dev, synth.table16(), 4, 16, 1, dim, 64)
    t = Tokens(dev, rng, tokens, heads, 1, dim, dtype, specials=False)
    before = t.x.clone()
    cos, sin = angles(9000, rotary)
    c, s = torch.from_numpy(cos).to(dev), torch.from_numpy(sin).to(dev)
    positions = rng.integers(0, 9000, tokens).astype(np.int64)
    slots = torch.full((tokens,), -1, dtype=torch.int64, device=dev)  # queries rotate all the same
    call(pool, bq.rotation(c, s, rotary, interleaved), dtype, t, torch.from_numpy(positions).to(dev), slots, t.q)
    torch.cuda.synchronize()
    check_queries(t.q, rotated(before[:, :heads].float().cpu().numpy(), cos, sin, positions, rotary, interleaved), dtype)
    assert torch.equal(t.x[:, heads:], before[:, heads:])
    assert torch.isnan(pool.absmax[0]).all() and (pool.packed[0] == 0xA5).all()


@pytest.mark.parametrize("heads", [1, 5, 32])
def test_many_tokens_out_of_place(dev, orc, heads):
    """Four heads to a lane of the queries, the last group not full; every key and value."""
    tokens, dim, rotary = 3001, 64, 48
    rng = np.random.default_rng(heads)
    pool = Pool(dev, synth.table256(), 100, 32, 2, dim, 64)
    t = Tokens(dev, rng, tokens, heads, 2, dim, "bfloat16")
    cos, sin = angles(4096, rotary)
    c, s = torch.from_numpy(cos).to(dev), torch.from_numpy(sin).to(dev)
    slots, positions = places(rng, pool, tokens, 4096)
    out = torch.full((tokens, heads, dim), 5.0, dtype=torch.bfloat16, device=dev)
    call(pool, bq.rotation(c, s, rotary), "bfloat16", t, torch.from_numpy(positions).to(dev), torch.from_numpy(slots).to(dev), out)
    torch.cuda.synchronize()
    safe = np.where((positions >= 0) & (positions < 4096), positions, 0)
    check_pool(orc, pool, rotated(t.host(t.k), cos, sin, safe, rotary, False), t.host(t.v), slots, positions, 4096)
    want = rotated(t.host(t.q), cos, sin, safe, rotary, False)
    want[safe != positions] = 5.0
    check_queries(out, want, "bfloat16")


def test_without_queries_and_with_wide_tables(dev, orc):
    """No queries at all; rows of the tables longer than they need be; another code table (a search by halving)."""
    rng = np.random.default_rng(3)
    table = np.sort(np.concatenate([rng.uniform(-1, -0.01, 128), rng.uniform(0.01, 1, 128)])).astype(np.float32)
    pool = Pool(dev, table, 3, 16, 3, 64, 32)
    t = Tokens(dev, rng, 20, 2, 3, 64, "float16")
    cos, sin = angles(30, 64)
    wide = torch.zeros(30, 2, 40, device=dev)
    wide[:, 0, :32], wide[:, 1, :32] = torch.from_numpy(cos).to(dev), torch.from_numpy(sin).to(dev)
    rot = bq.rotation(wide[:, 0], wide[:, 1], 64)
    assert rot.stride == 80
    slots, positions = places(rng, pool, 20, 30)
    call(pool, rot, "float16", t, torch.from_numpy(positions).to(dev), torch.from_numpy(slots).to(dev))
    torch.cuda.synchronize()
    safe = np.where((positions >= 0) & (positions < 30), positions, 0)
    check_pool(orc, pool, rotated(t.host(t.k), cos, sin, safe, 64, False), t.host(t.v), slots, positions, 30)


def test_unrotated_positions_equal_a_write(dev):
    """At position 0 (cosine 1, sine 0) the cache is what bq_kv_write makes of the same tokens."""
    rng = np.random.default_rng(5)
    pools = [Pool(dev, synth.table16(), 8, 16, 4, 128, 64) for _ in range(2)]
    t = Tokens(dev, rng, 100, 4, 4, 128, "bfloat16", specials=False)
    cos, sin = angles(1, 128)
    c, s = torch.from_numpy(cos).to(dev), torch.from_numpy(sin).to(dev)
    slots = torch.from_numpy(rng.permutation(128)[:100].astype(np.int64)).to(dev)
    call(pools[0], bq.rotation(c, s, 128), "bfloat16", t, torch.zeros(100, dtype=torch.int64, device=dev), slots)
    bq.check(bq.bq_kv_write(pools[1].cache, bq.BQ_BF16, t.k, t.v, 100, t.k.stride(0), t.v.stride(0), slots))
    torch.cuda.synchronize()
    for side in range(2):
        assert torch.equal(pools[0].packed[side], pools[1].packed[side])
        assert torch.equal(pools[0].absmax[side].nan_to_num(-1.0), pools[1].absmax[side].nan_to_num(-1.0))


def test_captured_on_another_stream(dev, orc):
    """A captured call reads positions and slots anew at each replay."""
    rng = np.random.default_rng(8)
    tokens, heads, dim = 24, 8, 128
    pool = Pool(dev, synth.table16(), 4, 16, 2, dim, 64)
    t = Tokens(dev, rng, tokens, heads, 2, dim, "bfloat16")
    cos, sin = angles(64, dim)
    c, s = torch.from_numpy(cos).to(dev), torch.from_numpy(sin).to(dev)
    rot = bq.rotation(c, s, dim)
    slots, positions = (torch.zeros(tokens, dtype=torch.int64, device=dev) for _ in range(2))
    out = torch.zeros(tokens, heads, dim, dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(pool, rot, "bfloat16", t, positions, slots, out)
    for _ in range(3):
        sl, po = places(rng, pool, tokens, 64)
        slots.copy_(torch.from_numpy(sl))
        positions.copy_(torch.from_numpy(po))
        for i in range(2):
            pool.packed[i].fill_(0xA5)
            pool.absmax[i].fill_(float("nan"))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        safe = np.where((po >= 0) & (po < 64), po, 0)
        check_pool(orc, pool, rotated(t.host(t.k), cos, sin, safe, dim, False), t.host(t.v), sl, po, 64)
        want = rotated(t.host(t.q), cos, sin, safe, dim, False)
        want[safe != po] = 5.0
        check_queries(out, want, "bfloat16")
