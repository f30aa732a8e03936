"""bq_kv_attention against attention in binary64 on the cached values, within the bound that the
kernel's documented roundings allow (kv_helpers.reference)."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
import synth
from gpu_helpers import BQ_DT
from kv_helpers import Batch, Pool, check_attention, hide_unused, queries, reference, run_attention

pytestmark = pytest.mark.gpu

TABLES = {4: synth.table16(), 8: synth.table256()}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


def setup(dev, seed, lens, heads, kv_heads, dim, B, ps, bits, spare=3, table=None, std=1.0):
    rng = np.random.default_rng(seed)
    pages = sum(-(-kv // ps) for _, kv in lens) + spare
    pool = Pool(dev, TABLES[bits] if table is None else table, pages, ps, kv_heads, dim, B)
    pool.fill(rng, std)
    batch = Batch(dev, pool, lens, rng)
    hide_unused(pool, batch)
    return rng, pool, batch


SHAPES = [(d, b) for d in (64, 128, 256) for b in (32, 64, 128, 256) if b <= d]
ONE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 31), (1, 33), (1, 63), (1, 64), (1, 65), (1, 129), (1, 700)]
FEW = [(2, 2), (5, 5), (3, 40), (8, 300), (7, 129), (0, 0), (4, 64), (1, 1)]
MANY = [(40, 40), (130, 300), (1, 257), (0, 0), (65, 513), (16, 700), (257, 257)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim,B", SHAPES)
@pytest.mark.parametrize("lens", [ONE, FEW, MANY], ids=["one", "few", "many"])
def test_shapes(dev, lens, dim, B, bits):
    """Every head size and block size, tokens from one to a few hundred, keys that end anywhere in a
    page and a tile."""
    dtype = "bfloat16" if (dim // B + bits) % 2 else "float16"
    rng, pool, batch = setup(dev, dim + B + bits, lens, 4, 2, dim, B, 16 if bits == 4 else 64, bits)
    q = queries(dev, rng, batch.tokens, 4, dim, dtype)
    check_attention(dev, pool, batch, q, dtype, dim ** -0.5)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("group,kv_heads", [(1, 3), (2, 1), (3, 2), (5, 1), (7, 2), (8, 1), (16, 1), (17, 1), (40, 1)])
def test_head_groups(dev, group, kv_heads, dtype):
    rng, pool, batch = setup(dev, group, [(1, 70), (3, 90), (20, 200), (1, 16)], group * kv_heads, kv_heads, 64, 32, 32, 4)
    q = queries(dev, rng, batch.tokens, group * kv_heads, 64, dtype)
    check_attention(dev, pool, batch, q, dtype, 0.125)


@pytest.mark.parametrize("causal,window", [(1, 1), (1, 7), (1, 64), (1, 100), (1, 100000), (1, 2 ** 31 - 1), (0, 0),
                                           (0, 5), (0, 130)])
@pytest.mark.parametrize("lens", [[(1, 5), (1, 300), (2, 130)], [(50, 60), (200, 450), (3, 3)]], ids=["few", "many"])
def test_masks(dev, lens, causal, window):
    rng, pool, batch = setup(dev, causal * 7 + window % 1000, lens, 6, 2, 128, 64, 16, 8)
    q = queries(dev, rng, batch.tokens, 6, 128, "float16")
    check_attention(dev, pool, batch, q, "float16", 0.09, causal, window)


@pytest.mark.parametrize("lens", [[(4, 2), (3, 0), (1, 0), (2, 1)], [(300, 40), (90, 0), (70, 69), (5, 200)],
                                  [(500, 40), (450, 0), (70, 69), (5, 200)]], ids=["few", "many", "chunk"])
def test_rows_without_keys(dev, lens):
    """More new tokens than keys: the first ones stand before the first key and see nothing."""
    rng, pool, batch = setup(dev, 11, lens, 4, 4, 64, 64, 16, 4)
    q = queries(dev, rng, batch.tokens, 4, 64, "bfloat16")
    out, lse = check_attention(dev, pool, batch, q, "bfloat16", 0.125)
    assert bool((out[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    check_attention(dev, pool, batch, q, "bfloat16", 0.125, causal=0)


@pytest.mark.parametrize("lens", [[(1, 200), (2, 150)], [(80, 200), (150, 150)]], ids=["few", "many"])
def test_pages_outside_the_pool_are_hidden(dev, lens):
    rng, pool, batch = setup(dev, 12, lens, 4, 2, 128, 128, 16, 8)
    for s, p, bad in ((0, 0, -1), (0, 3, pool.num_pages), (0, 4, 2 ** 31 - 1), (1, 2, -2 ** 31), (1, 7, -7)):
        batch.table[s, p] = bad
    batch.dev[2].copy_(torch.from_numpy(batch.table))
    q = queries(dev, rng, batch.tokens, 4, 128, "float16")
    check_attention(dev, pool, batch, q, "float16", 0.09)


@pytest.mark.parametrize("lens", [[(1, 400)], [(100, 400)]], ids=["one", "many"])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_one_key_takes_all(dev, lens, dtype):
    """Keys of powers of two and a scale that leaves one key of each row: the result is that key's
    values, exactly.  A key, value or row in a wrong place shows."""
    table = np.float32([-1, -0.875, -0.75, -0.625, -0.5, -0.375, -0.25, -0.125, 0, 0.125, 0.25, 0.375, 0.5, 0.625,
                        0.75, 1])
    rng, pool, batch = setup(dev, 13, lens, 8, 2, 128, 32, 16, 4, table=table)
    for side in range(2):  # block maxima that are powers of two
        e = torch.from_numpy(rng.integers(-2, 3, pool.absmax[side].numel()).astype(np.float32)).to(dev)
        pool.absmax[side].copy_(torch.where(torch.isnan(pool.absmax[side]), pool.absmax[side], torch.exp2(e)))
    n, kv = lens[0]
    keys = np.nan_to_num(pool.values(0))[batch.table[0, np.arange(kv) // 16], :, np.arange(kv) % 16]  # (kv, 2, 128)
    vals = np.nan_to_num(pool.values(1))[batch.table[0, np.arange(kv) // 16], :, np.arange(kv) % 16]
    sign = np.sign(rng.standard_normal((n, 8, 128))).astype(np.float32)
    q = torch.from_numpy(sign).to(torch.float16 if dtype == "float16" else torch.bfloat16).to(dev)
    out, _ = run_attention(dev, pool, batch, q, dtype, 4096.0)
    got = out.double().cpu().numpy()
    for h in range(8):
        z = sign[:, h].astype(np.float64) @ keys[:, h // 4].T
        z[np.arange(kv) > (kv - n + np.arange(n))[:, None]] = -np.inf
        best = z.argmax(1)
        second = np.sort(z, 1)[:, -2] if kv > 1 else np.full(n, -np.inf)
        clear = z.max(1) - second >= 1 / 32  # logits differ by 4096 / 32 = 128: the rest is below 2^-180
        assert clear.mean() > 0.5
        assert np.array_equal(got[clear, h], vals[best[clear], h // 4])


@pytest.mark.parametrize("lens", [[(1, 300)], [(90, 300)], [(220, 300)]], ids=["one", "many", "chunk"])
@pytest.mark.parametrize("std_q,std", [(1e-3, 1e-3), (30.0, 4.0), (1e-20, 1e18), (1e3, 1e-6)])
def test_magnitudes(dev, lens, std_q, std):
    """Queries and caches far from one (bfloat16), and logits in the hundreds."""
    rng, pool, batch = setup(dev, 14, lens, 4, 2, 128, 64, 64, 8, std=std)
    q = queries(dev, rng, batch.tokens, 4, 128, "bfloat16", std_q)
    check_attention(dev, pool, batch, q, "bfloat16", 0.09)


@pytest.mark.parametrize("lens", [[(1, 96)], [(96, 96)], [(207, 96)]], ids=["one", "many", "chunk"])
def test_zero_cache_and_zero_queries(dev, lens):
    rng, pool, batch = setup(dev, 15, lens, 4, 2, 64, 32, 16, 4)
    q = queries(dev, rng, batch.tokens, 4, 64, "float16")
    check_attention(dev, pool, batch, torch.zeros_like(q), "float16", 0.125)
    for a in pool.absmax:
        a.copy_(torch.where(torch.isnan(a), a, torch.zeros_like(a)))
    out, lse = run_attention(dev, pool, batch, q, "float16", 0.125)
    assert bool((out == 0).all())
    seen = torch.arange(96 - lens[0][0] + 1, 97, device=dev).clamp(min=0).float()[:, None].expand_as(lse)
    want = torch.log(seen)  # -infinity where no key is seen
    assert bool(((lse == want) | ((lse - want).abs() <= 2.0 ** -20 * 6)).all())


def test_weak_values_of_the_strongest_key(dev):
    """The key that takes nearly all of the weight has values 2^-17 of the others': the result is its
    values and what little the others add, not what their rounding leaves."""
    rng, pool, batch = setup(dev, 16, [(1, 64)], 4, 1, 128, 128, 64, 8)
    a0 = pool.absmax[0].view(pool.num_pages, 1, 64, 1)
    a1 = pool.absmax[1].view(pool.num_pages, 1, 64, 1)
    page = int(batch.table[0, 0])
    k = pool.values(0)[page, 0, 5]
    q = torch.from_numpy(np.tile(np.sign(k), (1, 4, 1)).astype(np.float32)).to(torch.float16).to(dev)
    a0[page, 0, 5] *= 8.0
    a1[page, 0, 5] = 2.0 ** -17
    check_attention(dev, pool, batch, q, "float16", 0.09)
    out, _ = run_attention(dev, pool, batch, q, "float16", 1.0)
    want = pool.values(1)[page, 0, 5]  # the other keys' weight is below 2^-100 here
    # one rounding of the codes, one of the probability and the last one, each 2^-12 of the value;
    # a step of a subnormal result is 2^-24
    assert np.all(np.abs(out.double().cpu().numpy()[0] - want) <= 3.1 * 2.0 ** -12 * np.abs(want) + 2.0 ** -25 + 2.0 ** -30)


@pytest.mark.parametrize("lens", [[(1, 130), (1, 40)], [(70, 130), (33, 40)], [(250, 300), (3, 9)]],
                         ids=["one", "many", "chunk"])
def test_strides_and_no_lse(dev, lens):
    """q and out as parts of wider rows, on a stream that is not the default one; nothing outside is
    touched."""
    rng, pool, batch = setup(dev, 17, lens, 4, 2, 64, 64, 16, 4)
    wide = torch.zeros(batch.tokens, 4 * 64 + 24, dtype=torch.bfloat16, device=dev)
    q = queries(dev, rng, batch.tokens, 4, 64, "bfloat16")
    wide[:, 8:8 + 256] = q.reshape(batch.tokens, -1)
    out = torch.full((batch.tokens + 2, 300 // 4 * 4 + 4), 5.0, dtype=torch.bfloat16, device=dev)
    want, _ = run_attention(dev, pool, batch, q, "bfloat16", 0.125)
    size = bq.bq_kv_attention_workspace_bytes(pool.cache, batch.batch, bq.BQ_BF16, 4)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    bq.check(bq.bq_kv_attention(pool.cache, batch.batch, bq.BQ_BF16, wide[:, 8:], wide.stride(0), 4, 0.125, 1, 0,
                                out, out.stride(0), None, ws, size, stream))
    torch.cuda.synchronize()
    assert torch.equal(out[:batch.tokens, :256].reshape(q.shape), want)
    assert bool((out[:, 256:] == 5.0).all()) and bool((out[batch.tokens:] == 5.0).all())


def test_bounds_of_the_batch(dev):
    """max_kv_len, the page table's width and max_q_len cut off what lies behind them; rows of no
    sequence stay as they are."""
    rng, pool, batch = setup(dev, 18, [(1, 200), (1, 64)], 4, 2, 64, 64, 16, 4)
    q = queries(dev, rng, 4, 4, 64, "float16")

    def call(b, tokens):
        out = torch.full((4, 4, 64), 9.0, dtype=torch.float16, device=dev)
        size = bq.bq_kv_attention_workspace_bytes(pool.cache, b, bq.BQ_F16, 4)
        ws = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
        bq.check(bq.bq_kv_attention(pool.cache, b, bq.BQ_F16, q, 256, 4, 0.125, 0, 0, out, 256, None, ws, size))
        torch.cuda.synchronize()
        return out

    plain = call(bq.kv_batch(*batch.dev, 2, 1, 200), 2)
    assert bool((plain[2:] == 9.0).all())
    short = torch.tensor([96, 64], dtype=torch.int32, device=dev)
    want = call(bq.kv_batch(batch.dev[0], short, batch.dev[2], 2, 1, 200), 2)
    got = call(bq.kv_batch(*batch.dev, 2, 1, 96), 2)
    assert torch.equal(got[0], want[0]) or bool(((got[0] - want[0]).abs() <= 2.0 ** -9).all())
    narrow = batch.dev[2][:, :6].contiguous()
    got = call(bq.kv_batch(batch.dev[0], batch.dev[1], narrow, 2, 1, 200), 2)
    assert bool(((got[0] - want[0]).abs() <= 2.0 ** -9).all())
    negative = torch.tensor([-5, 64], dtype=torch.int32, device=dev)
    got = call(bq.kv_batch(batch.dev[0], negative, batch.dev[2], 2, 1, 200), 2)
    assert bool((got[0] == 0).all()) and bool(((got[1] - plain[1]).abs() <= 2.0 ** -9).all())


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("lens", [[(1, 20000)], [(4, 9000), (1, 3000)], [(300, 3500)]], ids=["one", "draft", "chunk"])
def test_long_contexts_repeat_bit_for_bit(dev, lens, dtype):
    rng, pool, batch = setup(dev, 19, lens, 8, 2, 128, 64, 64, 4)
    q = queries(dev, rng, batch.tokens, 8, 128, dtype, 2.0)
    out, lse = check_attention(dev, pool, batch, q, dtype, 0.09)
    for _ in range(3):
        again, lse2 = run_attention(dev, pool, batch, q, dtype, 0.09)
        torch.cuda.synchronize()
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(lse, lse2)


def test_offsets_beyond_32_bits(dev):
    """Keys in the last pages of a pool of more than 2^32 bytes of codes give what the same keys give
    in a small pool."""
    heads, dim, B, ps = 8, 256, 256, 64
    rng, small, batch = setup(dev, 20, [(1, 200), (2, 90), (60, 100)], 8, heads, dim, B, ps, 8, spare=0)
    pages = (1 << 32) // (heads * dim * ps) + small.num_pages + 5
    packed = [torch.zeros(pages * heads * ps * dim, dtype=torch.uint8, device=dev) for _ in range(2)]
    absmax = [torch.zeros(pages * heads * ps, dtype=torch.float32, device=dev) for _ in range(2)]
    first = pages - small.num_pages
    for i in range(2):
        packed[i][first * heads * ps * dim:] = small.packed[i]
        absmax[i][first * heads * ps:] = small.absmax[i]
    cache = bq.kv_cache(packed[0], absmax[0], packed[1], absmax[1], small.table, pages, ps, heads, dim, B)
    q = queries(dev, rng, batch.tokens, 8, dim, "float16")
    want, _ = run_attention(dev, small, batch, q, "float16", 0.06)
    moved = batch.dev[2] + first
    b = bq.kv_batch(batch.dev[0], batch.dev[1], moved, batch.tokens, batch.max_q, batch.max_kv)
    size = bq.bq_kv_attention_workspace_bytes(cache, b, bq.BQ_F16, 8)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
    out = torch.empty_like(q)
    bq.check(bq.bq_kv_attention(cache, b, bq.BQ_F16, q, q.stride(0), 8, 0.06, 1, 0, out, out.stride(0), None, ws, size))
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dim,B,bits", [(64, 32, 4), (128, 128, 8), (256, 64, 4)])
@pytest.mark.parametrize("lens,window", [([(1, 200), (3, 150)], 70), ([(90, 300), (70, 110), (2, 90)], 37),
                                         ([(210, 500)], 100), ([(300, 700), (20, 110), (2, 90)], 37)],
                         ids=["few", "many", "alone", "mixed"])
def test_keys_that_no_row_sees_may_be_nan(dev, lens, window, dim, B, bits):
    """Behind the window (within a page and a tile that later keys share) the cache holds NaN maxima."""
    rng, pool, batch = setup(dev, 21, lens, 4, 2, dim, B, 32, bits)
    for s, (n, kv) in enumerate(lens):
        j = np.arange(max(0, kv - n - window + 1))
        page, slot = torch.from_numpy(batch.table[s, j // 32]).long().to(dev), torch.from_numpy(j % 32).to(dev)
        for side in range(2):
            pool.absmax[side].view(pool.num_pages, 2, 32, dim // B)[page, :, slot] = float("nan")
    q = queries(dev, rng, batch.tokens, 4, dim, "bfloat16")
    check_attention(dev, pool, batch, q, "bfloat16", 0.09, 1, window)


@pytest.mark.parametrize("lens", [[(1, 130)], [(5, 3000)], [(2, 40), (110, 400)], [(100, 5000)]],
                         ids=["one", "splits", "mixed", "chunk splits"])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_queries_that_are_not_finite(dev, lens, bad):
    """A query that is not finite makes its own result NaN and no other."""
    rng, pool, batch = setup(dev, 22, lens, 8, 2, 128, 64, 16, 4)
    q = queries(dev, rng, batch.tokens, 8, 128, "bfloat16")
    want, want_lse, tol, tol_lse = reference(pool, batch, q, "bfloat16", 0.09)
    rows = [(batch.tokens - 1, 3), (0, 6)]
    for token, head in rows:
        q[token, head, 5 + head] = float(bad)
    out, lse = run_attention(dev, pool, batch, q, "bfloat16", 0.09)
    torch.cuda.synchronize()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for token, head in rows:
        assert np.isnan(out[token, head]).all()
        assert bad != "nan" or np.isnan(lse[token, head])
        out[token, head], lse[token, head] = want[token, head], want_lse[token, head]
    assert (np.abs(out - want) <= tol).all() and (np.abs(lse - want_lse) <= tol_lse).all()


@pytest.mark.parametrize("seed", range(24))
def test_mixed_sizes(dev, seed):
    """Heads, head sizes, pages, blocks and batches of single tokens, drafts and chunks, drawn."""
    rng = np.random.default_rng(1000 + seed)
    dim, B = SHAPES[rng.integers(len(SHAPES))]
    kv_heads, group = int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 5, 8]))
    lens = []
    for _ in range(rng.integers(1, 6)):
        n = int(rng.choice([0, 1, 1, 4, 37, 400]))
        lens.append((n, n + int(rng.choice([0, 3, 100, 800, 2500]))))
    lens.append((int(rng.choice([1, 3, 70])), int(rng.integers(70, 1500))))
    window = int(rng.choice([0, 0, 50, 700]))
    dtype = "float16" if rng.integers(2) else "bfloat16"
    rng, pool, batch = setup(dev, seed, lens, group * kv_heads, kv_heads, dim, B, int(rng.choice([16, 32, 128])),
                             int(rng.choice([4, 8])))
    q = queries(dev, rng, batch.tokens, group * kv_heads, dim, dtype)
    check_attention(dev, pool, batch, q, dtype, dim ** -0.5, int(seed % 5 != 0), window, tag=str(lens))
