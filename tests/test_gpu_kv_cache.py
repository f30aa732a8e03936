"""bq_kv_write and bq_kv_read against the oracle's quantize and dequantize, bit for bit: a block
lies in one token's head, so the codes and maxima of a token are those of its rows quantized as
a flat array, and only where they are put is new."""
import numpy as np
import pytest
import torch

import dequantization_block_absmax_amd as bq
import oracle
import synth
from gpu_helpers import BQ_DT, ORACLE_DT, TORCH_DT, assert_bytes_equal, assert_f32_bits_equal, host_bits
from kv_helpers import Pool

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "float16", "bfloat16"]
CLUSTERED = np.float32(np.sort(np.concatenate([np.linspace(-1, 0.45, 56), 0.5 + np.arange(200) * 2.0**-23 * 8])))
TABLES = {
    "t16": synth.table16(), "t256": synth.table256(), "even256": np.linspace(-1, 1, 256).astype(np.float32),
    "clustered256": CLUSTERED,  # takes the binary search
    "tiny16": np.float32(np.sort(np.concatenate([[-1, 0, 1, 2.0**-20, -2.0**-20, 2.0**-19],
                                                 np.linspace(0.1, 0.9, 10)]))),
}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def o():
    return oracle.Oracle()


def rows(rng, tokens, heads, dim, dtype, special=True):
    x = rng.standard_normal((tokens, heads, dim)).astype(np.float32)
    if special and tokens * heads * dim >= 64:
        f = x.reshape(-1)
        f[rng.integers(0, f.size, max(1, f.size // 60))] = np.nan
        f[rng.integers(0, f.size, max(1, f.size // 60))] = np.inf
        f[rng.integers(0, f.size, max(1, f.size // 60))] = -np.inf
        x[rng.integers(0, tokens), 0] = 0.0                       # zero blocks
        x[rng.integers(0, tokens), heads - 1] = np.nan             # a block with nothing finite
        x[rng.integers(0, tokens), 0] *= np.float32(1e-30)         # the power-of-two guards (binary32, bf16)
        x[rng.integers(0, tokens), heads - 1] *= np.float32(1e25)
    return torch.from_numpy(x).to(TORCH_DT[dtype])


def expected(o, pool, side, x, dtype, slots):
    """The pool's bytes after the write, from the oracle's codes of the rows."""
    packed, absmax = pool.packed[side].cpu().numpy().copy(), pool.absmax[side].cpu().numpy().copy()
    T, H, D, ps = x.shape[0], pool.kv_heads, pool.head_dim, pool.page_size
    a, p = o.quantize_blockwise(host_bits(x.contiguous()).reshape(-1), ORACLE_DT[dtype], pool.blocksize, pool.table)
    a, p = a.reshape(T, H, -1), p.reshape(T, H, -1)
    pv = packed.reshape(pool.num_pages, H, ps, -1)
    av = absmax.reshape(pool.num_pages, H, ps, -1)
    for t, s in enumerate(slots):
        if 0 <= s < pool.num_pages * ps:
            pv[s // ps, :, s % ps] = p[t]
            av[s // ps, :, s % ps] = a[t]
    return packed, absmax


CASES = [  # heads, head_dim, blocksize, page_size, tokens, table
    (1, 32, 32, 16, 1, "t16"), (3, 64, 32, 16, 37, "t16"), (5, 96, 32, 32, 19, "t256"), (8, 128, 64, 16, 50, "t16"),
    (2, 128, 128, 64, 131, "even256"), (1, 256, 256, 128, 77, "t256"), (7, 224, 32, 16, 9, "clustered256"),
    (4, 192, 64, 4096, 23, "tiny16"), (2, 160, 32, 16, 40, "tiny16"), (8, 128, 32, 32, 1030, "even256"),
    (6, 256, 128, 16, 2049, "t16"),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "h%d_d%d_b%d_p%d_t%d_%s" % c)
def test_write_and_read(dev, o, case, dtype):
    heads, dim, B, ps, tokens, name = case
    rng = np.random.default_rng(dim * 7 + tokens)
    pool = Pool(dev, TABLES[name], -(-tokens // ps) + 2, ps, heads, dim, B)
    total = pool.num_pages * ps
    slots = rng.permutation(total)[:tokens].astype(np.int64)
    if tokens > 8:  # slots outside the pool are skipped
        slots[1], slots[3], slots[5], slots[7] = -1, total, -(2 ** 40), 2 ** 40
    pad = 16 if dtype == "float32" else 32  # keys and values as parts of a wider row
    wide = torch.zeros(tokens, 2, heads * dim + pad, dtype=TORCH_DT[dtype])
    k, v = (rows(rng, tokens, heads, dim, dtype) for _ in range(2))
    wide[:, 0, :heads * dim], wide[:, 1, :heads * dim] = k.reshape(tokens, -1), v.reshape(tokens, -1)
    wide = wide.to(dev)
    want = [expected(o, pool, i, x, dtype, slots) for i, x in enumerate((k, v))]
    sd = torch.from_numpy(slots).to(dev)
    stride = wide.stride(0)
    bq.check(bq.bq_kv_write(pool.cache, BQ_DT[dtype], wide[:, 0], wide[:, 1], tokens, stride, stride, sd), "write")
    torch.cuda.synchronize()
    for i in range(2):
        assert_bytes_equal(pool.packed[i].cpu().numpy(), want[i][0], "codes %d" % i)
        assert_f32_bits_equal(pool.absmax[i].cpu().numpy(), want[i][1], "absmax %d" % i)

    # read back: other order, repeats, and rows of another stride and other types
    back = np.concatenate([slots, slots[:3], [-5, total]])
    bd = torch.from_numpy(back).to(dev)
    for out_dtype in DTYPES:
        out = [torch.full((len(back), heads * dim + pad), 7.0, dtype=TORCH_DT[out_dtype], device=dev) for _ in range(2)]
        bq.check(bq.bq_kv_read(pool.cache, BQ_DT[out_dtype], out[0], out[1], len(back), out[0].stride(0),
                               out[1].stride(0), bd), "read")
        torch.cuda.synchronize()
        for i in range(2):
            full = o.dequantize_blockwise(want[i][0], want[i][1], pool.elems, ORACLE_DT[out_dtype], B, pool.table)
            full = full.reshape(pool.num_pages, heads, ps, dim)
            ref = np.zeros((len(back), heads, dim), full.dtype)
            for t, s in enumerate(back):
                if 0 <= s < total:
                    ref[t] = full[s // ps, :, s % ps]
            got = host_bits(out[i][:, :heads * dim].contiguous()).reshape(ref.shape)
            if out_dtype == "float32":
                assert_f32_bits_equal(got, ref, "read %d" % i)
            else:
                assert_bytes_equal(got, ref, "read %d %s" % (i, out_dtype))
            assert bool((out[i][:, heads * dim:] == 7.0).all())


def test_large_write_takes_the_tiled_form(dev, o):
    """Enough units for four per lane, a ragged last tile; sampled tokens against the oracle."""
    rng = np.random.default_rng(5)
    heads, dim, B, ps, tokens = 8, 128, 64, 64, 9001
    pool = Pool(dev, TABLES["t16"], -(-tokens // ps), ps, heads, dim, B)
    slots = rng.permutation(pool.num_pages * ps)[:tokens].astype(np.int64)
    k, v = (rows(rng, tokens, heads, dim, "bfloat16", special=False) for _ in range(2))
    sd = torch.from_numpy(slots).to(dev)
    bq.check(bq.bq_kv_write(pool.cache, bq.BQ_BF16, k.to(dev), v.to(dev), tokens, heads * dim, heads * dim, sd), "write")
    out = [torch.empty(tokens, heads * dim, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    bq.check(bq.bq_kv_read(pool.cache, bq.BQ_BF16, out[0], out[1], tokens, heads * dim, heads * dim, sd), "read")
    torch.cuda.synchronize()
    for i, x in enumerate((k, v)):
        a, p = o.quantize_blockwise(host_bits(x).reshape(-1), oracle.BF16, B, pool.table)
        want = o.dequantize_blockwise(p, a, x.numel(), oracle.BF16, B, pool.table)
        assert_bytes_equal(host_bits(out[i]).reshape(-1), want, "side %d" % i)
        av = pool.absmax[i].view(pool.num_pages, heads, ps, -1)[sd // ps, :, sd % ps]
        assert_f32_bits_equal(av.cpu().numpy().reshape(-1), a, "absmax %d" % i)


def test_pool_is_a_blockwise_array(dev):
    """bq_dequantize_blockwise expands the whole pool to what bq_kv_read gives slot by slot."""
    rng = np.random.default_rng(6)
    pool = Pool(dev, TABLES["t256"], 5, 32, 3, 64, 32)
    pool.fill(rng)
    total = 5 * 32
    flat = torch.empty(pool.elems, dtype=torch.float16, device=dev)
    bq.check(bq.bq_dequantize_blockwise(flat, bq.BQ_F16, pool.elems, 32, pool.table, pool.absmax[1], pool.packed[1]))
    sd = torch.arange(total, device=dev)
    k, v = (torch.empty(total, 3 * 64, dtype=torch.float16, device=dev) for _ in range(2))
    bq.check(bq.bq_kv_read(pool.cache, bq.BQ_F16, k, v, total, 192, 192, sd))
    want = flat.view(5, 3, 32, 64).transpose(1, 2).reshape(total, 192)
    assert torch.equal(v.view(torch.int16), want.contiguous().view(torch.int16))


def test_offsets_beyond_32_bits(dev):
    """A pool of more than 2^32 bytes of codes: tokens written to its last page come back, and the page
    that a 32-bit offset would reach is left alone."""
    heads, dim, B, ps = 8, 256, 256, 64
    pages = (1 << 32) // (heads * dim * ps) + 40
    table = torch.from_numpy(TABLES["even256"]).to(dev)
    packed = [torch.zeros(pages * heads * ps * dim, dtype=torch.uint8, device=dev) for _ in range(2)]
    absmax = [torch.zeros(pages * heads * ps, dtype=torch.float32, device=dev) for _ in range(2)]
    cache = bq.kv_cache(packed[0], absmax[0], packed[1], absmax[1], TABLES["even256"], pages, ps, heads, dim, B)
    tokens = 70
    slots = torch.arange(pages * ps - tokens, pages * ps, device=dev)
    x = torch.randn(tokens, heads * dim, device=dev).to(torch.bfloat16)
    bq.check(bq.bq_kv_write(cache, bq.BQ_BF16, x, x, tokens, heads * dim, heads * dim, slots))
    k, v = (torch.empty_like(x) for _ in range(2))
    bq.check(bq.bq_kv_read(cache, bq.BQ_BF16, k, v, tokens, heads * dim, heads * dim, slots))
    torch.cuda.synchronize()
    a = x.float().view(tokens, heads, dim).abs().amax(-1, keepdim=True)
    y = x.float().view(tokens, heads, dim) * (1.0 / a)  # the normalize rule; midpoints are exact in binary64
    near = table[torch.bucketize(y.double(), (table[1:].double() + table[:-1].double()) / 2)]
    # half a step of the even table (1/255), the type's rounding, and the product's
    tol = a * (1 / 255 + 2.0 ** -20) + 2.0 ** -8 * a
    for got in (k, v):
        assert bool(((got.float().view(tokens, heads, dim) - near * a).abs() <= tol).all())
        assert bool(((got.float().view(tokens, heads, dim) - x.float().view(tokens, heads, dim)).abs() <= tol).all())
    wrapped = pages * ps * heads * dim - (1 << 32)
    for p in packed:
        assert int(p[:wrapped].count_nonzero()) == 0


def test_stream_and_graph(dev):
    """Write, read and attention captured in a graph on a stream of its own, replayed with new inputs
    each time and compared with the calls made eagerly."""
    from kv_helpers import Batch, queries, run_attention
    rng = np.random.default_rng(8)
    pool = Pool(dev, TABLES["t16"], 6, 16, 2, 64, 64)
    pool.fill(rng)
    batch = Batch(dev, pool, [(1, 33), (1, 17)], rng)
    slots = torch.tensor([int(batch.table[0, 2]) * 16, int(batch.table[1, 1]) * 16], device=dev)
    x = torch.zeros(2, 128, dtype=torch.bfloat16, device=dev)
    q = queries(dev, rng, 2, 8, 64, "bfloat16")
    k, v, out = torch.empty_like(x), torch.empty_like(x), torch.empty_like(q)
    size = bq.bq_kv_attention_workspace_bytes(pool.cache, batch.batch, bq.BQ_BF16, 8)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)

    def step(stream):
        bq.check(bq.bq_kv_write(pool.cache, bq.BQ_BF16, x, x, 2, 128, 128, slots, stream))
        bq.check(bq.bq_kv_read(pool.cache, bq.BQ_BF16, k, v, 2, 128, 128, slots, stream))
        bq.check(bq.bq_kv_attention(pool.cache, batch.batch, bq.BQ_BF16, q, 512, 8, 0.125, 1, 0, out, 512, None, ws, size,
                                    stream))

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for i in range(3):
        new = torch.from_numpy(rng.standard_normal((2, 128)).astype(np.float32)).to(torch.bfloat16).to(dev)
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (k, v, out, pool.packed[0], pool.absmax[1])]
        for t in (k, v, out):
            t.zero_()
        step(None)
        torch.cuda.synchronize()
        for a, b in zip(got, (k, v, out, pool.packed[0], pool.absmax[1])):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
