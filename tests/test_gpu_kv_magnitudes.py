"""bq_kv_attention where the sizes of cached keys and values differ from token to token, against binary64
sums within a bound that is relative to what the row itself adds up.

The cache is made of numbers that binary16 holds exactly (table entries of 4 or 8 bits, block maxima that are
powers of two, queries of a few bits), so that of the kernels' roundings only these are left:

  scores    binary32: a few roundings of numbers up to |z|, the row's largest score and an exponent of at
            most 128, together d_j = 2^-20 (|z_j| + |z_max|) + 2^-14 in the exponent of a weight
  weights   binary16, u = 2^-11 of each, and never less than 2^-25 of their unit; the unit is at least
            2^-3 times the row's largest weight times the largest value of its 64 keys, whose exponents
            differ by at most 4 (one bit more for the exponent itself): 2^-23 max_j p_j a_j for each key
  sums      binary32 over n keys: n 2^-24 of the sum of magnitudes
  result    one rounding of the type

The sum of the weights is rounded, or not, on its own: the same relative terms again, times the result."""
import numpy as np
import pytest
import torch

import synth
from kv_helpers import Batch, Pool, run_attention
from gpu_helpers import TORCH_DT

pytestmark = pytest.mark.gpu

RESULT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
SCALE, LEAD = 0.125, 16.0  # the first element of every query: a key's score is 2 * its own first element, and a bit


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    return torch.device("cuda:0")


def strength(target):
    """Sixteenths m and exponent e with 2 * (m / 16) * 2^e next to target, -16 <= m <= 14 and even (the
    entries of both tables)."""
    e = np.ceil(np.log2(np.maximum(np.abs(target), 2.0 ** -3) / 2 * 16 / 14)).astype(int)
    return 2 * np.rint(target / 4 * 16 / 2.0 ** e).astype(int), e


def put(pool, table_row, side, codes, maxima):
    """One sequence's codes (key, head, d) and block maxima (key, head, block) into its pages."""
    n, ps = len(codes), pool.page_size
    page, slot = torch.from_numpy(table_row[np.arange(n) // ps]).long(), torch.arange(n) % ps
    if pool.bits == 4:
        codes = codes[..., 0::2] << 4 | codes[..., 1::2]
    shape = (pool.num_pages, pool.kv_heads, ps, -1)
    dev = pool.packed[side].device
    pool.packed[side].view(shape)[page, :, slot] = torch.from_numpy(codes.astype(np.uint8)).to(dev)
    pool.absmax[side].view(shape)[page, :, slot] = torch.from_numpy(maxima.astype(np.float32)).to(dev)


def make(dev, seed, lens, plan, dim, B, bits, kv_heads=1, ps=32):
    """Pool and batch whose sequences hold keys and values after plan(rng, keys) -> (scores, exponents of the
    values; -inf: zeros)."""
    rng = np.random.default_rng(seed)
    size = 1 << bits
    pool = Pool(dev, synth.dyadic_table(size), sum(-(-kv // ps) for _, kv in lens) + 2, ps, kv_heads, dim, B)
    batch = Batch(dev, pool, lens, rng)
    for s, (_, kv) in enumerate(lens):
        if kv == 0:
            continue
        target, vexp = plan(rng, kv)
        m, e = strength(np.asarray(target, float))
        codes = np.full((kv, kv_heads, dim), size // 2)
        codes[:, :, 0] += (m * size // 32)[:, None]
        codes[:, :, B:] = rng.integers(0, size, (kv, kv_heads, dim - B))
        maxima = np.ones((kv, kv_heads, dim // B))
        maxima[:, :, 0] = np.exp2(e)[:, None]
        put(pool, batch.table[s], 0, codes, maxima)
        maxima = np.exp2(np.asarray(vexp, float)[:, None, None] - rng.integers(0, 2, (kv, kv_heads, dim // B)))
        # more positive values than negative ones: what many small weights add up to is not lost in the average
        put(pool, batch.table[s], 1, rng.integers(size // 4, size, (kv, kv_heads, dim)), maxima)
    return rng, pool, batch


def exact_queries(dev, rng, tokens, heads, dim, dtype):
    q = rng.integers(-4, 5, (tokens, heads, dim)) / 4.0
    q[:, :, 0] = LEAD
    return torch.from_numpy(q).to(TORCH_DT[dtype]).to(dev)


def bound(pool, batch, q, dtype, window, step=1):
    """(out, lse, tolerance of out, tolerance of lse) of every step-th row, see above."""
    k_all, v_all = pool.values(0), pool.values(1)
    a_all = pool.absmax[1].double().cpu().numpy().reshape(pool.num_pages, pool.kv_heads, pool.page_size, -1).max(-1)
    qs = q.double().cpu().numpy()
    heads, group, ps = qs.shape[1], qs.shape[1] // pool.kv_heads, pool.page_size
    out, lse, tol, tol_lse = (np.zeros(s) for s in (qs.shape, qs.shape[:2], qs.shape, qs.shape[:2]))
    for s, (n, kv) in enumerate(batch.lens):
        if n == 0:
            continue
        rows = slice(batch.starts[s], batch.starts[s] + n, step)
        j = np.arange(kv)
        page = batch.table[s, j // ps]
        t = kv - n + np.arange(n)[::step, None]
        seen = (j <= t) & ((j > t - window) if window else True)
        for head in range(heads):
            k, v, a = (x[page, head // group, j % ps] for x in (k_all, v_all, a_all))
            z = np.where(seen, SCALE * (qs[rows, head] @ k.T), -np.inf)
            top = z.max(1, keepdims=True)
            p = np.exp(z - top)
            total = p.sum(1, keepdims=True)
            p /= total
            o = p @ v
            d = np.minimum(2.0 ** -20 * (np.abs(np.where(seen, z, 0.0)) + np.abs(top)) + 2.0 ** -14, 1.0)
            u = 2.0 ** -11 + 2 * kv * 2.0 ** -24
            floor = kv * 2.0 ** -23 * (p * a).max(1, keepdims=True)
            err = (p * (d + u)) @ np.abs(v) + floor + np.abs(o) * ((p * (d + u)).sum(1, keepdims=True) + kv * 2.0 ** -23)
            out[rows, head], lse[rows, head] = o, (top + np.log(total))[:, 0]
            tol[rows, head] = err + RESULT[dtype] * (np.abs(o) + err) + (2.0 ** -25 if dtype == "float16" else 0.0)
            tol_lse[rows, head] = (p * d).sum(1) + kv * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(lse[rows, head]))
    return tuple(x[::step] for x in (out, lse, tol, tol_lse))


def check(dev, pool, batch, q, dtype, window=0, step=1):
    want, want_lse, tol, tol_lse = bound(pool, batch, q, dtype, window, step)
    for with_lse in (True, False):
        out, lse = run_attention(dev, pool, batch, q, dtype, SCALE, 1, window, with_lse)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()[::step]
        if dtype == "float16":  # a result beyond the type is an infinity
            got, want = (np.clip(x, -65504.0, 65504.0) for x in (got, want))
        over = np.abs(got - want) / tol
        at = np.unravel_index(np.argmax(np.where(np.isnan(over), np.inf, over)), over.shape)
        assert (over <= 1).all(), ("lse" if with_lse else "no lse", at, got[at], want[at], tol[at],
                                   np.linalg.norm(got - want) / np.linalg.norm(want))
        if with_lse:
            assert (np.abs(lse.double().cpu().numpy()[::step] - want_lse) <= tol_lse).all()


def mild(rng, n):
    return rng.integers(-4, 5, n) / 4.0


def spikes(k):
    """A few single tokens with values 2^k times the others', which weigh e^-56."""
    def plan(rng, n):
        t, x = mild(rng, n), np.zeros(n)
        at = rng.choice(n, 5, replace=False)
        t[at], x[at] = -56.0, k
        return t, x
    return plan


def heavy_spikes(k):
    """Values 2^k times the others' on tokens that weigh about 2^-k: both matter."""
    def plan(rng, n):
        t, x = mild(rng, n), np.zeros(n)
        at = rng.choice(n, 5, replace=False)
        t[at], x[at] = -k * np.log(2.0), k
        return t, x
    return plan


def first_tile(k):
    def plan(rng, n):
        t, x = mild(rng, n), np.zeros(n)
        t[:64], x[:64] = -56.0, k
        return t, x
    return plan


def steps(up, slope):
    """Values that grow (or shrink) by 2^6 from tile to tile, scores that take `slope` of it back."""
    def plan(rng, n):
        x = 6.0 * (np.arange(n) // 64 % 10)
        x = x if up else 54 - x
        return mild(rng, n) - slope * x, x - 20
    return plan


def sink(gain, k):
    """The first key takes most of the weight; its values are 2^k, the others' a half. The others weigh
    (nearly) the same, so that what is rounded off each of them adds up."""
    def plan(rng, n):
        t, x = np.zeros(n), np.full(n, -1.0)
        t[0], x[0] = gain, k
        return t, x
    return plan


def small(k, large):
    """Values of 2^k, every other key's 2^large with a weight that much smaller."""
    def plan(rng, n):
        t, x = mild(rng, n), np.full(n, float(k))
        t[1::2], x[1::2] = t[1::2] - (large - k) * np.log(2.0), large
        return t, x
    return plan


def zeros_beside(k, first):
    """Half of the keys hold zeros and weigh e^6 times as much as the other half, whose values are 2^k: they
    count in the denominator only."""
    def plan(rng, n):
        t, x = mild(rng, n), np.full(n, float(k))
        at = np.arange(n) < n // 2 if first else np.arange(n) >= n // 2
        t[at], x[at] = t[at] + 6.0, -np.inf
        return t, x
    return plan


def key_spikes(k):
    """Single keys of 2^k, whose scores are far below all others."""
    def plan(rng, n):
        t = mild(rng, n)
        t[rng.choice(n, 5, replace=False)] = -2.0 ** (k + 1)
        return t, np.zeros(n)
    return plan


PLANS = {
    "spikes 9": (700, spikes(9)), "spikes 24": (700, spikes(24)), "spikes 40": (700, spikes(40)),
    "heavy spikes 9": (700, heavy_spikes(9)), "heavy spikes 40": (700, heavy_spikes(40)),
    "first tile 16": (700, first_tile(16)), "first tile 24": (700, first_tile(24)),
    "first tile 40": (700, first_tile(40)), "up": (700, steps(True, 0.0)), "down": (700, steps(False, 0.0)),
    "up, level": (700, steps(True, np.log(2.0))), "down, level": (700, steps(False, np.log(2.0))),
    "small": (700, small(-78, -78)), "small beside large": (700, small(-78, 0)), "small beside 2^99": (700, small(-78, 99)),
    "zeros, then 20": (700, zeros_beside(20, True)), "zeros, then 60": (700, zeros_beside(60, True)),
    "zeros, then 99": (700, zeros_beside(99, True)), "60, then zeros": (700, zeros_beside(60, False)),
    "99, then zeros": (5000, zeros_beside(99, False)), "zeros, then 99, long": (5000, zeros_beside(99, True)),
    "key spikes 12": (700, key_spikes(12)),
    "key spikes 24": (700, key_spikes(24)), "key spikes 40": (700, key_spikes(40)),
}
ROWS = {"one": 1, "few": 9, "many": 200}


@pytest.mark.parametrize("dim,B,bits,dtype", [(64, 32, 4, "bfloat16"), (64, 64, 8, "float16"), (128, 64, 4, "float16"),
                                              (128, 128, 4, "bfloat16"), (256, 64, 8, "bfloat16")])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("name", PLANS)
def test_values_of_every_size(dev, name, rows, dim, B, bits, dtype):
    n, plan = PLANS[name]
    rng, pool, batch = make(dev, 31, [(ROWS[rows], n)], plan, dim, B, bits)
    check(dev, pool, batch, exact_queries(dev, rng, batch.tokens, 4, dim, dtype), dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("name", ["spikes 9", "spikes 40", "first tile 24", "key spikes 40"])
@pytest.mark.parametrize("window", [0, 150, 400])
def test_sequences_of_both_kinds(dev, window, name, dtype):
    """Long pieces, single tokens and drafts in one call, two key/value heads; a window that hides the large
    values from the later rows."""
    plan = PLANS[name][1]
    rng, pool, batch = make(dev, 32, [(230, 500), (1, 700), (0, 0), (300, 300), (6, 90)], plan, 64, 32, 4, kv_heads=2)
    check(dev, pool, batch, exact_queries(dev, rng, batch.tokens, 4, 64, dtype), dtype, window)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("gain,k", [(12.0, 0.0), (16.0, -10.0), (12.0, 9.0)])
@pytest.mark.parametrize("rows", [1, 2900])
def test_a_first_key_before_many(dev, rows, gain, k, dtype):
    """16384 keys under one that takes most of the weight: as large as they are, much smaller, much larger.
    So many rows that their keys are not split."""
    rng, pool, batch = make(dev, 33, [(rows, 16384)], sink(gain, k), 64, 64, 8, kv_heads=8)
    check(dev, pool, batch, exact_queries(dev, rng, batch.tokens, 32, 64, dtype), dtype, step=-(-rows // 6))
