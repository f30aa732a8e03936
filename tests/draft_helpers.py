"""Helpers of the tests of drafted tokens over the cache: rotation and quantization in binary32 on the host, trees, and
attention of a tree in binary64 from the definition, with a bound on what a kernel's roundings can change."""
from __future__ import annotations

import numpy as np
import torch

import dequantization_block_absmax_amd as bq
from gpu_helpers import BQ_DT, TORCH_DT

# What one rounding to the type can change, relative to the value: half a step.
HALF_STEP = {name: torch.finfo(t).eps / 2 for name, t in TORCH_DT.items()}


# ---- rotation ------------------------------------------------------------------------------

def angles(positions, rotary_dim, base=10000.0):
    """Tables of cosines and sines in binary32, positions x rotary_dim / 2."""
    a = np.arange(positions)[:, None] * base ** (-2.0 * np.arange(rotary_dim // 2) / rotary_dim)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def rotated(x, cos, sin, positions, rotary_dim, interleaved):
    """x (tokens, heads, head_dim) in binary32, each operation rounded once (numpy's binary32 arithmetic)."""
    x = np.asarray(x, np.float32)
    half = rotary_dim // 2
    first = np.arange(0, rotary_dim, 2) if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    c, s = cos[positions, :half][:, None], sin[positions, :half][:, None]
    a, b = x[..., first], x[..., second]
    out = x.copy()
    with np.errstate(all="ignore"):
        out[..., first] = a * c - b * s
        out[..., second] = b * c + a * s
    return out


# ---- trees ---------------------------------------------------------------------------------

def random_tree(rng, n, unused=0.0):
    """Parents of n tokens: each follows the context or any token before it; a part of them are unused places."""
    parents = [int(rng.integers(-1, i)) if i else -1 for i in range(n)]
    for i in range(n):
        if rng.random() < unused:
            parents[i] = int(rng.choice([-2, i, i + 1, n, 2 ** 31 - 1, -2 ** 31, 70000]))
    return parents


def chains(parents):
    """For each token the numbers of itself and its ancestors, nearest first, or None where it sees nothing."""
    out = []
    for i in range(len(parents)):
        chain, at = [i], i
        while True:
            up = parents[at]
            if up == -1:
                break
            if not 0 <= up < at:
                chain = None
                break
            chain.append(up)
            at = up
        out.append(chain)
    return out


def seen_by(parents, kv, window):
    """Which of kv keys each of the last len(parents) tokens sees: (tokens, keys), and the tokens' depths."""
    n = len(parents)
    seen = np.zeros((n, kv), bool)
    for i, chain in enumerate(chains(parents)):
        if chain is None:
            continue
        pos = kv - n + len(chain) - 1
        low = pos - window + 1 if window else -n
        seen[i, max(0, low):max(0, kv - n)] = True
        for c in chain[:window or None]:
            if kv - n + c >= 0:
                seen[i, kv - n + c] = True
    return seen


def reference(pool, batch, parents, q, dtype, scale, window=0, rows=None):
    """(out, lse, tolerance of out, tolerance of lse) in binary64; rows of no sequence hold 77.

    Keys, queries, values and weights may each be rounded once to binary16 on the way (2^-11 relative), products are
    summed in binary32.  A logit s = scale * sum q k then moves by at most e = (2 2^-11 + (D + 16) 2^-24) * scale *
    sum |q k|, each probability by the factor exp(2 e), and out by (exp(2 e) - 1 + 3 2^-11 + (n + D) 2^-24) sum p |v|,
    plus n times the smallest step of a weight in binary16 (2^-25) times the largest |v|, plus the result's rounding.
    lse is the sum of weights that are not rounded: it moves by e, and by binary32's roundings."""
    h, d, ps = pool.kv_heads, pool.head_dim, pool.page_size
    k_all, v_all = pool.values(0), pool.values(1)
    qs = q.float().cpu().numpy().astype(np.float64)
    heads = qs.shape[1]
    group = heads // h
    w, last = 2.0 ** -11, HALF_STEP[dtype]
    out = np.full(qs.shape, 77.0)
    lse = np.full(qs.shape[:2], 77.0)
    tol, tol_lse = np.zeros(qs.shape), np.zeros(qs.shape[:2])
    for s, (n, kv) in enumerate(batch.lens):
        if n == 0:
            continue
        at = slice(batch.starts[s], batch.starts[s] + min(n, batch.max_q))
        j = np.arange(kv)
        page = batch.table[s, j // ps]
        listed = (page >= 0) & (page < pool.num_pages)
        page = np.where(listed, page, 0)
        seen = seen_by(parents[batch.starts[s]:batch.starts[s] + n], kv, window)[:at.stop - at.start] & listed
        some = seen.any(1)
        for head in range(heads):
            k = np.nan_to_num(k_all[page, head // group, j % ps])
            v = np.nan_to_num(v_all[page, head // group, j % ps])
            qh = qs[at, head]
            z = np.where(seen, scale * (qh @ k.T), -np.inf)
            top = np.where(some, z.max(1, initial=-np.inf), 0.0)
            e = np.exp(z - top[:, None])
            total = e.sum(1)
            p = e / np.where(some, total, 1.0)[:, None]
            out[at, head] = p @ v
            with np.errstate(divide="ignore"):
                lse[at, head] = np.where(some, top + np.log(total), -np.inf)
            slack = (2 * w + (d + 16) * 2.0 ** -24) * abs(scale) * np.where(seen, np.abs(qh) @ np.abs(k).T, 0.0)
            slack = slack.max(1, initial=0.0)
            vmax = np.where(seen.any(0)[:, None], np.abs(v), 0.0).max(initial=0.0)
            bound = (np.expm1(2 * slack) + 3 * w + (kv + d) * 2.0 ** -24)[:, None] * (p @ np.abs(v))
            tol[at, head] = bound + kv * 2.0 ** -25 * vmax + last * (np.abs(out[at, head]) + bound) + 2.0 ** -25
            tol_lse[at, head] = slack + 2.0 ** -20 * (1 + np.abs(np.where(some, lse[at, head], 0.0)))
    return out, lse, tol, tol_lse


def run_tree(dev, pool, batch, parents, q, dtype, scale, window=0, with_lse=True, stream=None):
    """q: (tokens, heads, head_dim) of dtype on the device (rows may be strided)."""
    heads = q.shape[1]
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device=dev)
    lse = torch.full(q.shape[:2], 77.0, dtype=torch.float32, device=dev) if with_lse else None
    size = bq.bq_kv_tree_attention_workspace_bytes(pool.cache, batch.batch, BQ_DT[dtype], heads)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device=dev)  # NaNs, whatever type is read
    par = torch.tensor(parents if parents else [0], dtype=torch.int64).to(torch.int32).to(dev)
    bq.check(bq.bq_kv_tree_attention(pool.cache, batch.batch, par, BQ_DT[dtype], q, q.stride(0), heads, scale, window,
                                     out, out.stride(0), lse, ws, size, stream), "tree attention")
    return out, lse


def compare(got, got_lse, want, want_lse, tol, tol_lse, tag=""):
    most = torch.finfo(got.dtype).max
    got, got_lse = got.double().cpu().numpy(), got_lse.double().cpu().numpy()
    # Where the exact result may lie past the type's largest number, rounding to the type gives infinity.
    past = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + tol >= most)
    bad = np.argwhere(~(np.where(past, 0.0, np.abs(got - want)) <= tol))
    assert bad.size == 0, (tag, len(bad), [(b.tolist(), got[tuple(b)], want[tuple(b)], tol[tuple(b)]) for b in bad[:4]])
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty), tag
    diff = np.abs(np.where(empty, 0.0, got_lse) - np.where(empty, 0.0, want_lse))
    bad = np.argwhere(~(diff <= tol_lse))
    assert bad.size == 0, (tag, "lse", [(b.tolist(), got_lse[tuple(b)], want_lse[tuple(b)], tol_lse[tuple(b)])
                                        for b in bad[:4]])


def check_tree(dev, pool, batch, parents, q, dtype, scale, window=0, tag="", stream=None):
    out, lse = run_tree(dev, pool, batch, parents, q, dtype, scale, window, stream=stream)
    torch.cuda.synchronize()
    compare(out, lse, *reference(pool, batch, parents, q, dtype, scale, window), tag)
    return out, lse
