"""Helpers of the cache and attention tests: a pool on the device, and attention in binary64 from
the definition, with a bound on what a kernel's roundings can change."""
from __future__ import annotations

import numpy as np
import torch

import dequantization_block_absmax_amd as bq
from gpu_helpers import BQ_DT, TORCH_DT

# Half a unit in the last place, relative: what one rounding to the type can change.
UNIT = {"float16": 2.0 ** -12, "bfloat16": 2.0 ** -9}


class Pool:
    """A cache on `dev`, every byte of it set to a pattern before anything is written."""

    def __init__(self, dev, table, num_pages, page_size, kv_heads, head_dim, blocksize):
        self.table = np.float32(table)
        self.bits = 4 if len(table) == 16 else 8
        self.num_pages, self.page_size, self.kv_heads = num_pages, page_size, kv_heads
        self.head_dim, self.blocksize = head_dim, blocksize
        self.elems = num_pages * kv_heads * page_size * head_dim
        self.packed = [torch.full((self.elems * self.bits // 8,), 0xA5, dtype=torch.uint8, device=dev)
                       for _ in range(2)]
        self.absmax = [torch.full((self.elems // blocksize,), float("nan"), dtype=torch.float32, device=dev)
                       for _ in range(2)]
        self.cache = bq.kv_cache(self.packed[0], self.absmax[0], self.packed[1], self.absmax[1], self.table,
                                 num_pages, page_size, kv_heads, head_dim, blocksize)

    def fill(self, rng, std=1.0):
        """Random codes, and block maxima spread over a few octaves, in every slot."""
        for i in range(2):
            codes = rng.integers(0, 256, self.packed[i].numel(), dtype=np.uint8)
            self.packed[i].copy_(torch.from_numpy(codes))
            a = (std * np.exp(0.4 * rng.standard_normal(self.absmax[i].numel()))).astype(np.float32)
            self.absmax[i].copy_(torch.from_numpy(a))

    def values(self, side):
        """All of a side in binary64, (page, head, slot, d)."""
        p = self.packed[side].cpu().numpy()
        q = p if self.bits == 8 else np.stack((p >> 4, p & 15), -1).reshape(-1)
        v = self.table[q].astype(np.float64).reshape(-1, self.blocksize)
        v = v * self.absmax[side].cpu().numpy().astype(np.float64)[:, None]
        return v.reshape(self.num_pages, self.kv_heads, self.page_size, self.head_dim)


class Batch:
    """Sequences of (new tokens, keys) on pages of a pool, the pages in random order."""

    def __init__(self, dev, pool, lens, rng, max_q_len=None, max_kv_len=None):
        self.lens = lens
        need = [-(-kv // pool.page_size) for _, kv in lens]
        assert sum(need) <= pool.num_pages
        order = rng.permutation(pool.num_pages)
        self.table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.starts = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
        self.tokens = int(self.starts[-1])
        self.dev = [torch.from_numpy(a).to(dev) for a in
                    (self.starts, np.array([kv for _, kv in lens], np.int32), self.table)]
        self.max_q = max(q for q, _ in lens) if max_q_len is None else max_q_len
        self.max_kv = max(kv for _, kv in lens) if max_kv_len is None else max_kv_len
        self.batch = bq.kv_batch(*self.dev, self.tokens, self.max_q, self.max_kv)


def hide_unused(pool, batch):
    """NaN block maxima in every slot that no sequence's keys are in."""
    used = np.zeros((pool.num_pages, pool.page_size), bool)
    for s, (_, kv) in enumerate(batch.lens):
        j = np.arange(kv)
        used[batch.table[s, j // pool.page_size], j % pool.page_size] = True
    keep = torch.from_numpy(used).to(pool.absmax[0].device)[:, None, :, None]
    for side in range(2):
        a = pool.absmax[side].view(pool.num_pages, pool.kv_heads, pool.page_size, -1)
        a.copy_(torch.where(keep, a, torch.full_like(a, float("nan"))))


def run_attention(dev, pool, batch, q, dtype, scale, causal=1, window=0, with_lse=True, stream=None):
    """q: (tokens, heads, head_dim) of dtype on the device (rows may be strided)."""
    heads = q.shape[1]
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device=dev)
    lse = torch.full(q.shape[:2], 77.0, dtype=torch.float32, device=dev) if with_lse else None
    size = bq.bq_kv_attention_workspace_bytes(pool.cache, batch.batch, BQ_DT[dtype], heads)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device=dev)  # NaNs, whatever type is read
    bq.check(bq.bq_kv_attention(pool.cache, batch.batch, BQ_DT[dtype], q, q.stride(0), heads, scale, causal, window,
                                out, out.stride(0), lse, ws, size, stream), "attention")
    return out, lse


def reference(pool, batch, q, dtype, scale, causal=1, window=0):
    """(out, lse, tolerance of out, tolerance of lse) in binary64.

    With w one rounding of the type (relative): keys, queries and probabilities may each be rounded once
    to 16 bits, values too, products are summed in binary32.  A logit s = scale * sum q k then moves by
    at most e = (2 w + (D + 16) 2^-24) * scale * sum |q k|, each probability by the factor exp(2 e), and
    out by (exp(2 e) - 1 + 3 w + (n + D) 2^-24) sum p |v|, plus n times the smallest step of a
    probability in 16 bits (2^-25) times the largest |v|, plus the last rounding."""
    h, d, ps = pool.kv_heads, pool.head_dim, pool.page_size
    k_all, v_all = pool.values(0), pool.values(1)
    qs = q.float().cpu().numpy().astype(np.float64)
    heads = qs.shape[1]
    group = heads // h
    w = UNIT[dtype]
    out = np.full(qs.shape, 77.0)
    lse = np.full(qs.shape[:2], 77.0)
    tol, tol_lse = np.zeros(qs.shape), np.zeros(qs.shape[:2])
    for s, (n, kv) in enumerate(batch.lens):
        rows = slice(batch.starts[s], batch.starts[s] + n)
        j = np.arange(kv)
        page = batch.table[s, j // ps]
        listed = (page >= 0) & (page < pool.num_pages)
        page = np.where(listed, page, 0)
        t = kv - n + np.arange(n)
        seen = np.broadcast_to(listed, (n, kv)).copy()
        if causal:
            seen &= j <= t[:, None]
        if window:
            seen &= j > t[:, None] - window
        some = seen.any(1)
        for head in range(heads):
            k = np.nan_to_num(k_all[page, head // group, j % ps])
            v = np.nan_to_num(v_all[page, head // group, j % ps])
            qh = qs[rows, head]
            z = np.where(seen, scale * (qh @ k.T), -np.inf)
            top = np.where(some, z.max(1, initial=-np.inf), 0.0)
            e = np.exp(z - top[:, None])
            total = e.sum(1)
            p = e / np.where(some, total, 1.0)[:, None]
            out[rows, head] = p @ v
            with np.errstate(divide="ignore"):
                lse[rows, head] = np.where(some, top + np.log(total), -np.inf)
            slack = (2 * w + (d + 16) * 2.0 ** -24) * abs(scale) * np.where(seen, np.abs(qh) @ np.abs(k).T, 0.0)
            slack = slack.max(1, initial=0.0)
            vmax = np.where(seen.any(0)[:, None], np.abs(v), 0.0).max(initial=0.0)
            bound = (np.expm1(2 * slack) + 3 * w + (kv + d) * 2.0 ** -24)[:, None] * (p @ np.abs(v))
            tol[rows, head] = bound + kv * 2.0 ** -25 * vmax + w * (np.abs(out[rows, head]) + bound) + 2.0 ** -25
            tol_lse[rows, head] = slack + 2.0 ** -20 * (1 + np.abs(np.where(some, lse[rows, head], 0.0)))
    return out, lse, tol, tol_lse


def check_attention(dev, pool, batch, q, dtype, scale, causal=1, window=0, tag="", stream=None):
    out, lse = run_attention(dev, pool, batch, q, dtype, scale, causal, window, stream=stream)
    torch.cuda.synchronize()
    want, want_lse, tol, tol_lse = reference(pool, batch, q, dtype, scale, causal, window)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert bad.size == 0, (tag, len(bad), [(b.tolist(), got[tuple(b)], want[tuple(b)], tol[tuple(b)]) for b in bad[:4]])
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty), tag
    diff = np.abs(np.where(empty, 0.0, got_lse) - np.where(empty, 0.0, want_lse))
    bad = np.argwhere(~(diff <= tol_lse))
    assert bad.size == 0, (tag, "lse", [(b.tolist(), got_lse[tuple(b)], want_lse[tuple(b)], tol_lse[tuple(b)])
                                        for b in bad[:4]])
    return out, lse


def queries(dev, rng, tokens, heads, head_dim, dtype, std=1.0):
    q = torch.from_numpy((std * rng.standard_normal((max(tokens, 1), heads, head_dim))).astype(np.float32))
    return q.to(TORCH_DT[dtype]).to(dev)[:tokens] if tokens else q.to(TORCH_DT[dtype]).to(dev)
