"""Speculative decoding over the paged key/value cache in blockwise codes, as it is measured: new
tokens' keys (and queries) rotated to their positions on the way into the cache, attention of a
tree of drafted tokens over it, and the accepted path of the tree moved to the front of its draft.

The cache is that of perf/operators.py: element (page, head, slot, d) of a pool is flat element
((page * kv_heads + head) * page_size + slot) * head_dim + d of an array quantized blockwise, its
value table[code] * absmax[flat // blocksize]; 4-bit codes are two to a byte, the first of a pair
in the high nibble.

Rotation: with (c, s) the cosine and sine of a token's position for pair i of a head, the pair
(x, y) becomes (x c - y s, y c + x s), every product and sum rounded to 32 bits; pair i is elements
i and i + rotary_dim / 2, or elements 2 i and 2 i + 1 (interleaved).  Elements from rotary_dim on
stay.  Keys are quantized from the rotated 32-bit values, queries rounded once to their type.

Tree: new token i of a sequence's n has the parent parents[i] < i among them, or -1 (it follows the
context); any other number makes it, and what descends from it, see nothing.  It stands at position
kv_len - n + depth and sees the context and its ancestors and itself, within the window.

Accepted path: the new tokens path[0] < path[1] < ... become tokens kv_len - n + 0, 1, ...

`run` takes a state of `prepare` through one pass, in elementary torch operations where `own` is
false and through the library's entry points where it is true.
"""
import math
import random
import statistics

import torch

own = False

_DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
_POSITIONS = 32768  # rows of the tables of cosines and sines


# ---- cases ----------------------------------------------------------------------------------

def listed():
    return [
        # One decoding step of a serving batch, a token to a sequence: the smallest, all latency.
        dict(name="append_step", op="append", dtype="bfloat16", tokens=48, fresh=1, heads=32, kv_heads=8, head_dim=128,
             rotary_dim=128, interleaved=False, page_size=16, blocksize=64, bits=4),
        # A long prompt enters an 8-bit cache, one scale to a head.
        dict(name="append_prompt", op="append", dtype="bfloat16", tokens=16384, fresh=16384, heads=32, kv_heads=8,
             head_dim=128, rotary_dim=128, interleaved=False, page_size=64, blocksize=128, bits=8),
        # Ragged prompts of a smaller model kept in binary32, odd head counts, half of each head rotated in
        # neighbouring pairs.
        dict(name="append_ragged", op="append", dtype="float32", tokens=4099, fresh=333, heads=15, kv_heads=5,
             head_dim=64, rotary_dim=32, interleaved=True, page_size=32, blocksize=32, bits=4),
        # One user's draft after a short dialogue: the smallest attention, all latency.
        dict(name="tree_single", op="tree", dtype="bfloat16", seqs=1, nodes=26, kv_len=1026, lens=1, heads=32,
             kv_heads=8, head_dim=128, page_size=16, blocksize=64, bits=4, window=0),
        # The verifying step of a serving batch, ragged contexts and drafts.
        dict(name="tree_batch", op="tree", dtype="bfloat16", seqs=24, nodes=32, kv_len=8192, lens=2, heads=32,
             kv_heads=8, head_dim=128, page_size=64, blocksize=64, bits=4, window=0),
        # Drafts over few long contexts, 8-bit cache.
        dict(name="tree_long", op="tree", dtype="float16", seqs=2, nodes=48, kv_len=131072, lens=3, heads=16,
             kv_heads=2, head_dim=128, page_size=128, blocksize=128, bits=8, window=0),
        # Small drafts, small heads, a sliding window.
        dict(name="tree_window", op="tree", dtype="float16", seqs=20, nodes=13, kv_len=10000, lens=4, heads=20,
             kv_heads=5, head_dim=64, page_size=32, blocksize=32, bits=8, window=4000),
        # One key/value head, wide heads.
        dict(name="tree_wide", op="tree", dtype="bfloat16", seqs=5, nodes=21, kv_len=6000, lens=5, heads=8,
             kv_heads=1, head_dim=256, page_size=64, blocksize=128, bits=8, window=0),
        # The largest tree, over a long context: the most arithmetic.
        dict(name="tree_large", op="tree", dtype="bfloat16", seqs=2, nodes=256, kv_len=18432, lens=6, heads=32,
             kv_heads=4, head_dim=128, page_size=64, blocksize=64, bits=4, window=0),
        # One user's accepted path.
        dict(name="accept_single", op="accept", dtype="bfloat16", seqs=1, nodes=26, path=5, kv_len=1026, lens=7,
             kv_heads=8, head_dim=128, page_size=16, blocksize=64, bits=4),
        # The accepted paths of a large serving batch, 8-bit cache.
        dict(name="accept_batch", op="accept", dtype="float16", seqs=512, nodes=64, path=9, kv_len=2100, lens=8,
             kv_heads=8, head_dim=128, page_size=64, blocksize=128, bits=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "append", "tree", "tree", "tree", "accept"])
    dim = rng.choice([64, 128, 128, 256])
    case = dict(op=op, head_dim=dim, page_size=rng.choice([16, 32, 64, 128]), bits=rng.choice([4, 8]),
                blocksize=rng.choice([b for b in (32, 64, 128, 256) if b <= dim]))
    if op == "append":
        group, kv_heads = rng.choice([1, 2, 3, 4, 7, 8]), rng.randint(1, 8)
        kv_heads = max(1, min(kv_heads, 32 // group))
        size = 2 if (dtype := rng.choice(["float32", "float16", "bfloat16"])) == "float32" else 1
        tokens = _log_int(rng, 1, min(16384, 16384 * 48 * 128 // (size * (group + 2) * kv_heads * dim)))
        case.update(dtype=dtype, heads=group * kv_heads, kv_heads=kv_heads, tokens=tokens, fresh=_log_int(rng, 1, tokens),
                    rotary_dim=rng.choice([dim, dim, dim // 2, 16 * rng.randint(1, dim // 16)]),
                    interleaved=rng.random() < 0.4)
    elif op == "tree":
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        kv_heads = rng.randint(1, max(1, min(8, 32 // group)))
        heads = group * kv_heads
        nodes = _log_int(rng, 1, 256)
        seqs = _log_int(rng, 1, 48)
        # at most the listed cases' cache and arithmetic
        most = min(131072, 24 * 8192 * 8 * 128 // (seqs * kv_heads * dim),
                   2 * 256 * 18432 * 32 * 128 // (seqs * nodes * heads * dim))
        nodes = min(nodes, max(1, most))
        kv_len = _log_int(rng, max(nodes, min(16, most)), max(nodes, most))
        window = 0 if rng.random() < 0.7 else _log_int(rng, 4, 8192)
        case.update(dtype=rng.choice(["float16", "bfloat16"]), seqs=seqs, nodes=nodes, kv_len=kv_len,
                    lens=rng.randint(1, 1 << 30), heads=heads, kv_heads=kv_heads, window=window)
    else:
        kv_heads = rng.randint(1, 8)
        path = rng.randint(1, 12)
        nodes = max(4 * path, _log_int(rng, 8, 256))
        case.update(dtype=rng.choice(["float32", "float16", "bfloat16"]), kv_heads=kv_heads, nodes=nodes, path=path,
                    seqs=_log_int(rng, 1, min(512, 512 * 1024 // (kv_heads * dim))), lens=rng.randint(1, 1 << 30),
                    kv_len=nodes + rng.randint(0, 2000))
    return case


def _lengths(case):
    """(drafted tokens, context and draft) of each sequence: the first has the most of both; in larger
    batches one in eight is an unused place."""
    rng = random.Random(case["lens"])
    out = []
    for s in range(case["seqs"]):
        if s == 0:
            out.append((case["nodes"], case["kv_len"]))
        elif rng.random() < 0.125:
            out.append((0, 0))
        else:
            n = rng.randint(max(1, case["nodes"] // 2), case["nodes"])
            out.append((n, max(n, rng.randint(max(1, case["kv_len"] // 4), case["kv_len"]))))
    return out


def _token_bytes(case):
    """Bytes of one token's keys and values in the cache."""
    row = case["kv_heads"] * case["head_dim"]
    return 2 * (row * case["bits"] // 8 + 4 * (row // case["blocksize"]))


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    row = case["kv_heads"] * case["head_dim"]
    if case["op"] == "append":  # inputs, the cache written, queries out, the values read back
        t, q = case["tokens"], case["heads"] * case["head_dim"]
        angles = min(t, _POSITIONS) * case["rotary_dim"] * 4
        return {"bytes": t * (2 * row * size + _token_bytes(case) + 2 * row * size + 2 * q * size + 16) + angles,
                "flops": t * (6 * row + 3 * (q + row))}
    if case["op"] == "accept":  # the moved tokens out of and into the cache, the kept ones read back
        kept = sum(_path_lengths(case))
        return {"bytes": kept * (3 * _token_bytes(case) + 2 * row * size + 12), "flops": 2 * kept * row}
    tokens = pairs = cached = 0
    for n, kv in _lengths(case):
        tokens += n
        seen = min(kv - n, case["window"]) if case["window"] else kv - n
        cached += seen + n
        pairs += n * (seen + 1)
    head_row = case["heads"] * case["head_dim"]
    return {"bytes": 2 * tokens * head_row * size + cached * _token_bytes(case), "flops": 4 * pairs * head_row}


# ---- inputs ---------------------------------------------------------------------------------

def _table(bits):
    """Sorted codes in [-1, 1]: quantiles of the normal distribution around zero (4 bits), evenly
    spaced ones (8 bits)."""
    if bits == 8:
        return [(2 * k - 255) / 255 for k in range(256)]
    n = statistics.NormalDist()
    top = n.inv_cdf(1 - 1 / 32)
    low = [-n.inv_cdf(1 - 1 / 32 - k * (0.5 - 1 / 32) / 7) / top for k in range(7)]
    high = [n.inv_cdf(1 - 1 / 32 - k * (0.5 - 1 / 32) / 8) / top for k in range(8)]
    return sorted(low + [0.0] + high)


def _new_pool(case, pages, device):
    """An empty cache; its statistics begin as zeros."""
    shape = (pages, case["kv_heads"], case["page_size"])
    row = case["head_dim"] * case["bits"] // 8
    blocks = case["head_dim"] // case["blocksize"]
    return {k: (torch.zeros(*shape, row, dtype=torch.uint8, device=device),
                torch.zeros(*shape, blocks, dtype=torch.float32, device=device)) for k in ("k", "v")}


def _filled_pool(case, pages, gen, device):
    """A cache of values as they come about: codes as normal values of a block have them, maxima of a
    few octaves, keys with some strong channels."""
    pool = _new_pool(case, pages, device)
    blocks = case["head_dim"] // case["blocksize"]
    table = torch.tensor(_table(case["bits"]), dtype=torch.float32, device=device)
    mid = (table[1:] + table[:-1]) / 2
    n = pool["k"][0].numel() * 8 // case["bits"]
    for key in ("k", "v"):
        packed, absmax = pool[key]
        flat = packed.view(-1)
        for at in range(0, n, 1 << 26):  # in pieces, to keep the temporaries small
            m = min(1 << 26, n - at)
            x = torch.randn(m, generator=gen, device=device).mul_(0.38)
            codes = torch.bucketize(x, mid, out_int32=True).to(torch.uint8)
            if case["bits"] == 8:
                flat[at:at + m] = codes
            else:
                flat[at // 2:(at + m) // 2] = (codes[0::2] << 4) | codes[1::2]
        a = torch.randn(absmax.shape, generator=gen, device=device).mul_(0.25).add_(0.95).exp_()
        if key == "k":
            a *= torch.exp(0.4 * torch.randn(case["kv_heads"], 1, blocks, generator=gen, device=device))
        absmax.copy_(a)
    return pool


def _token_slots(case, tokens, fresh, gen, device):
    """Cache slots of `tokens` tokens that come in runs of `fresh`, each run on pages of its own
    (from a slot inside its first page on), pages in any order.  Returns slots and page count."""
    ps = case["page_size"]
    runs = -(-tokens // fresh)
    per_run = -(-fresh // ps) + 1
    pages = torch.randperm(runs * per_run, generator=gen, device=device).reshape(runs, per_run)
    start = torch.randint(0, ps, (runs, 1), generator=gen, device=device)
    pos = start + torch.arange(fresh, device=device)
    slots = torch.gather(pages, 1, pos // ps) * ps + pos % ps
    return slots.reshape(-1)[:tokens].contiguous(), runs * per_run


def _tree(rng, n):
    """Parents of n drafted tokens, level by level, a parent's first continuations the likeliest to be
    continued; one draft in six ends in unused places."""
    used = max(1, n - rng.randint(1, 3)) if rng.random() < 1 / 6 else n
    parents = []
    level, size = [-1], max(1, min(8, used // 3))
    while len(parents) < used:
        m = min(size, used - len(parents))
        new = sorted(level[min(len(level) - 1, int(len(level) * rng.random() ** 2))] for _ in range(m))
        level = list(range(len(parents), len(parents) + m))
        parents += new
        size = max(1, min(2 * size, used // 3)) if len(parents) < used // 2 else max(1, size // 2)
    return parents + [-2] * (n - used)


def _path_lengths(case):
    """Accepted tokens of each sequence, the first the most."""
    rng = random.Random(case["lens"] + 1)
    return [min(case["path"], n // 2) if s == 0 else rng.randint(1, min(case["path"], n // 2)) if n else 0
            for s, (n, _) in enumerate(_lengths(case))]


def _path(rng, n, length):
    """An accepted path of a draft laid out level by level: its first tokens in place, the others behind."""
    stay = rng.randint(0, min(1, length - 1))
    return list(range(stay)) + sorted(rng.sample(range(length, n), length - stay))


def _library():
    import dequantization_block_absmax_amd as bq
    return bq


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    h, d, ps = case["kv_heads"], case["head_dim"], case["page_size"]
    dtype = _DTYPES[case["dtype"]]
    st = {"case": case, "dtype": dtype, "table": torch.tensor(_table(case["bits"]), dtype=torch.float32, device=device)}
    if case["op"] == "append":
        t, heads = case["tokens"], case["heads"]
        slots, pages = _token_slots(case, t, case["fresh"], gen, device)
        # queries, keys and values are parts of the projection's output; keys with strong channels and offsets
        qkv = torch.randn(t, heads + 2 * h, d, generator=gen, device=device)
        qkv[:, heads:heads + h] *= torch.exp(0.5 * torch.randn(h, d, generator=gen, device=device))
        qkv[:, heads:heads + h] += 0.5 * torch.randn(h, d, generator=gen, device=device)
        qkv = qkv.to(dtype)
        runs = -(-t // case["fresh"])
        first = torch.randint(0, max(1, _POSITIONS - case["fresh"]), (runs, 1), generator=gen, device=device)
        positions = (first + torch.arange(case["fresh"], device=device)).reshape(-1)[:t].contiguous()
        pair = torch.arange(case["rotary_dim"] // 2, device=device, dtype=torch.float64)
        angle = torch.arange(_POSITIONS, device=device, dtype=torch.float64)[:, None] * 10000.0 ** (-2 * pair / case["rotary_dim"])
        st.update(slots=slots, positions=positions, q=qkv[:, :heads], k=qkv[:, heads:heads + h], v=qkv[:, heads + h:],
                  cos=angle.cos().float(), sin=angle.sin().float(), pool=_new_pool(case, pages, device),
                  q_out=torch.empty(t, heads, d, dtype=dtype, device=device))
    else:
        lens = _lengths(case)
        need = [-(-kv // ps) for _, kv in lens]
        pages, width = max(1, sum(need)), max(1, max(need))
        order = torch.randperm(pages, generator=gen, device=device).to(torch.int32).cpu()
        page_table = torch.full((len(lens), width), -1, dtype=torch.int32)
        starts = [0]
        at = 0
        for s, (n, _) in enumerate(lens):
            page_table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
            starts.append(starts[-1] + n)
        pool = _filled_pool(case, pages, gen, device)
        for s, (_, kv) in enumerate(lens):  # slots behind a sequence's end were never written
            if kv % ps:
                last = int(page_table[s, kv // ps])
                pool["k"][1][last, :, kv % ps:] = float("nan")
                pool["v"][1][last, :, kv % ps:] = float("nan")
        st.update(pool=pool, page_table=page_table.to(device), tokens=starts[-1],
                  q_start=torch.tensor(starts, dtype=torch.int32, device=device),
                  kv_len=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=device))
        if case["op"] == "tree":
            parents = [p for n, _ in lens if n for p in _tree(rng, n)]
            st.update(parents=torch.tensor(parents, dtype=torch.int32, device=device), scale=1.0 / math.sqrt(d),
                      q=(2 * torch.randn(starts[-1], case["heads"], d, generator=gen, device=device)).to(dtype))
        else:
            longest, count = case["path"], _path_lengths(case)
            path = torch.full((len(lens), longest), -1, dtype=torch.int32)
            for s, (n, _) in enumerate(lens):
                path[s, :count[s]] = torch.tensor(_path(rng, n, count[s]) if count[s] else [], dtype=torch.int32)
            at = torch.tensor([kv - n for n, kv in lens])[:, None] + torch.arange(longest)
            page = page_table[torch.arange(len(lens))[:, None], (at // ps).clamp(max=width - 1)].long()
            kept = torch.arange(longest) < torch.tensor(count)[:, None]
            st.update(path=path.to(device), path_len=torch.tensor(count, dtype=torch.int32, device=device),
                      slots=(page * ps + at % ps)[kept].contiguous().to(device))
            for key in ("k", "v"):  # a slot that this batch never writes: its statistics are zeros
                pool[key][1].nan_to_num_(0.0)
    if case["op"] != "tree":  # where tokens are read back to
        n = st["slots"].numel()
        st["k_out"] = torch.empty(n, h, d, dtype=dtype, device=device)
        st["v_out"] = torch.empty(n, h, d, dtype=dtype, device=device)
    if own:
        bq = _library()
        st["cache"] = bq.kv_cache(st["pool"]["k"][0], st["pool"]["k"][1], st["pool"]["v"][0], st["pool"]["v"][1],
                                  st["table"].cpu().numpy(), st["pool"]["k"][0].shape[0], ps, h, d, case["blocksize"])
        if case["op"] == "append":
            st["rotation"] = bq.rotation(st["cos"], st["sin"], case["rotary_dim"], case["interleaved"])
        else:
            st["batch"] = bq.kv_batch(st["q_start"], st["kv_len"], st["page_table"], st["tokens"], case["nodes"],
                                      case["kv_len"])
        if case["op"] == "tree":
            st["out"] = torch.empty_like(st["q"])
            size = bq.bq_kv_tree_attention_workspace_bytes(st["cache"], st["batch"], dtype, case["heads"])
            st["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device=device)
    return st


# ---- one pass -------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "tree": _own_tree, "accept": _own_accept}[op](state)
    return {"append": _plain_append, "tree": _plain_tree, "accept": _plain_accept}[op](state)


def _own_read(st):
    bq = _library()
    k, v = st["k_out"], st["v_out"]
    bq.check(bq.bq_kv_read(st["cache"], st["dtype"], k, v, k.shape[0], k.stride(0), v.stride(0), st["slots"]))
    return k, v, st["pool"]["k"][1], st["pool"]["v"][1]


def _own_append(st):
    bq = _library()
    q, k, v, out = st["q"], st["k"], st["v"], st["q_out"]
    bq.check(bq.bq_kv_append(st["cache"], st["rotation"], st["dtype"], k, v, k.shape[0], k.stride(0), v.stride(0),
                             st["positions"], st["slots"], q, q.stride(0), q.shape[1], out, out.stride(0)))
    return (out, *_own_read(st))


def _own_tree(st):
    bq = _library()
    q, out = st["q"], st["out"]
    bq.check(bq.bq_kv_tree_attention(st["cache"], st["batch"], st["parents"], st["dtype"], q, q.stride(0),
                                     st["case"]["heads"], st["scale"], st["case"]["window"], out, out.stride(0), None,
                                     st["workspace"]))
    return out


def _own_accept(st):
    bq = _library()
    bq.check(bq.bq_kv_tree_accept(st["cache"], st["batch"], st["path"], st["path"].stride(0), st["path_len"]))
    return _own_read(st)


def _quantize(x, table, blocksize):
    """Codes (one a byte) and block maxima of x, blocks along its last axis, in binary32."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // blocksize, blocksize)
    finite = torch.isfinite(b)
    a = torch.where(finite, b, 0.0).abs().amax(-1, keepdim=True)
    s = torch.where(a < 2.0 ** -64, 2.0 ** 64, torch.where(a > 2.0 ** 64, 2.0 ** -64, 1.0))
    y = (b * s) * (1.0 / (a * s))
    y = torch.where(finite & (a > 0), y, 0.0)
    c = table.double()
    mid = (c[1:] + c[:-1]) / 2  # exact in binary64; the code is the number of midpoints below y
    codes = torch.bucketize(y.double(), mid).to(torch.uint8)
    return codes.reshape(x.shape), a.squeeze(-1)


def _pack(codes, bits):
    return codes if bits == 8 else (codes[..., 0::2] << 4) | codes[..., 1::2]


def _unpack(packed, bits):
    return packed if bits == 8 else torch.stack((packed >> 4, packed & 15), -1).flatten(-2)


def _values(st, packed, absmax):
    """Cached values in binary32 of codes and maxima with any leading axes."""
    codes = _unpack(packed, st["case"]["bits"])
    return st["table"][codes.int()] * absmax.repeat_interleave(st["case"]["blocksize"], -1)


def _plain_read(st):
    ps = st["case"]["page_size"]
    page, slot = st["slots"] // ps, st["slots"] % ps
    k, v = (_values(st, st["pool"][key][0][page, :, slot], st["pool"][key][1][page, :, slot]).to(st["dtype"])
            for key in ("k", "v"))
    return k, v, st["pool"]["k"][1], st["pool"]["v"][1]


def _rotate(st, x):
    case = st["case"]
    r = case["rotary_dim"]
    c, s = st["cos"][st["positions"]][:, None], st["sin"][st["positions"]][:, None]
    x = x.float()
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _plain_append(st):
    case, ps = st["case"], st["case"]["page_size"]
    page, slot = st["slots"] // ps, st["slots"] % ps
    q = _rotate(st, st["q"]).to(st["dtype"])
    for key, x in (("k", _rotate(st, st["k"])), ("v", st["v"].float())):
        codes, a = _quantize(x, st["table"], case["blocksize"])
        st["pool"][key][0][page, :, slot] = _pack(codes, case["bits"])
        st["pool"][key][1][page, :, slot] = a
    return (q, *_plain_read(st))


def _plain_accept(st):
    ps, width = st["case"]["page_size"], st["page_table"].shape[1]
    n = st["q_start"][1:] - st["q_start"][:-1]
    first = (st["kv_len"] - n).long()[:, None]
    i = torch.arange(st["path"].shape[1], device=first.device)
    keep = i < st["path_len"][:, None]

    def places(at):  # page and slot of each sequence's tokens `at`
        at = torch.where(keep, at, 0)
        page = torch.gather(st["page_table"].long(), 1, (at // ps).clamp(max=width - 1))
        return page.clamp(min=0), at % ps

    to = places(first + i)
    # an unused entry moves its sequence's last accepted token again
    last = (st["path_len"] - 1).clamp(min=0).long()[:, None]
    src = places(first + torch.where(keep, st["path"], 0).long())
    src, to = (tuple(torch.where(keep, t, torch.gather(t, 1, last)) for t in pair) for pair in (src, to))
    none = (st["path_len"] == 0)[:, None]  # the first sequence has a path: its first move again
    src, to = (tuple(torch.where(none, t[:1, :1], t) for t in pair) for pair in (src, to))
    for key in ("k", "v"):
        for part in st["pool"][key]:
            part[to[0], :, to[1]] = part[src[0], :, src[1]]
    return _plain_read(st)


def _plain_tree(st):
    """All sequences side by side, padded to the longest context and draft."""
    case = st["case"]
    h, d, ps, n = case["kv_heads"], case["head_dim"], case["page_size"], case["nodes"]
    group = case["heads"] // h
    table = st["page_table"].clamp(min=0).long()
    seqs, keys = table.shape[0], table.shape[1] * ps
    dev = table.device
    j = torch.arange(keys, device=dev)
    kv, nq = st["kv_len"].long()[:, None], (st["q_start"][1:] - st["q_start"][:-1]).long()[:, None]
    k, v = (torch.where((j < kv)[:, None, :, None],
                        _values(st, *(t[table].transpose(1, 2).reshape(seqs, h, keys, -1) for t in st["pool"][key])), 0.0)
            for key in ("k", "v"))
    # ancestors of each drafted token, itself among them: powers of the matrix of parents
    i = torch.arange(n, device=dev)
    used = i < nq
    rows = torch.where(used, st["q_start"][:-1].long()[:, None] + i, 0)
    parent = torch.where(used, st["parents"][rows].long(), -2)
    fine = (parent >= -1) & (parent < i)
    above = ((parent[..., None] == i) & fine[..., None]).float() + torch.eye(n, device=dev)
    for _ in range(8):  # paths of up to 256 tokens
        above = (torch.matmul(above, above) > 0).float()
    above = above > 0
    fine = fine & ~(above & ~fine[:, None]).any(-1)  # no unused place among the ancestors
    above = above & fine[..., None]
    depth = above.sum(-1) - 1
    # what each sees: the context, and the drafted tokens on its path, within the window
    context = kv - nq
    node = j - context
    on_path = torch.gather(above, 2, node.clamp(0, n - 1)[:, None].expand(seqs, n, keys))
    at = torch.where(node < 0, j, context + torch.gather(depth, 1, node.clamp(0, n - 1)))[:, None]  # positions of keys
    pos = (context + depth)[..., None]
    seen = torch.where((node < 0)[:, None], fine[..., None], on_path & (node < nq)[:, None])
    if case["window"]:
        seen = seen & (at > pos - case["window"])
    q = st["q"][rows].float().reshape(seqs, n, h, group, d).permute(0, 2, 1, 3, 4).reshape(seqs * h, n * group, d)
    score = torch.matmul(q, k.reshape(seqs * h, keys, d).transpose(1, 2).contiguous()) * st["scale"]
    score = torch.where(seen[:, None, :, None], score.reshape(seqs, h, n, group, keys), float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.reshape(seqs * h, n * group, keys), v.reshape(seqs * h, keys, d))
    o = o.reshape(seqs, h, n, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, n, h * group, d).to(st["dtype"])
    out = torch.zeros(st["tokens"] + 1, h * group, d, dtype=st["dtype"], device=dev)
    out[torch.where(used, rows, st["tokens"])] = o
    return out[:-1]


# ---- in 64 bits -----------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    table = torch.tensor(_table(case["bits"]), dtype=torch.float32, device=st["table"].device).double()
    return {"append": _exact_append, "tree": _exact_tree, "accept": _exact_accept}[case["op"]](case, st, table)


def _exact_values(case, packed, absmax, table):
    """Every value of (part of) a pool, as code times block maximum."""
    p = packed.long()
    if case["bits"] == 4:
        p = torch.cat(((p // 16).unsqueeze(-1), (p % 16).unsqueeze(-1)), -1).reshape(*p.shape[:-1], case["head_dim"])
    v = table[p].reshape(*absmax.shape, case["blocksize"]) * absmax.double().unsqueeze(-1)
    return v.reshape(p.shape)


def _fl32(t):
    return t.to(torch.float32).to(torch.float64)


def _exact_rotated(case, st, x):
    """The definition: products of two 32-bit numbers are exact in 64 bits, then rounded to 32; a sum of
    two 32-bit numbers is rounded to 64 bits and then to 32 (more than twice the bits: as if once)."""
    x = x.double()
    half = case["rotary_dim"] // 2
    out = x.clone()
    pair = torch.arange(half, device=x.device)
    first = 2 * pair if case["interleaved"] else pair
    second = first + 1 if case["interleaved"] else pair + half
    cos, sin = st["cos"].double()[st["positions"]].unsqueeze(1), st["sin"].double()[st["positions"]].unsqueeze(1)
    out[..., first] = _fl32(_fl32(x[..., first] * cos) - _fl32(x[..., second] * sin))
    out[..., second] = _fl32(_fl32(x[..., second] * cos) + _fl32(x[..., first] * sin))
    return out


def _exact_append(case, st, table):
    h, d, b = case["kv_heads"], case["head_dim"], case["blocksize"]
    mid = (table[:-1] + table[1:]) * 0.5
    values, stats = [], []
    for key in ("k", "v"):
        x = _exact_rotated(case, st, st["k"]) if key == "k" else st["v"].double()
        x = x.reshape(case["tokens"], h, d // b, b)
        ok = ~(torch.isnan(x) | torch.isinf(x))
        a = torch.where(ok, x.abs(), torch.zeros_like(x)).max(dim=-1, keepdim=True).values
        one = torch.ones_like(a)
        s = torch.where(a < 2.0 ** -64, one * 2.0 ** 64, one)
        s = torch.where(a > 2.0 ** 64, one * 2.0 ** -64, s)
        y = _fl32(_fl32(x * s) * _fl32(1.0 / _fl32(a * s)))
        y = torch.where(ok & (a > 0), y, torch.zeros_like(y))
        code = torch.searchsorted(mid, y.reshape(-1)).reshape(y.shape)
        values.append((table[code] * a).reshape(case["tokens"], h, d))
        pages = st["pool"][key][1].shape[0]
        flat = torch.zeros(pages * case["page_size"], h, d // b, dtype=torch.float64, device=x.device)
        flat[st["slots"]] = a.squeeze(-1)
        stats.append(flat.reshape(pages, case["page_size"], h, d // b).transpose(1, 2).contiguous())
    return (_exact_rotated(case, st, st["q"]), *values, *stats)


def _exact_accept(case, st, table):
    """Token by token on the host."""
    ps = case["page_size"]
    moved = {key: [t.clone() for t in st["pool"][key]] for key in ("k", "v")}
    pages, path, count = st["page_table"].tolist(), st["path"].tolist(), st["path_len"].tolist()
    src, to = [], []
    for s, (n, kv) in enumerate(_lengths(case)):
        for i in range(count[s]):
            a, b = kv - n + path[s][i], kv - n + i
            src.append(pages[s][a // ps] * ps + a % ps)
            to.append(pages[s][b // ps] * ps + b % ps)
    src, to = torch.tensor(src, device=table.device), torch.tensor(to, device=table.device)
    out = []
    for key in ("k", "v"):
        for part, old in zip(moved[key], st["pool"][key]):
            part[to // ps, :, to % ps] = old[src // ps, :, src % ps]
        codes, a = moved[key]
        out.append(_exact_values(case, codes[to // ps, :, to % ps], a[to // ps, :, to % ps], table))
    return (*out, moved["k"][1].double(), moved["v"][1].double())


def _exact_tree(case, st, table):
    h, d, g = case["kv_heads"], case["head_dim"], case["heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    parents = st["parents"].tolist()
    row = 0
    for s, (n, kv) in enumerate(_lengths(case)):
        rows = slice(row, row + n)
        row += n
        if not n:
            continue
        hidden = torch.ones(n, kv, dtype=torch.bool)
        for i in range(n):
            chain, at = [], i
            while at >= 0:
                chain.append(at)
                up = parents[rows.start + at]
                at = up if up < at else -2
            if at != -1:
                continue
            reach = case["window"] or kv  # tokens back from and with the last
            hidden[i, [kv - n + c for c in chain[:reach]]] = False
            hidden[i, max(0, kv - n + len(chain) - reach):kv - n] = False
        hidden = hidden.to(out.device)
        pages = st["page_table"][s, : -(-kv // case["page_size"])].long()
        for head in range(h):
            side = {}
            for key in ("k", "v"):
                packed, absmax = (t[pages, head] for t in st["pool"][key])
                side[key] = _exact_values(case, packed, absmax, table).reshape(-1, d)[:kv]
            for j in range(g):
                z = (st["q"][rows, head * g + j].double() @ side["k"].T) * st["scale"]
                z = z.masked_fill(hidden, -math.inf)
                p = torch.softmax(z, dim=-1)
                out[rows, head * g + j] = torch.where(hidden.all(-1, keepdim=True), 0.0, p) @ side["v"]
    return out
