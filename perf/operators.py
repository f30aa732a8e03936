"""The paged key/value cache held in blockwise codes, as it is measured: writing new tokens'
keys and values into it, reading tokens back, and attention of new tokens over it.

A cache is a pool of pages.  Element (page, head, slot, d) of the pool is flat element
((page * kv_heads + head) * page_size + slot) * head_dim + d of an array quantized blockwise:
its value is table[code] * absmax[flat // blocksize].  4-bit codes are two to a byte, the first
of a pair in the high nibble; 8-bit codes one to a byte.

`run` takes a state of `prepare` through one pass, in elementary torch operations where `own` is
false and through the library's entry points where it is true.
"""
import math
import random
import statistics

import torch

own = False

_DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


# ---- cases ----------------------------------------------------------------------------------

def listed():
    return [
        # One decoding step of a serving batch: every sequence appends one token to a page of its
        # own.  The smallest write, all latency.
        dict(name="write_step", op="write", dtype="bfloat16", tokens=48, fresh=1, kv_heads=8, head_dim=128,
             page_size=16, blocksize=64, bits=4),
        # A long prompt enters an 8-bit cache, one scale to a head.
        dict(name="write_prompt", op="write", dtype="bfloat16", tokens=16384, fresh=16384, kv_heads=8, head_dim=128,
             page_size=64, blocksize=128, bits=8),
        # Ragged prompts of a smaller model kept in binary32, odd head count, smallest blocks.
        dict(name="write_ragged", op="write", dtype="float32", tokens=4099, fresh=333, kv_heads=5, head_dim=64,
             page_size=32, blocksize=32, bits=4),
        # A short prefix is taken out of the cache (to move it to another card).
        dict(name="read_short", op="read", dtype="float16", tokens=517, kv_heads=4, head_dim=64, page_size=16,
             blocksize=64, bits=8),
        # A long context is taken out of the cache.
        dict(name="read_long", op="read", dtype="bfloat16", tokens=32768, kv_heads=8, head_dim=128, page_size=64,
             blocksize=64, bits=4),
        # One user's next token after a short dialogue: the smallest attention, all latency.
        dict(name="decode_single", op="attend", dtype="bfloat16", seqs=1, q_len=1, kv_len=1000, lens=1, heads=32,
             kv_heads=8, head_dim=128, page_size=16, blocksize=64, bits=4, window=0),
        # The decoding step of a serving batch, ragged contexts.
        dict(name="decode_batch", op="attend", dtype="bfloat16", seqs=64, q_len=1, kv_len=8192, lens=2, heads=32,
             kv_heads=8, head_dim=128, page_size=64, blocksize=64, bits=4, window=0),
        # Next tokens of few long contexts, 8-bit cache.
        dict(name="decode_long", op="attend", dtype="float16", seqs=3, q_len=1, kv_len=131072, lens=3, heads=16,
             kv_heads=2, head_dim=128, page_size=128, blocksize=128, bits=8, window=0),
        # A few drafted tokens per sequence are scored at once, small heads, sliding window.
        dict(name="draft_window", op="attend", dtype="float16", seqs=24, q_len=6, kv_len=10000, lens=4, heads=20,
             kv_heads=5, head_dim=64, page_size=32, blocksize=32, bits=8, window=4000),
        # Mixed batch: some sequences decode, others bring part of a prompt.
        dict(name="chunk_ragged", op="attend", dtype="float16", seqs=9, q_len=700, kv_len=5000, lens=5, heads=16,
             kv_heads=4, head_dim=64, page_size=16, blocksize=64, bits=4, window=0),
        # A piece of a prompt, one key/value head, wide heads.
        dict(name="chunk_wide", op="attend", dtype="bfloat16", seqs=1, q_len=777, kv_len=6000, lens=6, heads=8,
             kv_heads=1, head_dim=256, page_size=64, blocksize=128, bits=8, window=0),
        # A large piece of a long prompt: the most arithmetic.
        dict(name="chunk_long", op="attend", dtype="bfloat16", seqs=1, q_len=2048, kv_len=18432, lens=7, heads=32,
             kv_heads=8, head_dim=128, page_size=64, blocksize=64, bits=4, window=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    case = dict(op=op, head_dim=dim, page_size=rng.choice([16, 32, 64, 128]), bits=rng.choice([4, 8]),
                blocksize=rng.choice([b for b in (32, 64, 128, 256) if b <= dim]))
    if op == "write":
        kv_heads = rng.randint(1, 8)
        tokens = _log_int(rng, 1, min(16384, (16384 * 1024) // (kv_heads * dim)))
        case.update(dtype=rng.choice(["float32", "float16", "bfloat16"]), kv_heads=kv_heads, tokens=tokens,
                    fresh=_log_int(rng, 1, tokens))
    elif op == "read":
        kv_heads = rng.randint(1, 8)
        tokens = _log_int(rng, 1, min(32768, (32768 * 1024) // (kv_heads * dim)))
        case.update(dtype=rng.choice(["float32", "float16", "bfloat16"]), kv_heads=kv_heads, tokens=tokens)
    else:
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        kv_heads = rng.randint(1, max(1, min(8, 32 // group)))
        heads = group * kv_heads
        q_len = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 2048)])
        # at most the decoding and prompt cases' cache and arithmetic
        seqs = _log_int(rng, 1, 64 if q_len <= 8 else 8)
        most = min(131072, 64 * 8192 * 8 * 128 // (seqs * kv_heads * dim),
                   2048 * 18432 * 32 * 128 // (seqs * q_len * heads * dim))
        q_len = min(q_len, most)
        kv_len = _log_int(rng, max(q_len, min(16, most)), most)
        window = 0 if rng.random() < 0.7 else _log_int(rng, 16, 8192)
        case.update(dtype=rng.choice(["float16", "bfloat16"]), seqs=seqs, q_len=q_len, kv_len=kv_len,
                    lens=rng.randint(1, 1 << 30), heads=heads, kv_heads=kv_heads, window=window)
    return case


def _lengths(case):
    """(new tokens, context) of each sequence of an attention case: the first has the most of
    both; the others are spread, and in larger batches one in eight is an unused place."""
    rng = random.Random(case["lens"])
    out = []
    for s in range(case["seqs"]):
        if s == 0:
            out.append((case["q_len"], case["kv_len"]))
        elif rng.random() < 0.125:
            out.append((0, 0))
        else:
            q = case["q_len"] if case["q_len"] <= 8 else _log_int(rng, 1, case["q_len"])
            out.append((q, max(q, rng.randint(max(1, case["kv_len"] // 4), case["kv_len"]))))
    return out


def _token_bytes(case):
    """Bytes of one token's keys and values in the cache."""
    row = case["kv_heads"] * case["head_dim"]
    return 2 * (row * case["bits"] // 8 + 4 * (row // case["blocksize"]))


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    row = case["kv_heads"] * case["head_dim"]
    if case["op"] == "write":  # inputs, the cache written, the values read back
        t = case["tokens"]
        return {"bytes": t * (2 * row * size + _token_bytes(case) + 2 * row * size + 8), "flops": 6 * t * row}
    if case["op"] == "read":
        t = case["tokens"]
        return {"bytes": t * (_token_bytes(case) + 2 * row * size + 8), "flops": 2 * t * row}
    tokens = pairs = cached = 0
    for q, kv in _lengths(case):
        tokens += q
        w = case["window"] or kv
        cached += min(kv, w + q - 1) if q else 0
        # query i sees the min(window, kv - q + i + 1) last keys up to its own
        first = kv - q + 1
        full = max(0, min(q, w - first))
        pairs += full * first + full * (full - 1) // 2 + (q - full) * min(w, kv)
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


def _quantize(x, table, blocksize):
    """Codes (one a byte) and block maxima of x, blocks along its last axis, in binary32."""
    x = x.float()
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


def _new_pool(case, pages, device):
    """An empty cache; its statistics begin as zeros."""
    shape = (pages, case["kv_heads"], case["page_size"])
    row = case["head_dim"] * case["bits"] // 8
    blocks = case["head_dim"] // case["blocksize"]
    return {k: (torch.zeros(*shape, row, dtype=torch.uint8, device=device),
                torch.zeros(*shape, blocks, dtype=torch.float32, device=device)) for k in ("k", "v")}


def _keys_values(case, tokens, gen, device):
    """Keys with a few strong channels and an offset per channel, plain values; (tokens, heads, dim)."""
    h, d = case["kv_heads"], case["head_dim"]
    channel = torch.exp(0.5 * torch.randn(h, d, generator=gen, device=device))
    offset = 0.5 * torch.randn(h, d, generator=gen, device=device)
    k = torch.randn(tokens, h, d, generator=gen, device=device) * channel + offset
    v = torch.randn(tokens, h, d, generator=gen, device=device)
    return k, v


def _library():
    import dequantization_block_absmax_amd as bq
    return bq


def _own_cache(case, pool, table):
    bq = _library()
    return bq.kv_cache(pool["k"][0], pool["k"][1], pool["v"][0], pool["v"][1], table.cpu().numpy(),
                       pool["k"][0].shape[0], case["page_size"], case["kv_heads"], case["head_dim"],
                       case["blocksize"])


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


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    table = torch.tensor(_table(case["bits"]), dtype=torch.float32, device=device)
    dtype = _DTYPES[case["dtype"]]
    h, d = case["kv_heads"], case["head_dim"]
    st = {"case": case, "table": table, "dtype": dtype}
    if case["op"] == "write":
        t = case["tokens"]
        slots, pages = _token_slots(case, t, case["fresh"], gen, device)
        k, v = _keys_values(case, t, gen, device)
        # keys and values are views of the projection's output, behind the queries
        qkv = torch.empty(t, 4 * h, d, dtype=dtype, device=device)
        qkv[:, 2 * h:3 * h] = k
        qkv[:, 3 * h:] = v
        st.update(slots=slots, k=qkv[:, 2 * h:3 * h], v=qkv[:, 3 * h:], pool=_new_pool(case, pages, device))
    elif case["op"] == "read":
        t = case["tokens"]
        slots, pages = _token_slots(case, t, t, gen, device)
        st.update(slots=slots, pool=_filled_pool(case, pages, table, gen, device))
    else:
        lens = _lengths(case)
        ps = case["page_size"]
        need = [-(-kv // ps) for _, kv in lens]
        pages = max(1, sum(need))
        width = max(1, max(need))
        order = torch.randperm(pages, generator=gen, device=device).to(torch.int32)
        page_table = torch.full((len(lens), width), -1, dtype=torch.int32, device=device)
        at = 0
        for s, n in enumerate(need):
            page_table[s, :n] = order[at:at + n]
            at += n
        pool = _filled_pool(case, pages, table, gen, device)
        for s, (_, kv) in enumerate(lens):  # slots behind a sequence's end were never written
            if kv % ps:
                last = page_table[s, kv // ps].long()
                pool["k"][1][last, :, kv % ps:] = float("nan")
                pool["v"][1][last, :, kv % ps:] = float("nan")
        starts = [0]
        for q, _ in lens:
            starts.append(starts[-1] + q)
        tokens = starts[-1]
        q = (2 * torch.randn(tokens, case["heads"], d, generator=gen, device=device)).to(dtype)
        st.update(pool=pool, page_table=page_table, q=q, lens=lens, starts=starts,
                  q_start=torch.tensor(starts, dtype=torch.int32, device=device),
                  kv_len=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=device),
                  scale=1.0 / math.sqrt(d))
    if own:
        bq = _library()
        st["cache"] = _own_cache(case, st["pool"], table)
        if case["op"] in ("write", "read"):
            st["k_out"] = torch.empty(case["tokens"], h, d, dtype=dtype, device=device)
            st["v_out"] = torch.empty(case["tokens"], h, d, dtype=dtype, device=device)
        else:
            st["out"] = torch.empty_like(st["q"])
            st["batch"] = bq.kv_batch(st["q_start"], st["kv_len"], st["page_table"], tokens, case["q_len"],
                                      case["kv_len"])
            size = bq.bq_kv_attention_workspace_bytes(st["cache"], st["batch"], dtype, case["heads"])
            st["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device=device)
    return st


def _filled_pool(case, pages, table, gen, device):
    pool = _new_pool(case, pages, device)
    ps = case["page_size"]
    step = max(1, (1 << 24) // (case["kv_heads"] * ps * case["head_dim"]))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        for key, x in zip("kv", _keys_values(case, n * ps, gen, device)):
            x = x.reshape(n, ps, case["kv_heads"], case["head_dim"]).transpose(1, 2)
            codes, a = _quantize(x, table, case["blocksize"])
            pool[key][0][at:at + n] = _pack(codes, case["bits"])
            pool[key][1][at:at + n] = a
    return pool


# ---- one pass -------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "attend": _own_attend}[op](state)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](state)


def _own_write(st):
    bq = _library()
    k, v = st["k"], st["v"]
    bq.check(bq.bq_kv_write(st["cache"], st["dtype"], k, v, k.shape[0], k.stride(0), v.stride(0), st["slots"]))
    return (*_own_read(st), st["pool"]["k"][1], st["pool"]["v"][1])


def _own_read(st):
    bq = _library()
    k, v = st["k_out"], st["v_out"]
    bq.check(bq.bq_kv_read(st["cache"], st["dtype"], k, v, k.shape[0], k.stride(0), v.stride(0), st["slots"]))
    return k, v


def _own_attend(st):
    bq = _library()
    q, out = st["q"], st["out"]
    bq.check(bq.bq_kv_attention(st["cache"], st["batch"], st["dtype"], q, q.stride(0), st["case"]["heads"],
                                st["scale"], 1, st["case"]["window"], out, out.stride(0), None, st["workspace"]))
    return out


def _plain_write(st):
    case, ps = st["case"], st["case"]["page_size"]
    page, slot = st["slots"] // ps, st["slots"] % ps
    for key in ("k", "v"):
        codes, a = _quantize(st[key], st["table"], case["blocksize"])
        st["pool"][key][0][page, :, slot] = _pack(codes, case["bits"])
        st["pool"][key][1][page, :, slot] = a
    return (*_plain_read(st), st["pool"]["k"][1], st["pool"]["v"][1])


def _values(st, key, page, slot):
    """Cached values of the tokens at (page, slot) in binary32, (tokens, kv_heads, head_dim)."""
    codes = _unpack(st["pool"][key][0][page, :, slot], st["case"]["bits"])
    a = st["pool"][key][1][page, :, slot]
    return st["table"][codes.int()] * a.repeat_interleave(st["case"]["blocksize"], -1)


def _plain_read(st):
    ps = st["case"]["page_size"]
    page, slot = st["slots"] // ps, st["slots"] % ps
    return tuple(_values(st, key, page, slot).to(st["dtype"]) for key in ("k", "v"))


def _plain_attend(st):
    case = st["case"]
    ps, window = case["page_size"], case["window"]
    h, d = case["kv_heads"], case["head_dim"]
    group = case["heads"] // h
    out = torch.zeros_like(st["q"])
    for s, (nq, kv) in enumerate(st["lens"]):
        if nq == 0 or kv == 0:
            continue
        j = torch.arange(kv, device=out.device)
        page, slot = st["page_table"][s, j // ps].long(), j % ps
        k, v = _values(st, "k", page, slot), _values(st, "v", page, slot)
        at = st["starts"][s]
        q = st["q"][at:at + nq].float().reshape(nq, h, group, d)
        pos = torch.arange(kv - nq, kv, device=out.device)[:, None]
        seen = j <= pos
        if window:
            seen = seen & (j > pos - window)
        for head in range(h):
            score = torch.matmul(q[:, head].reshape(nq * group, d), k[:, head].t().contiguous()) * st["scale"]
            score = torch.where(seen[:, None], score.reshape(nq, group, kv), float("-inf"))
            p = torch.exp(score - score.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            o = torch.matmul(p.reshape(nq * group, kv), v[:, head].contiguous())
            out[at:at + nq, head * group:(head + 1) * group] = o.reshape(nq, group, d).to(out.dtype)
    return out


# ---- in 64 bits -----------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    table = torch.tensor(_table(case["bits"]), dtype=torch.float32, device=st["table"].device).double()
    if case["op"] == "write":
        return _exact_write(case, st, table)
    flat = {key: _exact_pool(case, *st["pool"][key], table) for key in ("k", "v")} if case["op"] == "read" else None
    if case["op"] == "read":
        return tuple(flat[key].transpose(1, 2).reshape(-1, case["kv_heads"], case["head_dim"])[st["slots"]]
                     for key in ("k", "v"))
    return _exact_attend(case, st, table)


def _exact_pool(case, packed, absmax, table):
    """Every value of (part of) a pool, as code times block maximum."""
    p = packed.long()
    if case["bits"] == 4:
        p = torch.cat(((p // 16).unsqueeze(-1), (p % 16).unsqueeze(-1)), -1).reshape(*p.shape[:-1], case["head_dim"])
    v = table[p].reshape(*absmax.shape, case["blocksize"]) * absmax.double().unsqueeze(-1)
    return v.reshape(p.shape)


def _exact_write(case, st, table):
    """The definition: block maxima over finite elements, y rounded to binary32 as stated
    (fl32(x * s) * fl32(1 / fl32(a * s)), each product of two binary32 numbers exact in 64 bits), the
    first of the nearest codes."""
    out, stats = [], []
    h, d, b = case["kv_heads"], case["head_dim"], case["blocksize"]
    mid = (table[:-1] + table[1:]) * 0.5

    def fl32(t):
        return t.to(torch.float32).to(torch.float64)

    for key in ("k", "v"):
        x = st[key].to(torch.float64).reshape(case["tokens"], h, d // b, b)
        ok = ~(torch.isnan(x) | torch.isinf(x))
        a = torch.where(ok, x.abs(), torch.zeros_like(x)).max(dim=-1, keepdim=True).values
        one = torch.ones_like(a)
        s = torch.where(a < 2.0 ** -64, one * 2.0 ** 64, one)
        s = torch.where(a > 2.0 ** 64, one * 2.0 ** -64, s)
        inverse = fl32(1.0 / fl32(a * s))
        y = fl32(fl32(x * s) * inverse)
        y = torch.where(ok & (a > 0), y, torch.zeros_like(y))
        code = torch.searchsorted(mid, y.reshape(-1)).reshape(y.shape)
        out.append((table[code] * a).reshape(case["tokens"], h, d))
        pool = torch.zeros_like(st["pool"][key][1], dtype=torch.float64)
        flat = pool.transpose(1, 2).reshape(-1, h, d // b)
        flat[st["slots"]] = a.squeeze(-1)
        stats.append(flat.reshape(pool.shape[0], case["page_size"], h, d // b).transpose(1, 2).contiguous())
    return (*out, *stats)


def _exact_attend(case, st, table):
    h, d, g = case["kv_heads"], case["head_dim"], case["heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    row = 0
    for s, (nq, kv) in enumerate(_lengths(case)):
        rows = slice(row, row + nq)
        row += nq
        if not nq or not kv:
            continue
        pages = st["page_table"][s, : -(-kv // case["page_size"])].long()
        low = torch.arange(nq, device=out.device) + (kv - nq)  # the last key each query sees
        key_at = torch.arange(kv, device=out.device)
        hidden = key_at.unsqueeze(0) > low.unsqueeze(1)
        if case["window"]:
            hidden = hidden | (key_at.unsqueeze(0) <= low.unsqueeze(1) - case["window"])
        for head in range(h):
            side = {}
            for key in ("k", "v"):
                packed, absmax = (t[pages, head] for t in st["pool"][key])
                side[key] = _exact_pool(case, packed, absmax, table).reshape(-1, d)[:kv]
            for j in range(g):
                z = (st["q"][rows, head * g + j].double() @ side["k"].T) * st["scale"]
                z = z.masked_fill(hidden, -math.inf)
                out[rows, head * g + j] = torch.softmax(z, dim=-1) @ side["v"]
    return out
