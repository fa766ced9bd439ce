"""Long-context serving operators over the paged cache: inputs, plain forms and exact values.

Four operators, each as the program of a serving loop calls it:

``append8``  writes new K/V rows into pages held in 8 bits (e4m3) with one f32 scale for each block
             and KV head; the scale is a power of two that grows when a later row needs it.
``attend8``  decode attention over such pages.
``bounds``   keeps, for each block and KV head, the elementwise smallest and largest key of the rows.
``sparse``   scores every block by the largest product any of its keys could have with a query,
             takes the best ``top_k`` for each (sequence, KV head) and attends over those alone.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through
``quantized_kv_decode_partial_gb300``.
"""

from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------ cases
def _case(name, op, seqs, kv_heads, head_dim, block_size, len_lo, len_hi, *, rep=4, n_query=1, bits=16, n_new=0,
          top_k=0, first=1, last=1, window=0):
    if op in ("attend8", "append8"):
        bits = -8  # e4m3 with a scale for each block and KV head
    return {"name": name, "op": op, "seqs": seqs, "kv_heads": kv_heads, "head_dim": head_dim,
            "block_size": block_size, "len_lo": len_lo, "len_hi": len_hi, "rep": rep, "n_query": n_query,
            "bits": bits, "n_new": n_new, "top_k": top_k, "first": first, "last": last, "window": window}


def listed():
    return [
        # one user's chat turn: a single sequence, a token at a time; latency counts
        _case("attend8_one", "attend8", 1, 4, 256, 32, 8192, 8192),
        # a full serving batch of ragged lengths: the cache is the traffic
        _case("attend8_batch64", "attend8", 64, 8, 128, 32, 1024, 32768),
        # draft tokens checked four at a time over long contexts, in small pages
        _case("attend8_spec4", "attend8", 8, 8, 128, 16, 20001, 40003, n_query=4),
        # the batch's next token written into pages that hold others already; latency counts
        _case("append8_token", "append8", 64, 8, 128, 32, 777, 9000, n_new=1),
        # prompts written behind a shared prefix that ends inside a page
        _case("append8_prompt", "append8", 8, 8, 128, 32, 5, 300, n_new=8192),
        # the bounds of whole prompts, once they are in the cache
        _case("bounds_prompt", "bounds", 8, 8, 128, 32, 32001, 32768, n_new=32768),
        # the bounds after one more token; latency counts
        _case("bounds_token", "bounds", 64, 8, 256, 32, 1000, 30000, bits=8, n_new=1),
        # the bounds after a chunk of a prompt, in 8-bit pages
        _case("bounds_chunk_e4m3", "bounds", 16, 8, 128, 32, 700, 16001, bits=-8, n_new=512),
        # one user with a long document: blocks chosen from 32768 rows; latency counts
        _case("sparse_one", "sparse", 1, 8, 128, 32, 32768, 32768, top_k=64),
        # eight very long contexts, four draft tokens each, in pages of 16 rows
        _case("sparse_long_n4", "sparse", 8, 8, 128, 16, 131072, 131072, n_query=4, top_k=256, last=2),
        # a serving batch over 8-bit pages, some sequences shorter than the budget
        _case("sparse_batch64_e4m3", "sparse", 64, 8, 128, 32, 1024, 32768, bits=-8, top_k=64),
        # 4-bit pages of 256-dim heads, two draft tokens
        _case("sparse_u4_d256", "sparse", 16, 4, 256, 32, 4001, 20011, bits=4, n_query=2, top_k=48, first=2, last=3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend8", "append8", "bounds", "sparse"])
    head_dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    seqs = _log_int(rng, 1, 64)
    bits = rng.choice([16, -8, 8, 4]) if op in ("bounds", "sparse") else -8
    if bits in (8, 4) and head_dim == 64:
        head_dim = 128
    n_query = rng.choice([1, 1, 2, 4])
    rep = rng.choice([1, 2, 3, 4, 5, 8]) if op in ("attend8", "sparse") else 4
    block_size = rng.choice([16, 32, 64]) if bits == 16 else rng.choice([32, 64, 96])
    most = max(64, min(32768, 2 ** 28 // (seqs * kv_heads * head_dim)))
    len_hi = _log_int(rng, n_query, most)
    len_lo = rng.randint(n_query, len_hi) if len_hi > n_query else len_hi
    n_new = 0
    top_k, first, last, window = 0, 1, 1, 0
    if op == "append8":
        n_new = _log_int(rng, 1, max(1, min(len_hi, 65535)))
    elif op == "bounds":
        n_new = _log_int(rng, 1, len_hi)
    elif op == "sparse":
        first = rng.choice([0, 1, 2])
        last = 1 + (n_query - 1 + block_size - 1) // block_size + rng.choice([0, 1, 3])
        top_k = first + last + _log_int(rng, 1, 200)
    elif rng.random() < 0.25:
        window = _log_int(rng, 1, 8192)
    return {k: v for k, v in _case("", op, seqs, kv_heads, head_dim, block_size, len_lo, len_hi, rep=rep,
                                   n_query=n_query, bits=bits, n_new=n_new, top_k=top_k, first=first, last=last,
                                   window=window).items() if k != "name"}


def _lengths(c):
    """Ragged lengths in [len_lo, len_hi], the same for every seed."""
    span = c["len_hi"] - c["len_lo"]
    return [c["len_lo"] + int(round(span * ((b * 0.6180339887) % 1.0))) if b else c["len_hi"] for b in range(c["seqs"])]


def _row_bytes(c):
    d = c["head_dim"]
    return {16: 2 * d, -8: d, 8: d + d // 16, 4: d // 2 + d // 16}[c["bits"]]


def work(case):
    c = case
    lens, hk, d, bs, n = _lengths(c), c["kv_heads"], c["head_dim"], c["block_size"], c["n_query"]
    hq = hk * c["rep"]
    io = 2 * c["seqs"] * hq * n * d * 2  # queries in, outputs out (bf16)
    if c["op"] == "attend8":
        rows = [min(l, c["window"] + n - 1) if c["window"] else l for l in lens]
        blocks = sum(-(-r // bs) for r in rows)
        return {"bytes": io + hk * (sum(rows) * 2 * d + blocks * 8), "flops": 4.0 * d * n * hq * sum(rows)}
    if c["op"] == "append8":
        values = 2 * c["seqs"] * hk * c["n_new"] * d
        return {"bytes": 3 * values + 8 * hk * c["seqs"] * (1 + c["n_new"] // bs), "flops": 2.0 * values}
    if c["op"] == "bounds":
        rows = sum(min(l, c["n_new"]) for l in lens)
        blocks = sum((l - 1) // bs - max(0, l - c["n_new"]) // bs + 1 for l in lens)
        return {"bytes": hk * (rows * _row_bytes(c) + blocks * 4 * d), "flops": 2.0 * hk * rows * d}
    blocks = sum(-(-l // bs) for l in lens)
    rows = sum(min(l, c["top_k"] * bs) for l in lens)
    return {"bytes": io + hk * (blocks * 4 * d + rows * 2 * _row_bytes(c)),
            "flops": 4.0 * d * n * hq * (blocks + rows)}


# ----------------------------------------------------------------------------------------- inputs
class _State:
    pass


def _codes(shape, gen, dev):
    # values whose block spreads over the type's range, as the writer leaves them
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16).mul_(96.0).clamp_(-E4M3_MAX, E4M3_MAX)
    return x.to(torch.float8_e4m3fn)


def _block_scales(nb, hk, gen, dev):
    e = torch.randint(-8, -5, (nb, hk), generator=gen, device=dev, dtype=torch.int32)
    return ((e + 127) << 23).view(torch.float32)


def _pool(c, nb, gen, dev):
    """One plane of rows and its scales and biases (None where the format has none)."""
    hk, bs, d, bits = c["kv_heads"], c["block_size"], c["head_dim"], c["bits"]
    if bits == 16:
        # keys of one block lie near one another, so that blocks differ for a query
        x = torch.randn((nb, hk, bs, d), generator=gen, device=dev, dtype=torch.bfloat16)
        return x.add_(torch.randn((nb, hk, 1, d), generator=gen, device=dev, dtype=torch.bfloat16).mul_(0.5)), None, None
    if bits == -8:
        return _codes((nb, hk, bs, d), gen, dev), _block_scales(nb, hk, gen, dev), None
    words = torch.randint(-2 ** 31, 2 ** 31, (nb, hk, bs, d * bits // 32), generator=gen, device=dev, dtype=torch.int32)
    levels = 2 ** bits - 1
    s = torch.rand((nb, hk, bs, d // 64), generator=gen, device=dev).add_(1.0).mul_(2.5 / levels).to(torch.bfloat16)
    z = torch.randn((nb, hk, bs, d // 64), generator=gen, device=dev).mul_(0.3).sub_(1.8).to(torch.bfloat16)
    return words, s, z


def prepare(case, seed):
    c, s = case, _State()
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    lens = _lengths(c)
    bs, hk, d, n = c["block_size"], c["kv_heads"], c["head_dim"], c["n_query"]
    held = [l + c["n_new"] for l in lens] if c["op"] == "append8" else lens
    pages = [-(-l // bs) for l in held]
    nb = sum(pages) + max(1, sum(pages) // 10)  # some free blocks, the others in no order
    perm = torch.randperm(nb, generator=gen, device=dev)
    width = max(pages)
    start = torch.tensor([sum(pages[:b]) for b in range(len(pages))], device=dev)
    col = torch.arange(width, device=dev)
    used = col < torch.tensor(pages, device=dev)[:, None]
    s.tables = torch.where(used, perm[(start[:, None] + col).clamp_(max=nb - 1)], 0).to(torch.int32)
    s.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    s.case, s.scale = c, 1.0 / math.sqrt(d)
    s.k, s.ks, s.kb = _pool(c, nb, gen, dev)
    if c["op"] != "bounds":
        s.v, s.vs, s.vb = _pool(c, nb, gen, dev)
    s.error = torch.zeros(1, dtype=torch.int32, device=dev)
    if c["op"] in ("attend8", "sparse"):
        s.q = torch.randn((c["seqs"], hk * c["rep"], n, d), generator=gen, device=dev).to(torch.bfloat16)
        s.out = torch.empty_like(s.q)
    if c["op"] == "append8":
        shape = (c["seqs"], hk, c["n_new"], d)
        s.k_new = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
        s.v_new = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    if c["op"] in ("bounds", "sparse"):
        s.bounds = torch.zeros((nb, hk, 2, d), dtype=torch.bfloat16, device=dev)
        # the state that earlier calls left (for a prompt there is none, and nothing of it is used)
        every = torch.arange(nb, device=dev, dtype=torch.int32)[:, None]
        full = torch.full((nb,), bs, dtype=torch.int32, device=dev)
        if c["op"] == "sparse":
            s.bounds = _bounds(c, s.k, s.ks, s.kb, every, full, s.bounds, bs)
        else:
            most = _log2_floor(bs)  # the first rows of every block, so that later rows still widen some bounds
            s.bounds = _bounds(c, s.k, s.ks, s.kb, every, torch.full_like(full, most), s.bounds, bs)
    s.blocks = torch.empty((c["seqs"], hk, max(1, c["top_k"])), dtype=torch.int32, device=dev)
    return s


def _log2_floor(x):
    return max(1, x.bit_length() - 1)


# ------------------------------------------------------------------------------------ plain forms
def _values(c, pool, scales, biases, at, heads=None):
    """The values of the blocks ``at`` (of all KV heads, or of ``heads``) in f32: [..., BS, D]."""
    pick = (at,) if heads is None else (at, heads)
    if c["bits"] == 16:
        return pool[pick].float()
    if c["bits"] == -8:
        x = pool.view(torch.uint8)[pick].view(torch.float8_e4m3fn).float()
        return x * scales[pick][..., None, None]
    bits, words = c["bits"], pool[pick]
    shift = torch.arange(0, 32, bits, device=words.device, dtype=torch.int32)
    codes = ((words[..., None] >> shift) & (2 ** bits - 1)).flatten(-2).float()
    return codes * scales[pick].float().repeat_interleave(64, -1) + biases[pick].float().repeat_interleave(64, -1)


def _attend(c, q, k, v, pos, lens, scale):
    """Softmax attention in f32. k, v: [B, HK, L, D]; pos [B, 1 or HK, L]: the rows' places (or past the length)."""
    b, hq, n, d = q.shape
    hk = c["kv_heads"]
    s = torch.matmul(q.float().reshape(b, hk, hq // hk * n, d), k.transpose(-1, -2)) * scale
    at = (lens.long()[:, None] - n + torch.arange(n, device=q.device)).repeat(1, hq // hk)[:, None, :, None]
    seen = pos[:, :, None, :] <= at
    if c["window"]:
        seen = seen & (pos[:, :, None, :] > at - c["window"])
    s = s.masked_fill(~seen, float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.reshape(b, hq, n, d).to(torch.bfloat16)


def _plain_attend8(s):
    c = s.case
    b, w = s.tables.shape
    at = s.tables.long()
    k = _values(c, s.k, s.ks, s.kb, at).transpose(1, 2).flatten(2, 3)
    v = _values(c, s.v, s.vs, s.vb, at).transpose(1, 2).flatten(2, 3)
    pos = torch.arange(w * c["block_size"], device=at.device).expand(b, 1, -1)
    return _attend(c, s.q, k, v, pos, s.lens, s.scale)


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (0 for no value but zero)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), torch.zeros_like(amax))


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _touched(c, tables, first_row, end_row, most):
    """Blocks [first_row // BS, ...] of each sequence: block ids, each row's place, which blocks hold rows."""
    bs = c["block_size"]
    t = min((bs - 1 + most - 1) // bs + 1, tables.shape[1])
    blk = first_row[:, None] // bs + torch.arange(t, device=tables.device)
    live = blk * bs < end_row[:, None]
    # a block past the end stands for the sequence's first one, and is written as that is
    use = torch.where(live, torch.arange(t, device=tables.device).expand_as(blk), 0)
    blk = blk.gather(1, use)
    phys = tables.long().gather(1, blk.clamp(max=tables.shape[1] - 1))
    pos = blk[:, :, None] * bs + torch.arange(bs, device=tables.device)
    return phys, blk, pos


def _plain_append_plane(c, new, pool, scales, tables, lens):
    first, n = lens.long(), c["n_new"]
    phys, blk, pos = _touched(c, tables, first, first + n, n)
    begin = first[:, None, None]
    is_new = ((pos >= begin) & (pos < begin + n))[:, :, None, :, None]
    is_old = (pos < begin)[:, :, None, :, None]
    rows = torch.arange(new.shape[0], device=new.device)[:, None, None]
    x = new.transpose(1, 2)[rows, (pos - begin).clamp(0, n - 1)].float().transpose(2, 3)  # [B, T, HK, BS, D]
    need = _pow2_scale(torch.where(is_new, x.abs(), 0.0).amax((-1, -2)))
    held = (blk * c["block_size"] < first[:, None])[:, :, None]
    before = torch.where(held, scales[phys], 0.0)
    after = torch.maximum(before, need)
    by = torch.where(after > 0, after, 1.0)
    now = pool.view(torch.uint8)[phys]
    kept = _e4m3(now.view(torch.float8_e4m3fn).float() * (before / by)[..., None, None])
    put = _e4m3(x / by[..., None, None])
    pool.view(torch.uint8)[phys] = torch.where(is_new, put, torch.where(is_old, kept, now))
    scales[phys] = after


def _outward(x, up):
    """f32 to bf16, never towards the middle: down (up = False) or up."""
    i = x.contiguous().view(torch.int32)
    cut = i & -65536
    away = (i < 0) if not up else (i >= 0)
    cut = torch.where((cut != i) & away, cut + 65536, cut)
    return cut.view(torch.float32).to(torch.bfloat16)


def _bounds(c, pool, scales, biases, tables, lens, bounds, n_new):
    bs, end = c["block_size"], lens.long()
    first = (end - n_new).clamp(min=0)
    if c["bits"] == -8:  # a block whose scale grew holds its earlier rows anew: it is taken whole
        first = first // bs * bs
    phys, blk, pos = _touched(c, tables, first, end, n_new + (bs if c["bits"] == -8 else 0))
    x = _values(c, pool, scales, biases, phys)
    inside = ((pos >= first[:, None, None]) & (pos < end[:, None, None]))[:, :, None, :, None]
    lo = torch.where(inside, x, float("inf")).amin(-2)
    hi = torch.where(inside, x, float("-inf")).amax(-2)
    partly = (blk * bs < first[:, None])[:, :, None, None]
    held = bounds[phys].float()
    lo = torch.where(partly, torch.minimum(lo, held[..., 0, :]), lo)
    hi = torch.where(partly, torch.maximum(hi, held[..., 1, :]), hi)
    bounds[phys] = torch.stack((_outward(lo, False), _outward(hi, True)), -2)
    return bounds


def _plain_sparse(s):
    c = s.case
    b, hq, n, d = s.q.shape
    hk, bs, top = c["kv_heads"], c["block_size"], c["top_k"]
    at, w = s.tables.long(), s.tables.shape[1]
    # scores in 64 bits: which of two near blocks is taken must not hang on the order of a sum
    box = s.bounds[at].permute(0, 2, 3, 4, 1).double()  # [B, HK, 2, D, W]
    q = s.q.double().reshape(b, hk, hq // hk * n, d)
    score = (torch.matmul(q.clamp(max=0), box[:, :, 0]) + torch.matmul(q.clamp(min=0), box[:, :, 1])).amax(2)
    blocks = ((s.lens.long() + bs - 1) // bs)[:, None, None]
    j = torch.arange(w, device=at.device)
    score = torch.where((j < c["first"]) | (j >= blocks - c["last"]), float("inf"), score)
    score = torch.where(j < blocks, score, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    order = torch.where(torch.arange(order.shape[-1], device=at.device) < blocks, order, w)
    order = torch.sort(order, dim=-1).values
    chosen = torch.where(order < w, order, -1)
    chosen = torch.nn.functional.pad(chosen, (0, top - chosen.shape[-1]), value=-1).to(torch.int32)
    phys = at[:, None, :].expand(b, hk, w).gather(2, order.clamp(max=w - 1))
    heads = torch.arange(hk, device=at.device)[None, :, None]
    k = _values(c, s.k, s.ks, s.kb, phys, heads).flatten(2, 3)
    v = _values(c, s.v, s.vs, s.vb, phys, heads).flatten(2, 3)
    pos = (order[..., None] * bs + torch.arange(bs, device=at.device)).flatten(2)
    return [chosen, _attend(c, s.q, k, v, pos, s.lens, s.scale)]


def _run_plain(s):
    op = s.case["op"]
    if op == "attend8":
        return _plain_attend8(s)
    if op == "append8":
        _plain_append_plane(s.case, s.k_new, s.k, s.ks, s.tables, s.lens)
        _plain_append_plane(s.case, s.v_new, s.v, s.vs, s.tables, s.lens)
        return [s.k, s.v, s.ks, s.vs]
    if op == "bounds":
        return _bounds(s.case, s.k, s.ks, s.kb, s.tables, s.lens, s.bounds, s.case["n_new"])
    return _plain_sparse(s)


# ------------------------------------------------------------------------------------- own kernels
def _run_own(s):
    import quantized_kv_decode_partial_gb300 as pkv

    c = s.case
    block = c["bits"] == -8
    fmt = {"bits": 8 if block else c["bits"], "group_size": pkv.PKV_GROUP_BLOCK if block else 64}
    if c["op"] == "attend8":
        return pkv.paged_decode_attention(s.q, s.k, s.v, s.tables, s.lens, s.scale, k_scales=s.ks, v_scales=s.vs,
                                          window=c["window"], error_flag=s.error, **fmt)
    if c["op"] == "append8":
        pkv.paged_append(s.k_new, s.v_new, s.tables, s.lens, s.k, s.v, k_scales=s.ks, v_scales=s.vs,
                         error_flag=s.error, **fmt)
        return [s.k, s.v, s.ks, s.vs]
    if c["op"] == "bounds":
        return pkv.update_block_bounds(s.k, s.tables, s.lens, s.bounds, n_new=c["n_new"], k_scales=s.ks,
                                       k_biases=s.kb, error_flag=s.error, **fmt)
    out = pkv.sparse_decode_attention(s.q, s.k, s.v, s.bounds, s.tables, s.lens, s.scale, top_k=c["top_k"],
                                      first_blocks=c["first"], last_blocks=c["last"], k_scales=s.ks, k_biases=s.kb,
                                      v_scales=s.vs, v_biases=s.vb, blocks=s.blocks, error_flag=s.error, **fmt)
    return [s.blocks, out]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------- in 64 bits
def _stored(c, pool, scales, biases, blk, h):
    """Rows of the blocks ``blk`` of KV head ``h`` in 64 bits: [len(blk) * BS, D]."""
    x = pool.view(torch.uint8)[blk, h].view(pool.dtype)
    if c["bits"] == 16:
        return x.double().flatten(0, 1)
    if c["bits"] == -8:
        return (x.double() * scales[blk, h].double()[:, None, None]).flatten(0, 1)
    per = 32 // c["bits"]
    unsigned = x.long() & 0xFFFFFFFF
    codes = torch.stack([unsigned // 2 ** (c["bits"] * i) % 2 ** c["bits"] for i in range(per)], -1).flatten(-2)
    g = codes.unflatten(-1, (-1, 64)).double()
    return (g * scales[blk, h].double()[..., None] + biases[blk, h].double()[..., None]).flatten(-2).flatten(0, 1)


def _softmax_rows(c, q, keys, values, places, length, scale):
    """q [rep, n, d] against rows at ``places`` of one KV head, query i at place length - n + i."""
    out = torch.empty(q.shape[:-1] + values.shape[-1:], dtype=torch.float64, device=q.device)
    for i in range(q.shape[1]):
        here = length - q.shape[1] + i
        seen = places <= here
        if c["window"]:
            seen &= places > here - c["window"]
        out[:, i] = torch.softmax(q[:, i].double() @ keys[seen].T * scale, -1) @ values[seen]
    return out


def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest_e4m3(x):
    a = x.abs().clamp(max=E4M3_MAX)
    step = _two_to((torch.frexp(a).exponent - 4).clamp(min=-9))
    return torch.copysign(torch.round(a / step) * step, x)


def _exact_append(c, new, pool, scales, tables, lens):
    values = pool.float().double()
    scale_out, bs = scales.double(), c["block_size"]
    for b, length in enumerate(lens):
        x = new[b].double()
        for j in range(length // bs, (length + c["n_new"] - 1) // bs + 1):
            phys = int(tables[b][j])
            lo, hi = max(length, j * bs), min(length + c["n_new"], (j + 1) * bs)
            part = x[:, lo - length:hi - length]
            top = part.abs().amax((1, 2))
            need = torch.where(top > 0, _two_to(torch.ceil(torch.log2(top / E4M3_MAX))), 0.0)
            before = scale_out[phys] if lo > j * bs else torch.zeros_like(need)
            after = torch.maximum(before, need)
            div = torch.where(after > 0, after, 1.0)[:, None, None]
            if lo > j * bs:
                old = values[phys, :, :lo - j * bs]
                values[phys, :, :lo - j * bs] = _nearest_e4m3(old * (before[:, None, None] / div))
            values[phys, :, lo - j * bs:hi - j * bs] = _nearest_e4m3(part / div)
            scale_out[phys] = after
    return values, scale_out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    lens, bs, hk, n = _lengths(c), c["block_size"], c["kv_heads"], c["n_query"]
    dev = s.tables.device
    if c["op"] == "append8":
        if c["seqs"] * (2 + c["n_new"] // bs) > 8000:
            return None
        tables = s.tables.tolist()
        k, ks = _exact_append(c, s.k_new, s.k, s.ks, tables, lens)
        v, vs = _exact_append(c, s.v_new, s.v, s.vs, tables, lens)
        return [k, v, ks, vs]
    if c["op"] == "bounds":
        if sum(lens) * hk * c["head_dim"] > 2 ** 31:
            return None
        out = s.bounds.double()
        for b, length in enumerate(lens):
            first = max(0, length - c["n_new"])
            j0 = first // bs
            blk = s.tables[b, j0:-(-length // bs)].long()
            for h in range(hk):
                rows = _stored(c, s.k, s.ks, s.kb, blk, h)[:length - j0 * bs]
                for lo, hi, at in _spans(c, first, length, j0, len(blk)):
                    part = rows[lo:hi].unflatten(0, (at[1] - at[0], -1))
                    low, high = part.amin(1), part.amax(1)
                    to = blk[at[0]:at[1]]
                    if c["bits"] != -8 and at[0] == 0 and first % bs:  # rows of earlier calls stay within
                        low, high = torch.minimum(low, out[to, h, 0]), torch.maximum(high, out[to, h, 1])
                    out[to, h, 0], out[to, h, 1] = low, high
        return out
    res = torch.empty(s.q.shape, dtype=torch.float64, device=dev)
    for b, length in enumerate(lens):
        blk = s.tables[b, :-(-length // bs)].long()
        for h in range(hk):
            rows = slice(h * c["rep"], (h + 1) * c["rep"])
            at, j = blk, torch.arange(len(blk), device=dev)
            if c["op"] == "sparse":
                j = _exact_choice(c, s.q[b, rows].double().flatten(0, 1), s.bounds[blk, h].double())
                at = blk[j]
            places = (j[:, None] * bs + torch.arange(bs, device=dev)).flatten()
            keys, values = (_stored(c, *p, at, h) for p in ((s.k, s.ks, s.kb), (s.v, s.vs, s.vb)))
            res[b, rows] = _softmax_rows(c, s.q[b, rows], keys, values, places, length, s.scale)
    return res if c["op"] == "attend8" else [None, res]


def _spans(c, first, length, j0, count):
    """Runs of blocks with equally many new rows: (row range, block range) counted from block j0."""
    bs = c["block_size"]
    begin = 0 if c["bits"] == -8 else first - j0 * bs
    end, got = length - j0 * bs, []
    if count == 1:
        return [(begin, end, (0, 1))]
    got.append((begin, bs, (0, 1)))
    if count > 2:
        got.append((bs, (count - 1) * bs, (1, count - 1)))
    got.append(((count - 1) * bs, end, (count - 1, count)))
    return got


def _exact_choice(c, q, box):
    count = box.shape[0]
    if count <= c["top_k"]:
        return torch.arange(count, device=box.device)
    best = torch.full((count,), -math.inf, dtype=torch.float64, device=box.device)
    for r in range(q.shape[0]):
        best = torch.maximum(best, torch.maximum(q[r] * box[:, 0], q[r] * box[:, 1]).sum(-1))
    best[:c["first"]] = math.inf
    best[count - c["last"]:] = math.inf
    return torch.sort(best, descending=True, stable=True).indices[:c["top_k"]].sort().values
