"""A prompt's way into the paged cache and over it: inputs, plain forms and exact values.

Three operators, each as the program of a serving loop calls it:

``rotate``   RMS norm of every query and key head and the rotation by its position, in one pass; a
             position may have several axes (time, height, width), each turning its own frequencies.
``append``   the same for a step's tokens, whose keys and values go straight into their pages
             (bf16, or e4m3 with one scale for each block and KV head).
``prefill``  attention of many new tokens of each sequence over the pages that hold them and the
             rows before them.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through
``quantized_kv_decode_partial_gb300``.
"""

from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def _rows(name, op, seqs, new_lo, new_hi, kv_heads, rep, head_dim, *, rot=0, base=1e6, adjacent=False, norm=True,
          offset=0.0, axes=1, sections="", turns="blocks", held_lo=0, held_hi=0, bits=16, block_size=32, window=0):
    """``sections``: how many frequencies each axis turns, as text; bits -8: e4m3 with block scales."""
    return {"name": name, "op": op, "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "kv_heads": kv_heads, "rep": rep,
            "head_dim": head_dim, "rot": rot or head_dim, "base": base, "adjacent": adjacent, "norm": norm,
            "offset": offset, "axes": axes, "sections": sections, "turns": turns, "held_lo": held_lo,
            "held_hi": held_hi, "bits": bits, "block_size": block_size, "window": window}


def listed():
    return [
        # one token of one user; latency counts
        _rows("rotate_token", "rotate", 1, 1, 1, 8, 4, 128),
        # images and video beside text: three axes in blocks of frequencies
        _rows("rotate_three_axes", "rotate", 4, 3001, 5003, 4, 7, 128, axes=3, sections="16,24,24"),
        # wide heads of which a part turns, neighbours as pairs, norm weights stored less one
        _rows("rotate_part_d256", "rotate", 2, 4097, 8191, 4, 4, 256, rot=64, base=1e4, adjacent=True, offset=1.0),
        # the next token of a full batch into bf16 pages; latency counts
        _rows("append_token", "append", 64, 1, 1, 8, 4, 128, held_lo=700, held_hi=9000),
        # up to four draft tokens into e4m3 pages; latency counts
        _rows("append_draft_e4m3", "append", 64, 1, 4, 8, 4, 128, held_lo=700, held_hi=9000, bits=-8),
        # whole prompts into bf16 pages, three axes turning by frequencies in turn
        _rows("append_prompt_axes", "append", 8, 1025, 4099, 8, 4, 128, axes=3, sections="24,20,20", turns="cycle"),
        # prompts behind a shared prefix that ends inside a page, into e4m3 pages, no norm
        _rows("append_prompt_e4m3", "append", 8, 2001, 8192, 8, 4, 128, held_lo=5, held_hi=300, bits=-8, norm=False),
        # a short first prompt; latency counts
        _rows("prefill_short", "prefill", 1, 37, 37, 8, 4, 128, held_lo=0, held_hi=0),
        # whole prompts of a batch
        _rows("prefill_prompts", "prefill", 8, 1025, 8192, 8, 4, 128),
        # a chunk of two long documents, pages of 16 rows
        _rows("prefill_chunk_long", "prefill", 2, 500, 1024, 8, 4, 128, held_lo=30011, held_hi=60000, block_size=16),
        # chunks of a mixed batch over e4m3 pages, five query heads to a KV head
        _rows("prefill_mixed_e4m3", "prefill", 16, 1, 512, 8, 5, 128, held_lo=700, held_hi=16000, bits=-8),
        # 256-dim heads over 8-bit affine pages under a sliding window
        _rows("prefill_window_u8_d256", "prefill", 4, 700, 4096, 4, 2, 256, held_lo=0, held_hi=6000, bits=8, window=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        c = _draw(rng)
        if work(c)["flops"] <= most:
            return c


def _draw(rng):
    op = rng.choice(["rotate", "append", "prefill", "prefill"])
    kv_heads, rep = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "prefill":
        bits = rng.choice([16, 16, -8, 8, 4])
        head_dim = rng.choice([64, 128, 128, 256] if bits in (16, -8) else [128, 128, 256])
        seqs = _log_int(rng, 1, 16)
        new_hi = _log_int(rng, 1, max(1, 8192 // seqs))
        held_hi = _log_int(rng, 1, max(1, 65536 // seqs)) if rng.random() < 0.7 else 0
        c = _rows("", op, seqs, rng.randint(1, new_hi), new_hi, kv_heads, rep, head_dim,
                  held_lo=rng.randint(0, held_hi), held_hi=held_hi, bits=bits, block_size=rng.choice([16, 32, 64, 96]) if bits == 16 else
                  rng.choice([32, 64, 96]), window=_log_int(rng, 1, 8192) if rng.random() < 0.2 else 0)
    else:
        head_dim = rng.choice([64, 128, 256])
        half = head_dim // 2 if rng.random() < 0.7 else rng.choice([n for n in (16, 32, 64) if 2 * n <= head_dim])
        axes = rng.choice([1, 1, 2, 3])
        turns = rng.choice(["blocks", "cycle"])
        sections = [half]
        if axes > 1:
            most = half // axes
            others = [rng.randint(max(1, most // 2), most) for _ in range(axes - 1)]
            sections = [half - sum(others)] + others
        seqs = _log_int(rng, 1, 64)
        new_hi = _log_int(rng, 1, max(1, 65536 // seqs // kv_heads))
        bits = rng.choice([16, -8]) if op == "append" else 16
        held_hi = _log_int(rng, 1, max(1, 2 ** 22 // (seqs * kv_heads * 16))) if op == "append" else 0
        c = _rows("", op, seqs, rng.randint(1, new_hi), new_hi, kv_heads, rep, head_dim, rot=2 * half,
                  base=rng.choice([1e4, 5e5, 1e6]), adjacent=rng.random() < 0.3, norm=rng.random() < 0.75,
                  offset=rng.choice([0.0, 0.0, 1.0]), axes=axes, sections=",".join(str(x) for x in sections) if axes > 1 else "",
                  turns=turns, held_lo=rng.randint(0, held_hi), held_hi=held_hi, bits=bits,
                  block_size=rng.choice([16, 32, 64]) if bits == 16 else rng.choice([32, 64, 96]))
    c.pop("name")
    return c


def _spread(lo, hi, count, step):
    """Ragged sizes in [lo, hi], the same for every seed; the first is hi."""
    return [hi if not b else lo + int(round((hi - lo) * ((b * step) % 1.0))) for b in range(count)]


def _sizes(c):
    """New rows and rows held before them of each sequence."""
    return (_spread(c["new_lo"], c["new_hi"], c["seqs"], 0.6180339887),
            _spread(c["held_lo"], c["held_hi"], c["seqs"], 0.7548776662))


def _seen(c):
    """(query, key) pairs of each sequence that the mask lets meet."""
    got = []
    for n, held in zip(*_sizes(c)):
        w, total = c["window"], held + n
        if not w or w >= total:
            got.append(n * held + n * (n + 1) // 2)
        else:
            grow = max(0, min(n, w - held))  # the queries that still see every row
            got.append(grow * held + grow * (grow + 1) // 2 + (n - grow) * w)
    return got


def _row_bytes(c):
    d = c["head_dim"]
    return {16: 2 * d, -8: d, 8: d + d // 16, 4: d // 2 + d // 16}[c["bits"]]


def work(case):
    c = case
    new, held = _sizes(c)
    t, hk, hq, d = sum(new), c["kv_heads"], c["kv_heads"] * c["rep"], c["head_dim"]
    if c["op"] == "rotate":
        return {"bytes": t * (hq + hk) * 4 * d + 4 * t * c["axes"], "flops": 10.0 * t * (hq + hk) * d}
    if c["op"] == "append":
        return {"bytes": t * (hq * 4 * d + 2 * hk * (2 * d + _row_bytes(c))), "flops": 10.0 * t * (hq + hk) * d}
    w = c["window"]
    rows = sum(min(n + h, w + n - 1) if w else n + h for n, h in zip(new, held))
    return {"bytes": t * hq * 4 * d + rows * hk * 2 * _row_bytes(c), "flops": 4.0 * d * hq * sum(_seen(c))}


# ----------------------------------------------------------------------------------------- inputs
class _State:
    pass


def _pages(c, s, lens, gen, dev):
    """Block tables whose pages lie in no order, with some free blocks."""
    pages = [-(-l // c["block_size"]) for l in lens]
    nb = sum(pages) + max(1, sum(pages) // 10)
    perm = torch.randperm(nb, generator=gen, device=dev)
    start = torch.tensor([sum(pages[:b]) for b in range(len(pages))], device=dev)
    col = torch.arange(max(pages), device=dev)
    used = col < torch.tensor(pages, device=dev)[:, None]
    s.tables = torch.where(used, perm[(start[:, None] + col).clamp_(max=nb - 1)], 0).to(torch.int32)
    return nb


def _pool(c, nb, gen, dev):
    """One plane of rows and its scales and biases (None where the format has none)."""
    hk, bs, d, bits = c["kv_heads"], c["block_size"], c["head_dim"], c["bits"]
    if bits == 16:
        return torch.randn((nb, hk, bs, d), generator=gen, device=dev, dtype=torch.bfloat16), None, None
    if bits == -8:
        x = torch.randn((nb, hk, bs, d), generator=gen, device=dev, dtype=torch.bfloat16).mul_(96.0)
        e = torch.randint(-8, -5, (nb, hk), generator=gen, device=dev, dtype=torch.int32)
        return x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), ((e + 127) << 23).view(torch.float32), None
    words = torch.randint(-2 ** 31, 2 ** 31, (nb, hk, bs, d * bits // 32), generator=gen, device=dev, dtype=torch.int32)
    levels = 2 ** bits - 1
    scales = torch.rand((nb, hk, bs, d // 64), generator=gen, device=dev).add_(1.0).mul_(2.5 / levels).to(torch.bfloat16)
    biases = torch.randn((nb, hk, bs, d // 64), generator=gen, device=dev).mul_(0.3).sub_(1.8).to(torch.bfloat16)
    return words, scales, biases


def _positions(c, new, held, gen, dev):
    """One axis: the rows' places. More: text counts on all alike, then a grid whose first axis is its time."""
    cols = []
    for b, n in enumerate(new):
        at = torch.arange(n, device=dev, dtype=torch.int32) + held[b]
        if c["axes"] == 1:
            cols.append(at[None])
            continue
        text = n // 4
        side = max(1, math.isqrt(max(1, n - text)) // 2)
        i = (torch.arange(n, device=dev, dtype=torch.int32) - text).clamp_(min=0)
        grid = [i // (side * side), i // side % side, i % side][:c["axes"]]
        cols.append(torch.stack([torch.where(at < held[b] + text, at, held[b] + text + g) for g in grid]))
    return torch.cat(cols, 1).to(torch.int32).contiguous()


def _sections(c):
    return [int(x) for x in c["sections"].split(",")] if c["axes"] > 1 else [c["rot"] // 2]


def prepare(case, seed):
    c, s = case, _State()
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    new, held = _sizes(c)
    t, hk, hq, d = sum(new), c["kv_heads"], c["kv_heads"] * c["rep"], c["head_dim"]
    s.case, s.scale = c, 1.0 / math.sqrt(d)
    s.error = torch.zeros(1, dtype=torch.int32, device=dev)
    s.starts = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=dev)
    if c["op"] != "rotate":
        lens = [n + h for n, h in zip(new, held)]
        nb = _pages(c, s, lens, gen, dev)
        s.k, s.ks, s.kb = _pool(c, nb, gen, dev)
        s.v, s.vs, s.vb = _pool(c, nb, gen, dev)
    if c["op"] == "prefill":
        s.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        s.q = torch.randn((t, hq, d), generator=gen, device=dev).to(torch.bfloat16)
        s.out = torch.empty_like(s.q)
        return s
    s.lens = torch.tensor(held, dtype=torch.int32, device=dev)
    # a projection's output holds a token's query, key and value heads side by side
    s.qkv = torch.randn((t, (hq + 2 * hk) * d), generator=gen, device=dev, dtype=torch.bfloat16)
    part = s.qkv.view(t, hq + 2 * hk, d)
    s.q, s.k_new, s.v_new = part[:, :hq], part[:, hq:hq + hk], part[:, hq + hk:]
    s.q_out, s.k_out = (torch.empty((t, h, d), dtype=torch.bfloat16, device=dev) for h in (hq, hk))
    s.positions = _positions(c, new, held, gen, dev)
    half = c["rot"] // 2
    s.freq = (c["base"] ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)).float()
    s.wq = s.wk = None
    if c["norm"]:
        s.wq, s.wk = ((torch.randn(d, generator=gen, device=dev) * 0.2 + 1.0 - c["offset"]).to(torch.bfloat16)
                      for _ in range(2))
    return s


# ------------------------------------------------------------------------------------ plain forms
def _axis_of(c, device):
    """The axis that turns each frequency."""
    sections, half = _sections(c), c["rot"] // 2
    i = torch.arange(half, device=device)
    if c["turns"] == "blocks":
        edge = torch.tensor(sections, device=device).cumsum(0)
        return (i[:, None] >= edge).sum(1)
    a = i % len(sections)
    return torch.where(i < len(sections) * torch.tensor(sections, device=device)[a], a, 0)


def _plain_turn(s, x, weight, cos, sin):
    """Norm and rotation of x [T, H, D] in f32."""
    c, half = s.case, s.case["rot"] // 2
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * (weight.float() + c["offset"])
    turned, rest = y[..., :2 * half], y[..., 2 * half:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if c["adjacent"] else (turned[..., :half], turned[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if c["adjacent"] else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1).to(torch.bfloat16)


def _plain_rotate(s):
    # angles of far positions in 64 bits
    angle = s.positions.double()[_axis_of(s.case, s.freq.device)].T * s.freq.double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return [_plain_turn(s, s.q, s.wq, cos, sin), _plain_turn(s, s.k_new, s.wk, cos, sin)]


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (0 for no value but zero)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), torch.zeros_like(amax))


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _token_places(s):
    """Sequence, place in it and physical block of every new row."""
    t = torch.arange(s.q.shape[0], device=s.q.device)
    seq = torch.searchsorted(s.starts[1:].long(), t, right=True)
    at = s.lens.long()[seq] + t - s.starts.long()[seq]
    return seq, at, s.tables[seq, at // s.case["block_size"]].long()


def _plain_write(s, rows, pool, scales):
    c, bs = s.case, s.case["block_size"]
    _, at, phys = _token_places(s)
    if c["bits"] == 16:
        pool[phys, :, at % bs] = rows
        return
    # every touched block once: the scale its new rows need, over the one its earlier rows have
    x = rows.float()
    used, inverse = torch.unique(phys, return_inverse=True)
    amax = torch.zeros((len(used), x.shape[1]), device=x.device)
    amax = amax.index_reduce_(0, inverse, x.abs().amax(-1), "amax")
    first = torch.full((len(used),), bs, device=x.device).index_reduce_(0, inverse, at % bs, "amin")
    before = torch.where((first > 0)[:, None], scales[used], 0.0)
    after = torch.maximum(before, _pow2_scale(amax))
    by = torch.where(after > 0, after, 1.0)
    now = pool.view(torch.uint8)[used]
    kept = _e4m3(now.view(torch.float8_e4m3fn).float() * (before / by)[..., None, None])
    old = (torch.arange(bs, device=x.device) < first[:, None])[:, None, :, None]
    pool.view(torch.uint8)[used] = torch.where(old, kept, now)
    pool.view(torch.uint8)[phys, :, at % bs] = _e4m3(x / by[inverse][..., None])
    scales[used] = after


def _values(c, pool, scales, biases, at):
    """The values of the blocks ``at`` in f32: [len(at), HK, BS, D]."""
    if c["bits"] == 16:
        return pool[at].float()
    if c["bits"] == -8:
        return pool.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scales[at][..., None, None]
    bits, words = c["bits"], pool[at]
    shift = torch.arange(0, 32, bits, device=words.device, dtype=torch.int32)
    codes = ((words[..., None] >> shift) & (2 ** bits - 1)).flatten(-2).float()
    return codes * scales[at].float().repeat_interleave(64, -1) + biases[at].float().repeat_interleave(64, -1)


def _plain_prefill(s):
    c, bs = s.case, s.case["block_size"]
    hk, rep, d = c["kv_heads"], c["rep"], c["head_dim"]
    new, held = _sizes(c)
    out, first = torch.empty_like(s.q), 0
    for b, n in enumerate(new):
        length = held[b] + n
        low = max(0, held[b] + 1 - c["window"]) // bs if c["window"] else 0
        at = s.tables[b, low:-(-length // bs)].long()
        k, v = (_values(c, *p, at).transpose(0, 1).flatten(1, 2)[:, :length - low * bs]
                for p in ((s.k, s.ks, s.kb), (s.v, s.vs, s.vb)))
        pos = torch.arange(low * bs, length, device=at.device)
        step = max(1, min(n, 2 ** 29 // (k.shape[1] * hk * rep)))
        for i in range(0, n, step):
            q = s.q[first + i:first + min(n, i + step)].float()
            m = q.shape[0]
            x = q.view(m, hk, rep, d).permute(1, 2, 0, 3).reshape(hk, rep * m, d)
            score = (torch.matmul(x, k.transpose(1, 2)) * s.scale).view(hk, rep, m, -1)
            here = held[b] + i + torch.arange(m, device=at.device)[:, None]
            hidden = pos > here
            if c["window"]:
                hidden = hidden | (pos <= here - c["window"])
            score.masked_fill_(hidden, float("-inf"))
            score = torch.exp(score.sub_(score.amax(-1, keepdim=True)))
            total = score.sum(-1, keepdim=True)
            o = torch.matmul(score.view(hk, rep * m, -1), v).view(hk, rep, m, d) / total
            out[first + i:first + i + m] = o.permute(2, 0, 1, 3).reshape(m, hk * rep, d).to(torch.bfloat16)
        first += n
    return out


def _run_plain(s):
    if s.case["op"] == "rotate":
        return _plain_rotate(s)
    if s.case["op"] == "prefill":
        return _plain_prefill(s)
    q, k = _plain_rotate(s)
    _plain_write(s, k, s.k, s.ks)
    _plain_write(s, s.v_new, s.v, s.vs)
    return [q, s.k, s.v] + ([] if s.ks is None else [s.ks, s.vs])


# ------------------------------------------------------------------------------------- own kernels
def _run_own(s):
    import quantized_kv_decode_partial_gb300 as pkv

    c = s.case
    block = c["bits"] == -8
    fmt = {"bits": 8 if block else c["bits"], "group_size": pkv.PKV_GROUP_BLOCK if block else 64}
    if c["op"] == "prefill":
        return pkv.paged_prefill_attention(s.q, s.k, s.v, s.tables, s.lens, s.starts, s.scale, window=c["window"],
                                           k_scales=s.ks, k_biases=s.kb, v_scales=s.vs, v_biases=s.vb, out=s.out,
                                           error_flag=s.error, **fmt)
    turn = {"q_weight": s.wq, "k_weight": s.wk, "eps": EPS, "weight_offset": c["offset"],
            "sections": _sections(c) if c["axes"] > 1 else None,
            "section_order": pkv.PKV_SECTIONS_CYCLE if c["turns"] == "cycle" else pkv.PKV_SECTIONS_BLOCKS,
            "pairing": pkv.PKV_PAIRS_ADJACENT if c["adjacent"] else pkv.PKV_PAIRS_HALVES}
    if c["op"] == "rotate":
        return list(pkv.norm_rotate(s.q, s.k_new, s.positions, s.freq, q_out=s.q_out, k_out=s.k_out, **turn))
    # positions on one axis are the rows' places in the cache, which is what the call takes by itself
    q = pkv.norm_rotate_append(s.q, s.k_new, s.v_new, s.positions if c["axes"] > 1 else None, s.freq, s.tables, s.lens,
                               s.k, s.v, query_starts=s.starts, k_scales=s.ks, v_scales=s.vs, q_out=s.q_out,
                               error_flag=s.error, **turn, **fmt)
    return [q, s.k, s.v] + ([] if s.ks is None else [s.ks, s.vs])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------- in 64 bits
def _exact_axis(c, i):
    """The axis of frequency i."""
    sections = _sections(c)
    if c["turns"] == "blocks":
        a = 0
        while i >= sum(sections[:a + 1]):
            a += 1
        return a
    a = i % len(sections)
    return a if i // len(sections) < sections[a] else 0


def _exact_turn(s, x, weight):
    """Pairs as complex numbers, each times e^(i position frequency)."""
    c, half = s.case, s.case["rot"] // 2
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / c["head_dim"] + EPS) * (weight.double() + c["offset"])
    axis = torch.tensor([_exact_axis(c, i) for i in range(half)], device=x.device)
    angle = s.positions.double().index_select(0, axis) * s.freq.double()[:, None]
    unit = torch.polar(torch.ones_like(angle), angle).T[:, None]
    out = y.clone()
    if c["adjacent"]:
        z = torch.view_as_complex(y[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * unit
        out[..., :2 * half] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :half], y[..., half:2 * half]) * unit
        out[..., :half], out[..., half:2 * half] = z.real, z.imag
    return out


def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest_e4m3(x):
    a = x.abs().clamp(max=E4M3_MAX)
    step = _two_to((torch.frexp(a).exponent - 4).clamp(min=-9))
    return torch.copysign(torch.round(a / step) * step, x)


def _exact_write(s, rows, pool, scales):
    """Each sequence's rows into its blocks, one block after the other."""
    c, bs = s.case, s.case["block_size"]
    values = pool.float().double()
    scale_out = None if scales is None else scales.double()
    new, held = _sizes(c)
    tables, first = s.tables.tolist(), 0
    for b, n in enumerate(new):
        end = held[b] + n
        for j in range(held[b] // bs, (end - 1) // bs + 1):
            phys = tables[b][j]
            lo, hi = max(held[b], j * bs), min(end, (j + 1) * bs)
            part = rows[first + lo - held[b]:first + hi - held[b]].transpose(0, 1)
            place = slice(lo - j * bs, hi - j * bs)
            if scales is None:
                values[phys, :, place] = part
                continue
            top = part.abs().amax((1, 2))
            need = torch.where(top > 0, _two_to(torch.ceil(torch.log2(top / E4M3_MAX))), 0.0)
            before = scale_out[phys] if lo > j * bs else torch.zeros_like(need)
            after = torch.maximum(before, need)
            div = torch.where(after > 0, after, 1.0)[:, None, None]
            if lo > j * bs:
                old = values[phys, :, :lo - j * bs]
                values[phys, :, :lo - j * bs] = _nearest_e4m3(old * (before[:, None, None] / div))
            values[phys, :, place] = _nearest_e4m3(part / div)
            scale_out[phys] = after
        first += n
    return values, scale_out


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


def _exact_prefill(s):
    c, bs = s.case, s.case["block_size"]
    new, held = _sizes(c)
    res, first = torch.empty(s.q.shape, dtype=torch.float64, device=s.q.device), 0
    for b, n in enumerate(new):
        blk = s.tables[b, :-(-(held[b] + n) // bs)].long()
        for h in range(c["kv_heads"]):
            k, v = (_stored(c, *p, blk, h)[:held[b] + n] for p in ((s.k, s.ks, s.kb), (s.v, s.vs, s.vb)))
            for i in range(0, n, 512):
                m = min(512, n - i)
                end = held[b] + i + m
                begin = max(0, held[b] + i + 1 - c["window"]) if c["window"] else 0
                gap = torch.arange(held[b] + i, end, device=s.q.device)[:, None] - torch.arange(begin, end, device=s.q.device)
                seen = gap >= 0
                if c["window"]:
                    seen &= gap < c["window"]
                for r in range(h * c["rep"], (h + 1) * c["rep"]):
                    x = s.q[first + i:first + i + m, r].double() @ k[begin:end].T * s.scale
                    res[first + i:first + i + m, r] = torch.softmax(torch.where(seen, x, -math.inf), -1) @ v[begin:end]
        first += n
    return res


def exact(case, seed):
    c = case
    if c["op"] == "prefill":
        if work(c)["flops"] > 5e12:
            return None
        return _exact_prefill(prepare(c, seed))
    if c["op"] == "append" and sum(n // c["block_size"] + 2 for n in _sizes(c)[0]) > 8000:
        return None
    s = prepare(c, seed)
    q, k = _exact_turn(s, s.q, s.wq), _exact_turn(s, s.k_new, s.wk)
    if c["op"] == "rotate":
        return [q, k]
    # the keys that are written are rounded to bf16 first, in every format
    pages = [_exact_write(s, rows, pool, scales) for rows, pool, scales in
             ((k if s.ks is None else k.to(torch.bfloat16).double(), s.k, s.ks), (s.v_new.double(), s.v, s.vs))]
    return [q, pages[0][0], pages[1][0]] + ([] if s.ks is None else [pages[0][1], pages[1][1]])
