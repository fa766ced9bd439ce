"""A prompt's write and attention at the edges: offsets past 32 bits, many sequences, overlapping graphs, in place.

Each case against the same call where nothing is at an edge, bit for bit: the arithmetic of one query row or cache row
does not depend on where its rows lie or on what other sequences there are.
"""

import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCK = dict(bits=8, group_size=pkv.PKV_GROUP_BLOCK)
FORMATS = [dict(), BLOCK, dict(bits=8), dict(bits=4)]
D = 128


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def freqs():
    return (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(torch.float32).to(DEV)


def pages(fmt, nb, hk, bs):
    """Pools and planes; only some of their blocks are ever looked at, so no others are filled in."""
    bits = fmt.get("bits", 16)
    if fmt is BLOCK:
        pools = [torch.empty(nb, hk, bs, D, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in "kv"]
        return pools, {n: torch.zeros(nb, hk, device=DEV) for n in ("k_scales", "v_scales")}
    if bits == 16:
        return [torch.empty(nb, hk, bs, D, dtype=torch.bfloat16, device=DEV) for _ in "kv"], {}
    pools = [torch.empty(nb, hk, bs, D * bits // 32, dtype=torch.int32, device=DEV) for _ in "kv"]
    return pools, {n: torch.empty(nb, hk, bs, D // 64, dtype=torch.bfloat16, device=DEV)
                   for n in ("k_scales", "k_biases", "v_scales", "v_biases")}


def write_and_attend(fmt, nb, hk, bs, tables, proj, hq, news, held, **kw):
    """A first write of `held` rows and a second one of `news`, then attention of those; the queries, the outputs and the
    bytes of the blocks in `tables`."""
    T, f, err = proj.shape[0], freqs(), torch.zeros(1, dtype=torch.int32, device=DEV)
    q, k, v = (x.unflatten(1, (-1, D)) for x in proj.split([hq * D, hk * D, hk * D], 1))
    pools, planes = pages(fmt, nb, hk, bs)
    used = tables[tables >= 0].long()
    for t in pools + list(planes.values()):
        t.view(torch.uint8)[used] = 0
    args = dict(error_flag=err, **planes, **fmt)
    ends = lambda x: i32([0] + torch.tensor(x).cumsum(0).tolist())
    assert T >= sum(held) + sum(news)
    a, b = slice(0, sum(held)), slice(sum(held), sum(held) + sum(news))
    pkv.norm_rotate_append(q[a], k[a], v[a], None, f, tables, i32([0] * len(held)), *pools, query_starts=ends(held), **args)
    q2 = pkv.norm_rotate_append(q[b], k[b], v[b], None, f, tables, i32(held), *pools, query_starts=ends(news), **args)
    out = pkv.paged_prefill_attention(q2, *pools, tables, i32([x + y for x, y in zip(held, news)]), ends(news), 0.09, **args, **kw)
    assert int(err) == 0
    return q2, out, [t.view(torch.uint8)[used] for t in pools + list(planes.values())]


@pytest.mark.parametrize("reading", [pkv.PKV_READING_DIRECT, pkv.PKV_READING_VALUES])
@pytest.mark.parametrize("fmt", FORMATS)
def test_blocks_past_32_bits(fmt, reading):
    if fmt.get("bits") and fmt is not BLOCK and reading == pkv.PKV_READING_DIRECT:
        return  # refused
    hq, hk, bs, held, news = 16, 8, 256, [300, 0, 511], [260, 33, 1]
    proj = randn(sum(held) + sum(news), (hq + 2 * hk) * D, seed=1)
    near = i32([[0, 1, 2], [3, -1, -1], [4, 5, -1]])
    want = write_and_attend(fmt, 6, hk, bs, near, proj, hq, news, held, reading=reading)
    # a block is 2^18 values: the last ones begin beyond 2^31 values, of codes of four bits beyond 2^31 bytes as well
    blocks = (1 << 14) + 100 if fmt.get("bits") == 4 else (1 << 13) + 100
    far = torch.where(near >= 0, near + blocks - 6, near)
    got = write_and_attend(fmt, blocks, hk, bs, far, proj, hq, news, held, reading=reading)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(x, y) for x, y in zip(got[2], want[2]))


def test_strides_past_32_bits():
    step = (1 << 31) + 8 * 1001
    room = torch.empty(step + 5 * 4 * D, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(step + 5 * 4 * D, dtype=torch.bfloat16, device=DEV)
    far, to = (x.as_strided((2, 5, 4, D), (step, 4 * D, D, 1)) for x in (room, out))
    q, f = randn(2, 5, 4, D, seed=2), freqs()
    far.copy_(q)
    pos = i32([[0, 1, 2, 3, 4], [70, 71, 72, 73, 74]])
    want, _ = pkv.norm_rotate(q, None, pos, f)
    got, _ = pkv.norm_rotate(far, None, pos, f, q_out=to)
    assert torch.equal(got, want)
    # attention of two tokens that far apart
    pool = [randn(4, 2, 32, D, seed=3 + i) for i in range(2)]
    tables, lens, starts = i32([[0, 1, 2, 3]]), i32([100]), i32([0, 2])
    want = pkv.paged_prefill_attention(want[:, 0].contiguous(), *pool, tables, lens, starts, 0.09)
    assert torch.equal(pkv.paged_prefill_attention(to[:, 0], *pool, tables, lens, starts, 0.09), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", [128, 129, 1100])
def test_many_sequences(fmt, B):
    """Alone, each sequence gets the same queries, pages and (up to the order of sums over splits, so one split) outputs."""
    hq, hk, bs = 6, 2, 16
    g = torch.Generator().manual_seed(B)
    held = torch.randint(0, 40, (B,), generator=g).tolist()
    news = [n if n != 4 else 90 for n in torch.randint(0, 5, (B,), generator=g).tolist()]
    proj = randn(sum(held) + sum(news), (hq + 2 * hk) * D, seed=B)
    per = [-(-(a + b) // bs) for a, b in zip(held, news)]
    perm = torch.randperm(sum(per), generator=g).tolist()
    tables = torch.full((B, max(per)), -1, dtype=torch.int32)
    for b, n in enumerate(per):
        for j in range(n):
            tables[b, j] = perm.pop()
    tables = tables.to(DEV)
    reading = dict(splits=1, reading=pkv.PKV_READING_VALUES)
    q2, out, used = write_and_attend(fmt, sum(per), hk, bs, tables, proj, hq, news, held, **reading)
    first, at, block = sum(held), 0, 0
    for b in range(B):
        if b in (0, 1, 31, 32, 63, 127, 128, 129, B // 2, B - 1):
            rows = torch.cat([torch.arange(sum(held[:b]), sum(held[:b + 1])), torch.arange(first + at, first + at + news[b])])
            own = torch.where(tables[b:b + 1] >= 0, torch.arange(tables.shape[1], dtype=torch.int32, device=DEV), -1)
            own = own.to(torch.int32).contiguous()
            if news[b]:
                q1, o1, u1 = write_and_attend(fmt, max(per), hk, bs, own, proj[rows.to(DEV)], hq, [news[b]], [held[b]], **reading)
                assert torch.equal(q2[at:at + news[b]], q1) and torch.equal(out[at:at + news[b]], o1)
                assert all(torch.equal(x[block:block + per[b]], y) for x, y in zip(used, u1))
        at += news[b]
        block += per[b]


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_in_place(fmt):
    hq, hk, bs, news = 8, 2, 32, [70, 0, 33]
    T, f = sum(news), freqs()
    tables, lens, starts = i32([[0, 1, 2], [3, 4, 5], [6, 7, 8]]), i32([5, 6, 7]), i32([0, 70, 70, 103])
    results = []
    for inside in (False, True):
        pools, planes = pages(fmt, 9, hk, bs)
        for t in pools + list(planes.values()):
            t.view(torch.uint8).zero_()
        q, k, v = (x.unflatten(1, (-1, D)) for x in randn(T, (hq + 2 * hk) * D, seed=4).split([hq * D, hk * D, hk * D], 1))
        out = pkv.norm_rotate_append(q, k, v, None, f, tables, lens, *pools, query_starts=starts, q_weight=randn(D, seed=5),
                                     k_weight=randn(D, seed=6), q_out=q if inside else None, **planes, **fmt)
        results.append([out] + [t.view(torch.uint8) for t in pools + list(planes.values())])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_graphs_replay_at_once(fmt):
    """Each captured call has a workspace of its own: values, factors and the states of splits."""
    hq, hk, bs, n = 8, 2, 32, 500
    tables, starts, lens = i32([list(range(16))]), i32([0, n]), i32([n])
    calls = []
    for seed in (7, 8):
        proj = randn(n, (hq + 2 * hk) * D, seed=seed)
        q, k, v = (x.unflatten(1, (-1, D)) for x in proj.split([hq * D, hk * D, hk * D], 1))
        pools, planes = pages(fmt, 16, hk, bs)
        q = pkv.norm_rotate_append(q, k, v, None, freqs(), tables, i32([0]), *pools, query_starts=starts, **planes, **fmt)
        call = lambda q=q, pools=pools, planes=planes: pkv.paged_prefill_attention(
            q, *pools, tables, lens, starts, 0.09, splits=3, reading=pkv.PKV_READING_VALUES, **planes, **fmt)
        want = call()
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            got = call()
        calls.append((graph, stream, got, want, call))  # (the call holds what the graph reads)
    for _ in range(20):
        for graph, stream, *_ in calls:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got, want) for _, _, got, want, _ in calls)


@pytest.mark.parametrize("reading", [pkv.PKV_READING_DIRECT, pkv.PKV_READING_VALUES])
@pytest.mark.parametrize("hq", [2, 6, 10])
@pytest.mark.parametrize("fmt", FORMATS)
def test_neighbours_in_the_batch_change_nothing(fmt, hq, reading):
    """Tokens of the next sequence lie in the same tile of query rows; theirs here are 2^8 to 2^24 times as large, so that
    their maxima rise and lie far from zero."""
    if fmt.get("bits") and fmt is not BLOCK and reading == pkv.PKV_READING_DIRECT:
        return  # refused
    hk, bs, n = 2, 32, 7
    tables = i32([list(range(16)), list(range(16, 32))])
    pools, planes = pages(fmt, 32, hk, bs)
    proj = randn(2 * 500, (hq + 2 * hk) * D, seed=9)
    q, k, v = (x.unflatten(1, (-1, D)) for x in proj.split([hq * D, hk * D, hk * D], 1))
    q = pkv.norm_rotate_append(q, k, v, None, freqs(), tables, i32([0, 0]), *pools, query_starts=i32([0, 500, 1000]),
                               **planes, **fmt)[:2 * n]
    call = lambda q, t, lens, starts: pkv.paged_prefill_attention(q, *pools, t, i32(lens), i32(starts), 0.09, splits=1,
                                                                  reading=reading, **planes, **fmt)
    alone = call(q[:n].contiguous(), tables[:1].contiguous(), [500], [0, n])
    for factor in (2.0 ** 8, 2.0 ** 16, 2.0 ** 24):
        both = torch.cat([q[:n], q[n:] * factor])
        assert torch.equal(call(both, tables, [500, 500], [0, n, 2 * n])[:n], alone)
