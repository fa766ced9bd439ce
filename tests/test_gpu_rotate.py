"""Norm and rotation, alone and with the write into pages, against the float64 oracle and the paged append."""

import numpy as np
import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv
from oracle import rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCK = dict(bits=8, group_size=pkv.PKV_GROUP_BLOCK)


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


def freqs(half, base=1e4):
    return (base ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(DEV)


def f64(t):
    return t.double().cpu().numpy()


def check(got, x, positions, freq, weight=None, **kw):
    """Half a bf16 step of the value (2^-8 of it), and 2^-18 of what the value was made of: angles are off by
    less than 2^-21, norm and turn by a dozen f32 roundings (2^-24 each)."""
    ref, size = rotate.norm_rotate(f64(x), positions.cpu().numpy(), f64(freq),
                                   None if weight is None else f64(weight), **kw)
    err = np.abs(f64(got) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * size).all(), float((err - 2.0 ** -8 * np.abs(ref)).max())


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (1, 32, 8), (3, 5, 2), (65, 7, 1), (700, 16, 4)])
@pytest.mark.parametrize("adjacent", [False, True])
def test_norm_and_rotation(D, T, hq, hk, adjacent):
    q, k = randn(T, hq, D, seed=1), randn(T, hk, D, seed=2, scale=30.0)
    wq, wk = randn(D, seed=3), randn(D, seed=4)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 37 + 5
    f = freqs(D // 2)
    a, b = pkv.norm_rotate(q, k, pos, f, q_weight=wq, k_weight=wk, pairing=int(adjacent))
    check(a, q, pos, f, wq, adjacent=adjacent)
    check(b, k, pos, f, wk, adjacent=adjacent)


@pytest.mark.parametrize("D,rot", [(64, 8), (128, 64), (192, 64), (256, 64), (256, 248), (128, 120)])
@pytest.mark.parametrize("adjacent", [False, True])
def test_part_of_the_head_turns(D, rot, adjacent):
    q, k, f = randn(33, 3, D, seed=1), randn(33, 3, D, seed=2), freqs(rot // 2)
    pos = torch.arange(33, dtype=torch.int32, device=DEV)
    a, b = pkv.norm_rotate(q, k, pos, f, pairing=int(adjacent))
    check(a, q, pos, f, adjacent=adjacent)
    assert torch.equal(a[..., rot:], q[..., rot:]) and torch.equal(b[..., rot:], k[..., rot:])
    assert torch.equal(a[0], q[0])  # position 0 turns nothing


@pytest.mark.parametrize("sections,cycle", [([16, 24, 24], 0), ([24, 20, 20], 1), ([22, 21, 21], 1), ([60, 4], 0),
                                            ([32, 32], 1), ([0, 64, 0], 0), ([16, 16, 16, 16], 1)])
def test_positions_of_several_axes(sections, cycle):
    T, axes = 41, len(sections)
    q, k, f = randn(T, 4, 128, seed=5), randn(T, 2, 128, seed=6), freqs(64)
    pos = torch.randint(-500, 70000, (axes, T), generator=torch.Generator().manual_seed(7), dtype=torch.int32).to(DEV)
    a, b = pkv.norm_rotate(q, k, pos, f, sections=sections, section_order=cycle)
    check(a, q, pos, f, sections=sections, cycle=bool(cycle))
    check(b, k, pos, f, sections=sections, cycle=bool(cycle))


def test_far_and_negative_positions_and_odd_frequencies():
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    f = freqs(64, 1e6)
    f[1], f[2], f[3], f[4] = -1.25, 0.0, 1e-30, 1.9999
    q = randn(len(pos), 2, 128, seed=8)
    a, _ = pkv.norm_rotate(q, None, pos, f)
    check(a, q, pos, f)


def test_weights_in_f32_offset_amplitude_and_one_norm_alone():
    q, k, f = randn(9, 3, 128, seed=1), randn(9, 2, 128, seed=2), freqs(64)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    w = randn(128, seed=3).float() * 0.1
    a, b = pkv.norm_rotate(q, k, pos, f, k_weight=w, weight_offset=1.0, amplitude=1.375, eps=0.5)
    check(a, q, pos, f, amplitude=1.375)
    check(b, k, pos, f, w, offset=1.0, amplitude=1.375, eps=0.5)
    zero = torch.zeros_like(q)
    a, _ = pkv.norm_rotate(zero, None, pos, f, q_weight=w)
    assert not a.any()


def test_strides_slices_in_place_and_the_decode_layout():
    B, N, hq, hk, D = 3, 4, 6, 2, 128
    qkv = randn(B, N, (hq + 2 * hk) * D, seed=1)
    part = qkv.view(B, N, hq + 2 * hk, D)
    q, k = part[:, :, :hq], part[:, :, hq:hq + hk]
    pos = torch.arange(B * N, dtype=torch.int32, device=DEV).view(B, N)
    f = freqs(64)
    a, b = pkv.norm_rotate(q, k, pos, f)
    flat = pkv.norm_rotate(q.reshape(B * N, hq, D), k.reshape(B * N, hk, D), pos.reshape(-1), f)
    assert torch.equal(a.view(B * N, hq, D), flat[0]) and torch.equal(b.view(B * N, hk, D), flat[1])
    heads_first = torch.zeros(B, hq, N, D, dtype=torch.bfloat16, device=DEV)
    pkv.norm_rotate(q, k, pos, f, q_out=heads_first.transpose(1, 2))
    assert torch.equal(heads_first.transpose(1, 2), a)
    v = part[:, :, hq + hk:].clone()
    pkv.norm_rotate(q, k, pos, f, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(part[:, :, hq + hk:], v)


def test_no_tokens_and_refusals():
    f = freqs(64)
    none = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=DEV)
    a, b = pkv.norm_rotate(none, none, torch.empty(0, dtype=torch.int32, device=DEV), f)
    assert a.shape == none.shape and b.shape == none.shape
    q, pos = randn(4, 2, 128), torch.arange(4, dtype=torch.int32, device=DEV)
    for bad in (dict(q=q.float()), dict(q=q[..., :96]), dict(positions=pos.long()), dict(positions=pos[:3]),
                dict(k=q[:3]), dict(inv_freq=f.double()), dict(positions=torch.stack([pos, pos])),
                dict(q_weight=q[0, 0, :64]), dict(q_weight=q[0, 0].half()), dict(q_out=q[:3]), dict(positions=pos.cpu()),
                dict(q=q.cpu()), dict(sections=[32, 32]), dict(q=q.transpose(1, 2)), dict(pairing=3)):
        args = {"q": q, "k": None, "positions": pos, "inv_freq": f, **bad}
        with pytest.raises((TypeError, ValueError, pkv.PkvError)):
            pkv.norm_rotate(args.pop("q"), args.pop("k"), args.pop("positions"), args.pop("inv_freq"), **args)


# ------------------------------------------------------------------------------------ with the write
def pages(fmt, nb, hk, bs, dk, dv):
    """Empty pools and planes of a format, filled with a pattern that must stay outside the written rows."""
    bits, block = fmt.get("bits", 16), fmt.get("group_size") == pkv.PKV_GROUP_BLOCK
    kw = {}
    if bits == 16:
        pools = [randn(nb, hk, bs, d, seed=50 + d) for d in (dk, dv)]
    elif block:
        pools = [randn(nb, hk, bs, d, seed=60 + d, scale=50.0).to(torch.float8_e4m3fn) for d in (dk, dv)]
        kw = {n: torch.full((nb, hk), 2.0 ** -7, device=DEV) for n in ("k_scales", "v_scales")}
    else:
        g = torch.Generator().manual_seed(9)
        pools = [torch.randint(-2 ** 31, 2 ** 31, (nb, hk, bs, d * bits // 32), generator=g, dtype=torch.int64)
                 .to(torch.int32).to(DEV) for d in (dk, dv)]
        kw = {n: randn(nb, hk, bs, (dk if n[0] == "k" else dv) // 64, seed=len(n))
              for n in ("k_scales", "k_biases", "v_scales", "v_biases")}
    return pools, kw


def raw(t):
    return t.contiguous().view(torch.uint8)


FORMATS = [(dict(), d) for d in ((64, 64), (128, 128), (256, 256), (192, 128), (256, 128), (128, 256))] + \
    [(dict(bits=b), d) for b in (4, 8) for d in ((128, 128), (256, 256), (256, 128), (128, 256))] + \
    [(BLOCK, d) for d in ((64, 64), (128, 128), (256, 256), (192, 128), (256, 128), (128, 256))]


def compare_with_two_calls(fmt, dims, news, held, hq, hk, bs, *, packed=True, positions=None, weights=True, extra=0,
                           scale=1.0, **turn):
    """The fused call against norm_rotate, then paged_append sequence by sequence: pages bit for bit."""
    dk, dv = dims
    T, B = sum(news) + extra, len(news)
    per = [-(-(n + h) // bs) for n, h in zip(news, held)]
    nb = sum(per) + 3
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(3)).tolist()
    width = max(max(per), 1)
    tables = torch.full((B, width), -7, dtype=torch.int32)
    for b in range(B):
        for j in range(per[b]):
            tables[b, j] = perm.pop()
    tables = tables.to(DEV)
    lens = torch.tensor(held, dtype=torch.int32, device=DEV)
    proj = randn(T, hq * dk + hk * dk + hk * dv, seed=11, scale=scale)
    q = proj[:, :hq * dk].view(T, hq, dk)
    k = proj[:, hq * dk:(hq + hk) * dk].view(T, hk, dk)
    v = proj[:, (hq + hk) * dk:].view(T, hk, dv)
    rot = turn.pop("rot", dk)
    f = freqs(rot // 2)
    if weights:
        turn.update(q_weight=randn(dk, seed=1), k_weight=randn(dk, seed=2))
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    pools, planes = pages(fmt, nb, hk, bs, dk, dv)
    mine, mine_planes = [p.clone() for p in pools], {n: t.clone() for n, t in planes.items()}
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full_like(q, 7.0).contiguous()
    args = dict(q_out=q_out, error_flag=err, **mine_planes, **fmt, **turn)
    if packed:
        pkv.norm_rotate_append(q, k, v, positions, f, tables, lens, *mine,
                               query_starts=torch.tensor(starts, dtype=torch.int32, device=DEV), **args)
    else:
        n = news[0]
        args["q_out"] = q_out.unflatten(0, (B, n))
        pkv.norm_rotate_append(*(x.unflatten(0, (B, n)) for x in (q, k, v)),
                               None if positions is None else positions.unflatten(-1, (B, n)), f, tables, lens, *mine, **args)
    pos = positions
    if pos is None:
        pos = torch.tensor([h + i for n, h in zip(news, held) for i in range(n)] + [0] * extra, dtype=torch.int32, device=DEV)
    want_q, want_k = pkv.norm_rotate(q, k, pos, f, **turn)
    end = starts[-1]
    assert torch.equal(q_out[:end], want_q[:end])
    assert (q_out[end:] == 7.0).all()
    for b in range(B):
        if not news[b]:
            continue
        rows = slice(starts[b], starts[b + 1])
        pkv.paged_append(want_k[rows].transpose(0, 1)[None].contiguous(), v[rows].transpose(0, 1)[None].contiguous(),
                         tables[b:b + 1].contiguous(), lens[b:b + 1].contiguous(), *pools, error_flag=err, **planes, **fmt)
    assert int(err) == 0
    for got, want in list(zip(mine, pools)) + [(mine_planes[n], planes[n]) for n in planes]:
        assert torch.equal(raw(got), raw(want))


@pytest.mark.parametrize("fmt,dims", FORMATS)
def test_write_equals_two_calls(fmt, dims):
    compare_with_two_calls(fmt, dims, [1, 70, 0, 33, 5, 64], [0, 31, 4, 32, 90, 1], 6, 3, 32)


@pytest.mark.parametrize("fmt", [dict(), dict(bits=4), dict(bits=8), BLOCK])
@pytest.mark.parametrize("news,held,packed", [
    ([1], [0], True), ([1], [500], False), ([1] * 67, list(range(67)), False), ([4] * 5, [0, 30, 31, 32, 63], False),
    ([0, 0, 0], [5, 0, 1], True), ([300], [3], True), ([2] * 40, [31] * 40, True)])
def test_write_of_few_and_many(fmt, news, held, packed):
    compare_with_two_calls(fmt, (128, 128), news, held, 8, 2, 32, packed=packed)


@pytest.mark.parametrize("fmt", [dict(), BLOCK])
@pytest.mark.parametrize("hk,bs", [(1, 8), (1, 16), (2, 96), (5, 64), (8, 32), (9, 32), (16, 32), (1, 256), (1, 1024)])
def test_write_heads_and_block_sizes(fmt, hk, bs):
    compare_with_two_calls(fmt, (128, 128), [37, 300, 1], [9, 700, 15], hk, hk, bs)
    compare_with_two_calls(fmt, (256, 256), [260, 2], [0, bs - 1], 2 * hk, hk, bs, rot=64)


@pytest.mark.parametrize("fmt,dims", [(dict(), (192, 128)), (dict(bits=4), (256, 256)), (BLOCK, (64, 64)), (BLOCK, (256, 256))])
def test_write_with_axes_part_turn_and_tail(fmt, dims):
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 9000, (3, 90), generator=g, dtype=torch.int32).to(DEV)
    compare_with_two_calls(fmt, dims, [40, 0, 47], [0, 7, 29], 4, 2, 32, positions=pos, extra=3, rot=32, sections=[6, 5, 5],
                           section_order=1, pairing=1, weight_offset=1.0, amplitude=0.5)


def test_write_grown_scales_zero_rows_and_no_norm():
    compare_with_two_calls(BLOCK, (128, 128), [3, 40], [20, 50], 2, 2, 32, weights=False, scale=1e4)
    compare_with_two_calls(BLOCK, (128, 128), [3, 40], [20, 64], 2, 2, 32, weights=False, scale=0.0)


@pytest.mark.parametrize("fmt", [dict(), dict(bits=8), BLOCK])
def test_bad_blocks_lengths_and_starts(fmt):
    hk, bs, D, T = 2, 32, 128, 12
    pools, planes = pages(fmt, 6, hk, bs, D, D)
    before = [p.clone() for p in pools]
    q, k, v, f = randn(T, 4, D, seed=1), randn(T, hk, D, seed=2), randn(T, hk, D, seed=3), freqs(64)
    tables = torch.tensor([[0, 1], [6, 2], [3, -1], [4, 5]], dtype=torch.int32, device=DEV)

    def call(lens, starts):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.full_like(q, 7.0)
        mine, kw = [p.clone() for p in pools], {n: t.clone() for n, t in planes.items()}
        pkv.norm_rotate_append(q, k, v, None, f, tables, torch.tensor(lens, dtype=torch.int32, device=DEV), *mine,
                               query_starts=torch.tensor(starts, dtype=torch.int32, device=DEV), q_out=out, error_flag=err,
                               **kw, **fmt)
        return int(err), out, mine

    err, out, mine = call([0, 0, 31, 0], [0, 3, 6, 9, 12])  # block 6 is none, nor is block -1
    assert err == 1
    assert not any(torch.equal(raw(m[0]), raw(b[0])) for m, b in zip(mine, before))
    assert all(torch.equal(raw(m[[1, 2, 5]]), raw(b[[1, 2, 5]])) for m, b in zip(mine, before))
    assert not (out == 7.0).all(-1).any()
    for bad in (-1, 62, 2 ** 31 - 1, -2 ** 31):
        err, out, mine = call([0, 0, bad, 0], [0, 3, 3, 6, 9])
        assert err == 2
        assert all(torch.equal(raw(m[[1, 2, 3, 5]]), raw(b[[1, 2, 3, 5]])) for m, b in zip(mine, before))
        assert (out[9:] == 7.0).all() and not (out[:9] == 7.0).all(-1).any()
    for starts in ([0, 5, 3, 9, 12], [0, 3, 6, 9, 13], [-2, 3, 6, 9, 12], [0, 0, 0, 0, 2 ** 31 - 1]):
        assert call([0, 0, 0, 0], starts)[0] & 2  # and whatever they say, nothing outside the tokens is touched
    err, out, mine = call([0, 0, 0, 0], [12, 12, 12, 12, 12])
    assert err == 0 and (out == 7.0).all() and all(torch.equal(raw(m), raw(b)) for m, b in zip(mine, before))


def test_write_on_another_stream_and_in_a_graph():
    hk, bs, D, B = 2, 32, 128, 3
    pools, _ = pages(dict(), 8, hk, bs, D, D)
    tables = torch.arange(6, dtype=torch.int32, device=DEV).view(3, 2)
    lens = torch.tensor([0, 5, 40], dtype=torch.int32, device=DEV)
    q, k, v, f = randn(B, 1, 4, D, seed=1), randn(B, 1, hk, D, seed=2), randn(B, 1, hk, D, seed=3), freqs(64)
    want = [p.clone() for p in pools]
    q_want = pkv.norm_rotate_append(q, k, v, None, f, tables, lens, *want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, q_out = [p.clone() for p in pools], torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.norm_rotate_append(q, k, v, None, f, tables, lens, *got, q_out=q_out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, q_want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_write_refusals():
    hk, bs, D = 2, 32, 128
    pools, planes = pages(BLOCK, 4, hk, bs, D, D)
    tables, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    q, k, v, f = randn(2, 4, D), randn(2, hk, D), randn(2, hk, D), freqs(64)
    good = dict(q=q, k=k, v=v, positions=None, inv_freq=f, block_tables=tables, seq_lens=lens, k_pool=pools[0],
                v_pool=pools[1], **planes, **BLOCK)
    pkv.norm_rotate_append(**good)
    for bad in (dict(k=k[:, :1]), dict(v=v.float()), dict(v=v[..., :64]), dict(seq_lens=lens.long()), dict(seq_lens=lens[:1]),
                dict(block_tables=tables[:1]), dict(k_scales=None), dict(k_scales=planes["k_scales"].half()),
                dict(query_starts=torch.tensor([0, 2], dtype=torch.int32, device=DEV)), dict(k_pool=pools[0].float()),
                dict(v_pool=pools[1][:3]), dict(block_tables=tables.cpu()), dict(q=q[:1]), dict(k_pool=pools[0].transpose(1, 2)),
                dict(positions=torch.zeros(2, 2, dtype=torch.int32, device=DEV)), dict(sections=[32, 32])):
        with pytest.raises((TypeError, ValueError, pkv.PkvError)):
            pkv.norm_rotate_append(**{**good, **bad})
