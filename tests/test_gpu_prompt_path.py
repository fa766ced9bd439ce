"""A prompt's whole way: projections normed and rotated into pages, attention over them in chunks, then a decode step,
against float64 attention over the rotated rows; and waits of the prompt attention that give up."""

import math

import numpy as np
import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv
from oracle import rotate
from test_gpu_rotate import BLOCK, freqs, pages, randn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rounded(x):
    """float64 to bf16 and back."""
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("fmt", [dict(), dict(bits=8), BLOCK])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("axes", [1, 3])
def test_prompt_in_two_chunks_and_a_decode_step(fmt, D, axes):
    hq, hk, bs, lens = 6, 2, 32, [200, 37, 129]
    cut, T = [150, 37, 1], sum(lens)
    f, wq, wk = freqs(D // 2), randn(D, seed=1), randn(D, seed=2)
    turn = dict(q_weight=wq, k_weight=wk)
    if axes == 3:
        half = D // 2
        turn.update(sections=[half - 2 * (half // 3), half // 3, half // 3], section_order=pkv.PKV_SECTIONS_CYCLE)
    rows = [randn(n + 1, hq + 2 * hk, D, seed=10 + b) for b, n in enumerate(lens)]  # the last token is decoded
    g = torch.Generator().manual_seed(3)
    pos = [torch.stack([torch.arange(n + 1)] + [torch.randint(0, 50, (n + 1,), generator=g) for _ in range(axes - 1)]).int()
           for n in lens]
    per = [-(-(n + 1) // bs) for n in lens]
    nb = sum(per) + 1
    order = torch.randperm(nb, generator=g).tolist()
    tables = torch.zeros(3, max(per), dtype=torch.int32)
    for b in range(3):
        for j in range(per[b]):
            tables[b, j] = order.pop()
    tables = tables.to(DEV)
    pools, planes = pages(fmt, nb, hk, bs, D, D)
    err, scale = torch.zeros(1, dtype=torch.int32, device=DEV), 1 / math.sqrt(D)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    outs = [[] for _ in lens]
    for lo, hi in (([0, 0, 0], cut), (cut, lens)):
        new = [h - l for l, h in zip(lo, hi)]
        x = torch.cat([rows[b][lo[b]:hi[b]] for b in range(3)])
        p = torch.cat([pos[b][:, lo[b]:hi[b]] for b in range(3)], 1).contiguous().to(DEV)
        starts = i32([0, new[0], new[0] + new[1], sum(new)])
        q = pkv.norm_rotate_append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], None if axes == 1 else p, f, tables, i32(lo), *pools,
                                   query_starts=starts, error_flag=err, **planes, **fmt, **turn)
        o = pkv.paged_prefill_attention(q, *pools, tables, i32(hi), starts, scale, error_flag=err, **planes, **fmt)
        for b, part in enumerate(o.split(new)):
            outs[b].append(part)
    x = torch.stack([rows[b][lens[b]:] for b in range(3)])  # [B, 1, heads, D]
    p = torch.stack([pos[b][:, lens[b]:] for b in range(3)], 1).contiguous().to(DEV)
    q = torch.empty(3, hq, 1, D, dtype=torch.bfloat16, device=DEV)
    pkv.norm_rotate_append(x[:, :, :hq], x[:, :, hq:hq + hk], x[:, :, hq + hk:], None if axes == 1 else p, f, tables, i32(lens),
                           *pools, q_out=q.transpose(1, 2), error_flag=err, **planes, **fmt, **turn)
    step = pkv.paged_decode_attention(q, *pools, tables, i32([n + 1 for n in lens]), scale, error_flag=err, **planes, **fmt)
    assert int(err) == 0
    f64 = lambda t: t.double().cpu().numpy()
    kw = dict(sections=turn.get("sections"), cycle=True)
    # rows as pages hold them: bf16 exactly; 8-bit affine codes within half a step of 1/255 of a group's range; e4m3
    # within 2^-4 of the value or half the smallest step of a block scaled to 448
    worst = {16: 0.0, 8: 0.03, -1: 2.0 ** -4}[-1 if fmt is BLOCK else fmt.get("bits", 16)]
    for b, n in enumerate(lens):
        qq = rounded(rotate.norm_rotate(f64(rows[b][:, :hq]), pos[b].numpy(), f64(f), f64(wq), **kw)[0])
        kk = rounded(rotate.norm_rotate(f64(rows[b][:, hq:hq + hk]), pos[b].numpy(), f64(f), f64(wk), **kw)[0])
        vv = f64(rows[b][:, hq + hk:])
        got = np.concatenate([f64(torch.cat(outs[b])), f64(step[b].transpose(0, 1))])
        for h in range(hq):
            s = qq[:, h] @ kk[:, h // 3].T * scale
            s[np.triu_indices(n + 1, 1)] = -np.inf
            w = np.exp(s - s.max(-1, keepdims=True))
            ref = w / w.sum(-1, keepdims=True) @ vv[:, h // 3]
            # rotated rows may round to the other neighbour (2^-8 of a value), weights and outputs round to bf16
            size = (np.abs(qq[:, h]) @ np.abs(kk[:, h // 3]).T * scale).max()
            tol = 2.0 ** -6 + (2 * size * (worst + 2.0 ** -7) + worst + 2.0 ** -7) * np.abs(vv[:, h // 3]).max()
            assert np.abs(got[:, h] - ref).max() <= tol
            assert np.abs(got[:, h] - ref).mean() <= 0.02  # values of unit variance: far below what lost rows would cost


@pytest.mark.parametrize("fmt", [dict(), BLOCK])
@pytest.mark.parametrize("splits", [1, 3])
def test_waits_that_run_out_give_up(fmt, splits):
    """A bound of 1 ns runs out once a wait outlasts a tick of the GPU's clock, as those for rows from HBM do (L2 holds
    other things before each call); the call flags it and the next one is as ever."""
    B, hk, bs, n = 4, 8, 32, 700
    per = -(-n // bs)
    pools, planes = pages(fmt, B * per, hk, bs, 128, 128)
    tables = torch.arange(B * per, dtype=torch.int32, device=DEV).view(B, per)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    starts = torch.arange(B + 1, dtype=torch.int32, device=DEV) * n
    q = randn(B * n, 32, 128, seed=3)
    other = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)

    def call():
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        other.fill_(1)
        out = pkv.paged_prefill_attention(q, *pools, tables, lens, starts, 0.09, splits=splits, error_flag=err,
                                          reading=pkv.PKV_READING_DIRECT, **planes, **fmt)
        torch.cuda.synchronize()
        return out, int(err)

    want, err = call()
    assert err == 0
    pkv.set_wait_limit_ns(1)
    try:
        seen = {call()[1] for _ in range(20)}
    finally:
        pkv.set_wait_limit_ns(0)
    assert 4 in seen and seen <= {0, 4}
    got, err = call()
    assert err == 0 and torch.equal(got, want)


def test_two_streams_at_once():
    n, hk, bs = 900, 2, 32
    per = -(-n // bs)
    pools = [randn(per, hk, bs, 128, seed=i) for i in (1, 2)]
    tables = torch.arange(per, dtype=torch.int32, device=DEV).view(1, per)
    lens, starts = torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    qs = [randn(300, 8, 128, seed=5 + i) for i in range(4)]
    want = [pkv.paged_prefill_attention(q, *pools, tables, lens, starts, 0.09, splits=3) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [None] * len(qs)
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = pkv.paged_prefill_attention(qs[i], *pools, tables, lens, starts, 0.09, splits=3)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
