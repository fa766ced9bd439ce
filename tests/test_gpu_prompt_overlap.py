"""Norm, rotation, write and prompt attention right behind a decode step with its write, which lets the next kernel start before
it has ended: what they read is what the step wrote."""

import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv
from test_gpu_rotate import BLOCK, DEV, freqs, pages, randn, raw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [dict(), dict(bits=8), dict(bits=4), BLOCK])
def test_behind_a_step_with_its_write(fmt):
    B, h, D, bs, per, steps = 3, 4, 128, 32, 12, 60
    f, scale = freqs(D // 2), 0.09
    tables = torch.arange(B * per, dtype=torch.int32, device=DEV).view(B, per)
    starts = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    new = randn(steps, 4, B, h, 1, D, seed=1)
    lens = torch.arange(1, steps + 1, dtype=torch.int32, device=DEV)[:, None].repeat(1, B) * 3
    pos = torch.zeros(B, 1, dtype=torch.int32, device=DEV)
    results = []
    for apart in (True, False):
        pools, planes = pages(fmt, B * per, h, bs, D, D)
        other, other_planes = pages(fmt, B * per, h, bs, D, D)
        for t in pools + other + list(planes.values()) + list(other_planes.values()):
            t.view(torch.uint8).zero_()
        wait = torch.cuda.synchronize if apart else (lambda: None)
        got = []
        for i in range(steps):
            q, k, v, x = new[i]
            wait()
            if fmt is BLOCK:  # (its step has no write of its own)
                pkv.paged_append(k, v, tables, lens[i] - 1, *pools, **planes, **fmt)
                wait()
                o = pkv.paged_decode_attention(q, *pools, tables, lens[i], scale, **planes, **fmt)
            else:
                o = pkv.paged_decode_append_attention(q, k, v, *pools, tables, lens[i], scale, **planes, **fmt)
            wait()
            # the row that it wrote, by attention of one token; its outputs, as keys and values of other pages
            a = pkv.paged_prefill_attention(q[:, :, 0], *pools, tables, lens[i], starts, scale, reading=pkv.PKV_READING_VALUES,
                                            **planes, **fmt)
            wait()
            o = pkv.paged_decode_attention(x, *pools, tables, lens[i], scale, **planes, **fmt)
            wait()
            r = pkv.norm_rotate_append(q.transpose(1, 2), o.transpose(1, 2), o.transpose(1, 2), pos, f, tables, lens[i] - 1, *other,
                                       **other_planes, **fmt)
            got += [o, a, r]
        torch.cuda.synchronize()
        results.append(got + [raw(t) for t in pools + other + list(planes.values()) + list(other_planes.values())])
    assert all(torch.equal(x, y) for x, y in zip(*results))
