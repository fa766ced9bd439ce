"""Prompt attention over affine pages with tables so wide that the sequences go through the workspace in groups, against tables
that are just as wide as the lengths need, bit for bit."""

import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv
from test_gpu_prefill import Cache, randn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("splits,window", [(1, 0), (3, 0), (1, 900000), (1, 77)])
def test_groups_of_sequences(bits, splits, window):
    lens, news = [700, 1, 33, 500, 90, 64, 129, 300, 11, 200, 5], [40, 1, 0, 130, 3, 64, 129, 70, 11, 0, 5]
    hk, hq, D, bs = 2, 6, 128, 32
    cache = Cache(lens, hk, D, D, bs, dict(bits=bits), seed=3)
    T = sum(news) + 9
    starts = [4]
    for n in news:
        starts.append(starts[-1] + n)
    q = randn(T, hq, D, seed=1)
    far = torch.nn.functional.pad(cache.tables, (0, 32768 - cache.tables.shape[1]), value=-1)
    layout = pkv.PoolLayout(cache.pools[0].shape[0], hk, bs, D, bits, 64, 0)
    plan = pkv.make_prefill_plan(layout, pkv.PrefillParams(len(lens), T, hq, far.shape[1], window, splits, 0))
    # 8 GB hold 65536 blocks of values: eight whole tables, nine windows of 900000 // 128 + 3 beside the tokens' 4, all of 77
    assert plan.units == T // plan.unit_tokens + {0: 8, 900000: 9, 77: 11}[window]
    for bad in (None, 3, 9):  # sequences whose length is none, in either group
        at = [l if b != bad else -1 for b, l in enumerate(lens)]
        outs = []
        for tables in (cache.tables, far):
            out, err = torch.full((T, hq, D), 5.0, dtype=torch.bfloat16, device=DEV), i32([0])
            pkv.paged_prefill_attention(q, *cache.pools, tables, i32(at), i32(starts), 0.09, bits=bits, splits=splits, window=window,
                                        out=out, error_flag=err, **cache.planes)
            outs.append((out, int(err)))
        assert torch.equal(outs[0][0], outs[1][0]) and outs[0][1] == outs[1][1] == (2 if bad == 3 else 0)
        assert (outs[1][0][:4] == 5.0).all() and (outs[1][0][-5:] == 5.0).all()


def test_starts_that_fall_between_groups_are_flagged():
    lens = [64] * 11
    cache = Cache(lens, 2, 128, 128, 32, dict(bits=8))
    q = randn(110, 4, 128, seed=2)
    far = torch.nn.functional.pad(cache.tables, (0, 32768 - cache.tables.shape[1]), value=-1)
    for at in (1, 7, 8, 9, 11):
        starts = [10 * i for i in range(12)]
        starts[at] = starts[at - 1] - 1
        out, err = torch.full((112, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV), i32([0])
        pkv.paged_prefill_attention(q, *cache.pools, far, i32(lens), i32(starts), 0.09, bits=8, out=out[1:111], error_flag=err,
                                    **cache.planes)
        assert int(err) & 2 and (out[0] == 5.0).all() and (out[111] == 5.0).all()
