"""A seeded sweep of decode calls over e4m3 pages: head-dim pairs, query rows, block sizes,
ragged lengths, windows, partitions, schedules and value scales drawn together, through the one
call and through its two passes, against float64 with the bound of tests/test_gpu_e4m3_scales.py
for every output row."""

import math
import random

import numpy as np
import pytest
import torch

import oracle
from oracle import block_scaled as O
from quantized_kv_decode_partial_gb300 import binding as B
from test_gpu_e4m3 import FMT, e4m3, make_pool, make_tables
from test_gpu_e4m3_scales import error_bound

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SHAPES = [(64, 64), (128, 128), (256, 256), (192, 128), (256, 128), (128, 256)]


def draw(i):
    rnd = random.Random(29000 + i)
    d, dv = rnd.choice(SHAPES)
    n = rnd.choice([1, 1, 2, 3, 4])
    rep = rnd.choice([r for r in (1, 2, 4, 5, 8, 16) if r * n <= 64])
    lens = [rnd.randint(n, rnd.choice([40, 300, 1500])) for _ in range(rnd.choice([1, 2, 5]))]
    kw = dict(window=rnd.choice([0, 0, 1, 9, 100]), partition_tokens=rnd.choice([0, 0, 32, 96, 160]),
              schedule=rnd.choice([B.PKV_SCHEDULE_AUTO, B.PKV_SCHEDULE_PARTITIONS, B.PKV_SCHEDULE_BALANCED]))
    return d, dv, rep, n, rnd.choice([1, 2, 3]), rnd.choice([8, 16, 32, 64, 96]), lens, rnd.choice([1, 9, 25]), kw


def prepare(i):
    d, dv, rep, n, hk, bs, lens, spread, kw = draw(i)
    rng = np.random.default_rng(i)
    tables, nb = make_tables(rng, lens, bs)
    kc, ks = make_pool(rng, nb, hk, bs, d, tables, lens)
    vc, vs = make_pool(rng, nb, hk, bs, dv, tables, lens, spread)
    q = torch.from_numpy(rng.normal(size=(len(lens), rep * hk, n, d))).to(torch.bfloat16)
    args = (q.to(DEV), e4m3(kc), e4m3(vc), torch.tensor(tables, dtype=torch.int32, device=DEV),
            torch.tensor(lens, dtype=torch.int32, device=DEV), 1 / math.sqrt(d))
    scales = dict(k_scales=torch.from_numpy(ks).to(DEV), v_scales=torch.from_numpy(vs).to(DEV))
    K, V = O.block_values(kc, ks), O.block_values(vc, vs)

    def check(out):
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        for b, length in enumerate(lens):
            k, v = oracle.gather_pages(K, tables[b], length), oracle.gather_pages(V, tables[b], length)
            for h in range(rep * hk):
                for j in range(n):
                    end = length - n + j + 1
                    lo = max(0, end - kw["window"]) if kw["window"] else 0
                    s = k[h // rep, lo:end] @ q[b, h, j].double().numpy() / math.sqrt(d)
                    w = np.exp(s - s.max())
                    ref = (w @ v[h // rep, lo:end]) / w.sum()
                    assert (np.abs(got[b, h, j] - ref) <= error_bound(w, v[h // rep, lo:end], ref)).all(), (b, h, j)

    return args, scales, kw, check


@pytest.mark.parametrize("i", range(60))
def test_random_calls_match_float64(i):
    args, scales, kw, check = prepare(i)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = B.paged_decode_attention(*args, error_flag=err, **scales, **kw, **FMT)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(out)


@pytest.mark.parametrize("i", range(60, 90))
def test_random_calls_in_two_passes(i):
    args, scales, kw, check = prepare(i)
    q, k, v, tables = args[:4]
    plan = B.make_plan(B.layout_for(k, q.shape[-1], 8, B.PKV_GROUP_BLOCK, v),
                       B.DecodeParams(q.shape[0], q.shape[1], q.shape[2], tables.shape[1], kw["partition_tokens"],
                                      kw["window"], 0, kw["schedule"]))
    out = torch.full(q.shape[:-1] + (v.shape[-1],), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.full((max(plan.workspace_bytes, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for passes in ("partial", "merge"):
        B.paged_decode_passes(*args, passes=passes, out=out, workspace=ws, error_flag=err, **scales, **kw, **FMT)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(out)
    assert torch.equal(out, B.paged_decode_attention(*args, **scales, **kw, **FMT))
