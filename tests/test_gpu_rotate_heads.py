"""Norm, rotation and write where there are fewer query than KV heads, so that warps begin with keys: good tables against two
calls, and bad blocks and lengths, whose keys have no place to go."""

import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv
from test_gpu_rotate import BLOCK, DEV, check, compare_with_two_calls, freqs, pages, randn, raw

pytestmark = pytest.mark.gpu

# tokens such that each one's heads are dealt to one, two, three and more warps of a GPU of 152 SMs
HEADS = [(128, 4, 16), (256, 2, 8), (128, 1, 64), (64, 3, 40)]
TOKENS = [1, 7, 700, 2000, 4000]


@pytest.mark.parametrize("D,hq,hk", HEADS)
@pytest.mark.parametrize("T", TOKENS)
def test_norm_and_rotation(D, hq, hk, T):
    q, k, w, f = randn(T, hq, D, seed=1), randn(T, hk, D, seed=2), randn(D, seed=3), freqs(D // 2)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    a, b = pkv.norm_rotate(q, k, pos, f, k_weight=w)
    check(a, q, pos, f)
    check(b, k, pos, f, w)


@pytest.mark.parametrize("fmt", [dict(), BLOCK, dict(bits=8), dict(bits=4)])
@pytest.mark.parametrize("D,hq,hk", HEADS)
@pytest.mark.parametrize("T", TOKENS)
def test_write_equals_two_calls(fmt, D, hq, hk, T):
    if D == 64 and fmt.get("bits") and fmt is not BLOCK:
        return  # affine pages have no rows of 64
    compare_with_two_calls(fmt, (D, D), [T], [5], hq, hk, 32)


@pytest.mark.parametrize("fmt", [dict(), BLOCK, dict(bits=8)])
@pytest.mark.parametrize("D,hq,hk", HEADS[:3])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("what", ["blocks", "length"])
def test_keys_without_a_place_go_nowhere(fmt, D, hq, hk, T, what):
    """The queries come out as ever; the pages, all bad or too few for the length, keep every byte."""
    bs, f = 32, freqs(D // 2)
    pools, planes = pages(fmt, 4, hk, bs, D, D)
    before = [t.clone() for t in pools + list(planes.values())]
    proj = randn(T, (hq + 2 * hk) * D, seed=4)
    q, k, v = (x.unflatten(1, (-1, D)) for x in proj.split([hq * D, hk * D, hk * D], 1))
    width = -(-T // bs)
    tables = torch.tensor([4, -1, 2 ** 31 - 1], dtype=torch.int32, device=DEV).repeat(width)[None, :width].contiguous()
    lens = torch.tensor([0 if what == "blocks" else width * bs], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    got = pkv.norm_rotate_append(q, k, v, pos, f, tables, lens, *pools, error_flag=err,
                                 query_starts=torch.tensor([0, T], dtype=torch.int32, device=DEV), **planes, **fmt)
    assert int(err) == (1 if what == "blocks" else 2)
    assert torch.equal(got, pkv.norm_rotate(q, None, pos, f)[0])
    assert all(torch.equal(raw(t), raw(b)) for t, b in zip(pools + list(planes.values()), before))
