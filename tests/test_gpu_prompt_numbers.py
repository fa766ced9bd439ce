"""Prompt attention where weights or scores span what the formats hold, against float64."""

import math

import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = dict(bits=8, group_size=pkv.PKV_GROUP_BLOCK)
FORMATS = [dict(), E4M3, dict(bits=8), dict(bits=4)]
D = 128


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def pages_of(fmt, codes, bs, scale):
    """A pool of one KV head whose rows, block after block, are `codes` [rows, D] (small whole numbers, not negative) times
    `scale` (a power of two): exact in every format. Planes by their suffix."""
    x = codes.view(-1, 1, bs, D)
    nb, bits = x.shape[0], fmt.get("bits", 16)
    if bits == 16:
        return (x * scale).to(torch.bfloat16), {}
    if fmt is E4M3:
        return x.float().to(torch.float8_e4m3fn), {"_scales": torch.full((nb, 1), scale, device=DEV)}
    planes = {"_scales": torch.full((nb, 1, bs, D // 64), scale, dtype=torch.bfloat16, device=DEV),
              "_biases": torch.zeros((nb, 1, bs, D // 64), dtype=torch.bfloat16, device=DEV)}
    per = 32 // bits
    w = (x.long().unflatten(-1, (-1, per)) << (torch.arange(per, device=DEV) * bits)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32), planes


def attend(fmt, q, k, v, bs, k_scale, v_scale, scale, **kw):
    """Outputs [T, HQ, D] of q's tokens, the newest of the rows of k and v (codes as for pages_of)."""
    (kp, ks), (vp, vs) = pages_of(fmt, k, bs, k_scale), pages_of(fmt, v, bs, v_scale)
    planes = {"k" + n: t for n, t in ks.items()} | {"v" + n: t for n, t in vs.items()}
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkv.paged_prefill_attention(q, kp, vp, torch.arange(kp.shape[0], dtype=torch.int32, device=DEV)[None], i32([k.shape[0]]),
                                      i32([0, q.shape[0]]), scale, error_flag=err, **planes, **fmt, **kw)
    assert int(err) == 0
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("below", [26, 30])
def test_one_key_against_a_million_small_ones(fmt, below):
    """The first key's weight is 2^below times each other's and its value is zero, so that the output is what the others add up
    to: 2^20 weights that fp16 could not hold beside 1."""
    rows, T, bs = 1 << 20, 3, 256
    k = torch.zeros(rows, D, dtype=torch.int32, device=DEV)
    v = torch.full((rows, D), 8, dtype=torch.int32, device=DEV)
    k[0], v[0] = 8, 0
    scale = below * math.log(2.0) / (8 * D)  # of queries of ones
    q = torch.ones(T, 2, D, dtype=torch.bfloat16, device=DEV)
    got = attend(fmt, q, k, v, bs, 1.0, 0.125, scale, splits=1).double()
    f32 = float(torch.tensor(scale, dtype=torch.float32))
    w = math.exp(-f32 * 8 * D)
    n = torch.arange(rows - T, rows, device=DEV, dtype=torch.float64)  # the other keys that a token sees
    want = (n * w / (1 + n * w))[:, None, None].expand_as(got)
    # a weight: half a step of bf16 (2^-8) or fp16 (2^-11, or 2^-25 where steps are even, of 2^7 for the maximum: 2^-32 in all); its
    # argument, near 30, in f32 and the exponential 2^-18; sums of n equal terms in f32 n * 2^-24 in pairs of four sums; the output
    rel = 2.0 ** -8 + 2.0 ** -18 + rows / 4 * 2.0 ** -24 + 2.0 ** -8
    tol = rel * want + (rows * 2.0 ** -32 if fmt.get("bits") and fmt is not E4M3 else 0.0)
    assert bool(((got - want).abs() <= tol).all()), (got[0, 0, 0].item(), want[0, 0, 0].item())


@pytest.mark.parametrize("fmt", FORMATS[:3])
@pytest.mark.parametrize("splits", [1, 2, 3, 7])
@pytest.mark.parametrize("scale", [0.2, 0.24, 0.28, 0.31])
def test_splits_far_from_zero_keep_their_differences(fmt, splits, scale):
    """Scores of 2^24 and, in the first half of the keys, 8 more, all exact in f32; the scale makes steps of about two of the 8.
    The second half's share of the weights is what the output says: parts of the keys join by the difference of their maxima."""
    rows, T, bs = 1792, 4, 256
    k = torch.zeros(rows, D, dtype=torch.int32, device=DEV)
    v = torch.zeros_like(k)
    k[:, 0] = 64
    k[:rows // 2, 1], v[rows // 2:] = 1, 8
    q = torch.zeros(T, 2, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0], q[..., 1] = 2.0 ** 18, 8.0
    got = attend(fmt, q, k, v, bs, 1.0, 0.125, scale, splits=splits).double()
    seen = rows // 2 - T + 1 + torch.arange(T, device=DEV, dtype=torch.float64)  # of the second half
    less = seen * math.exp(-8 * float(torch.tensor(scale, dtype=torch.float32)))
    want = (less / (less + rows // 2))[:, None, None].expand_as(got)
    # weights and outputs half a step of bf16 each (2^-8); of arguments up to 2^2, after the difference, c and the product are
    # rounded (2^2 * 2^-23) and the exponential is off by 2^-20; sums of 1792 terms
    tol = (2 * 2.0 ** -8 + 2.0 ** -18 + rows * 2.0 ** -24) * want
    assert bool(((got - want).abs() <= tol).all()), ((got - want).abs() / want).max().item()
