"""GPU parity of e4m3 decode where value scales differ from block to block, with an error bound
per output row: by the values that carry its weight, not by the cache's largest.

With w_t the softmax weights relative to the row's largest and l their sum, the kernel rounds
each weight to fp16: off by at most 2^-11 w_t, or 2^-25 (half a step of fp16's subnormals), and
never by more than w_t itself. The f32 scores of up to 2^7 (base 2; 2^-24 relative, and as much
from each of a dozen additions) and the exponential move a weight by less than 2^-13 of it, the f32
sums of products by less than 2^-16 of the magnitudes summed, and the output rounds to bf16,
2^-8 of its value or half a step of its subnormals, 2^-134. So

    |out - ref| <= 2^-8 |ref| + 2^-134 + sum_t (2^-10 w_t + 1.01 min(w_t, 2^-25)) |V_t| / l

whatever the block size: blocks of 8 and 16 rows share a chunk of the kernel with blocks of
other scales.
"""

import numpy as np
import pytest
import torch

from oracle import block_scaled as O
from quantized_kv_decode_partial_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FMT = dict(bits=8, group_size=B.PKV_GROUP_BLOCK)


def e4m3(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).to(DEV).view(torch.float8_e4m3fn)


def error_bound(w, v, ref):
    inner = ((2.0 ** -10 * w + 1.01 * np.minimum(w, 2.0 ** -25)) @ np.abs(v)) / w.sum()
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -134 + inner


def check_rows(q, kc, ks, vc, vs, length, bs, scale, n, window=0, **kw):
    """One sequence whose blocks lie in order; q [HQ, n, D] float64 (bf16 values)."""
    hk, pages = kc.shape[1], kc.shape[0]
    rep = q.shape[0] // hk
    tables = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = B.paged_decode_attention(torch.from_numpy(q)[None].to(torch.bfloat16).to(DEV), e4m3(kc), e4m3(vc), tables,
                                   torch.tensor([length], dtype=torch.int32, device=DEV), scale,
                                   k_scales=torch.from_numpy(ks).to(DEV), v_scales=torch.from_numpy(vs).to(DEV),
                                   window=window, error_flag=err, **FMT, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    got = out[0].double().cpu().numpy()
    assert np.isfinite(got).all()
    K, V = O.block_values(kc, ks), O.block_values(vc, vs)
    K, V = (x.transpose(1, 0, 2, 3).reshape(hk, pages * bs, -1) for x in (K, V))
    worst = -np.inf
    for h in range(q.shape[0]):
        for i in range(n):
            end = length - n + i + 1
            lo = max(0, end - window) if window else 0
            k, v = K[h // rep, lo:end], V[h // rep, lo:end]
            s = scale * (k @ q[h, i])
            w = np.exp(s - s.max())
            ref = (w @ v) / w.sum()
            diff = np.abs(got[h, i] - ref) - error_bound(w, v, ref)
            worst = max(worst, float(np.max(diff / (np.abs(ref).max() + 2.0 ** -126))))
    assert worst <= 0, f"beyond the bound by {worst:.3e} of the row's largest output"


def steered(rng, pages, hk, bs, d, dv, rep, n, heavy, gap):
    """Keys whose scores are about 0 in the pages `heavy` marks and `gap` (base 2) lower in the others."""
    sign = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    q = np.abs(rng.normal(size=(hk * rep, n, d))) + 0.25
    q = torch.from_numpy(q * sign).to(torch.bfloat16).double().numpy()
    kv = rng.normal(size=(pages, hk, bs, d)) * 0.05
    light = ~np.asarray(heavy)
    # a step of `gap` base-2 units for the mean row: scale <q, K> with K = -x sign, scale = 1 / d
    mean = np.abs(q).sum(-1).mean()
    kv[light] -= sign * gap * np.log(2.0) * d / mean
    ks = (np.abs(kv).max((2, 3)) / 400).astype(np.float32)
    kc = O.e4m3_codes(kv / ks[:, :, None, None].astype(np.float64))
    vc = O.e4m3_codes(np.clip(rng.normal(size=(pages, hk, bs, dv)) * 96, -448, 448))
    return q, kc, ks, vc, 1.0 / d


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (256, 256), (192, 128)])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("ratio,gap", [(0, 4), (8, 8), (9, 30), (12, 12), (16, 40), (20, 20), (24, 40), (40, 60)])
def test_blocks_of_small_scale_that_carry_the_weight(d, dv, bs, ratio, gap):
    rng = np.random.default_rng(d + dv + bs + ratio + gap)
    pages, hk, rep, n = 11, 2, 4, 1
    heavy = np.arange(pages) % 2 == 0
    q, kc, ks, vc, scale = steered(rng, pages, hk, bs, d, dv, rep, n, heavy, gap)
    vs = np.where(heavy[:, None], 2.0 ** -8, 2.0 ** (ratio - 8)) * rng.uniform(0.6, 1, size=(pages, hk))
    check_rows(q, kc, ks, vc, vs.astype(np.float32), pages * bs - 3, bs, scale, n)


@pytest.mark.parametrize("bs", [8, 16])
@pytest.mark.parametrize("d,rep,n", [(128, 1, 1), (128, 4, 4), (256, 2, 2), (64, 8, 8)])
@pytest.mark.parametrize("ratio", [10, 20, 30, 60])
def test_large_scales_behind_the_window(bs, d, rep, n, ratio):
    # the chunk that holds the window's first row holds blocks before it too, of far larger scale
    rng = np.random.default_rng(bs + d + ratio)
    pages, hk, window = 12, 2, bs + 3
    length = pages * bs - 2
    first = (length - n + 1 - window) // bs  # the first block that any query sees
    q, kc, ks, vc, scale = steered(rng, pages, hk, bs, d, d, rep, n, np.ones(pages, bool), 0)
    vs = np.full((pages, hk), 2.0 ** -10, np.float32)
    vs[:first] = 2.0 ** (ratio - 10)
    check_rows(q, kc, ks, vc, vs, length, bs, scale, n, window=window)


@pytest.mark.parametrize("bs", [8, 16])
def test_large_scales_hidden_by_the_causal_rule(bs):
    # the newest rows start a block of larger scale, which the earliest queries do not see
    rng = np.random.default_rng(bs)
    pages, hk, rep, n, d = 5, 2, 2, 4, 128
    q, kc, ks, vc, scale = steered(rng, pages, hk, bs, d, d, rep, n, np.ones(pages, bool), 0)
    vs = np.full((pages, hk), 2.0 ** -10, np.float32)
    vs[-1] = 2.0 ** 14
    check_rows(q, kc, ks, vc, vs, (pages - 1) * bs + n - 1, bs, scale, n)


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("low,high", [(2.0 ** -140, 2.0 ** -130), (2.0 ** -126, 2.0 ** -120), (2.0 ** 108, 2.0 ** 109),
                                      (0.0, 2.0 ** -5), (0.0, 0.0), (2.0 ** -100, 2.0 ** 100)])
def test_scales_at_the_ends_of_their_range(bs, low, high):
    rng = np.random.default_rng(bs)
    pages, hk, rep, n, d = 9, 2, 4, 1, 128
    heavy = np.arange(pages) % 2 == 0
    q, kc, ks, vc, scale = steered(rng, pages, hk, bs, d, d, rep, n, heavy, 2)
    vs = np.where(heavy[:, None], low, high) * np.ones((1, hk))
    check_rows(q, kc, ks, vc, vs.astype(np.float32), pages * bs - 3, bs, scale, n)


@pytest.mark.parametrize("bs", [8, 16])
def test_scales_far_apart_in_sparse_attention(bs):
    # any order of blocks may meet in a chunk of chosen ones
    rng = np.random.default_rng(bs)
    pages, hk, rep, n, d, top_k = 40, 2, 4, 1, 128, 12
    heavy = np.arange(pages) % 3 == 0
    q, kc, ks, vc, scale = steered(rng, pages, hk, bs, d, d, rep, n, heavy, 24)
    vs = np.where(heavy[:, None], 2.0 ** -8, 2.0 ** 14) * rng.uniform(0.6, 1, size=(pages, hk))
    vs, length = vs.astype(np.float32), pages * bs
    kd, vd = e4m3(kc), e4m3(vc)
    sc = dict(k_scales=torch.from_numpy(ks).to(DEV), v_scales=torch.from_numpy(vs).to(DEV))
    tables = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([length], dtype=torch.int32, device=DEV)
    bounds = torch.zeros((pages, hk, 2, d), dtype=torch.bfloat16, device=DEV)
    B.update_block_bounds(kd, tables, lens, bounds, n_new=length, k_scales=sc["k_scales"], **FMT)
    blocks = torch.empty((1, hk, top_k), dtype=torch.int32, device=DEV)
    out = B.sparse_decode_attention(torch.from_numpy(q)[None].to(torch.bfloat16).to(DEV), kd, vd, bounds, tables, lens,
                                    scale, top_k=top_k, first_blocks=2, last_blocks=3, blocks=blocks, **sc, **FMT)
    got, K, V = out[0].double().cpu().numpy(), O.block_values(kc, ks), O.block_values(vc, vs)
    for h in range(hk * rep):
        at = blocks[0, h // rep].tolist()
        k, v = (x[at, h // rep].reshape(top_k * bs, d) for x in (K, V))
        s = scale * (k @ q[h, 0])
        w = np.exp(s - s.max())
        ref = (w @ v) / w.sum()
        assert (np.abs(got[h, 0] - ref) <= error_bound(w, v, ref)).all(), h
