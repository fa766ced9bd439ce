"""The pass that writes 16-bit values of pages of codes before prompt attention: which rows it touches."""

import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv
from test_gpu_prefill import E4M3, Cache, randn, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("fmt", [E4M3, dict(bits=8), dict(bits=4)])
@pytest.mark.parametrize("wide", [0, 400])
@pytest.mark.parametrize("length,window", [(1000, 100), (1000, 1), (300, 100), (130, 500), (901, 128)])
def test_rows_below_the_window_have_no_values(fmt, wide, length, window):
    """Blocks below the window may be another's by now; the workspace shows that no value of their rows was made."""
    n, hk, hq, D, bs = 6, 2, 4, 128, 32
    cache = Cache([length], hk, D, D, bs, fmt)
    tables = torch.nn.functional.pad(cache.tables, (0, wide), value=-1)
    layout = pkv.PoolLayout(cache.pools[0].shape[0], hk, bs, D, fmt["bits"], fmt.get("group_size", 64), 0)
    plan = pkv.make_prefill_plan(layout, pkv.PrefillParams(1, n, hq, tables.shape[1], window, 1, pkv.PKV_READING_VALUES))
    ws = torch.full((plan.workspace_bytes,), 0xAB, dtype=torch.uint8, device=DEV)
    q, err = randn(n, hq, D, seed=1), i32([0])
    got = pkv.paged_prefill_attention(q, *cache.pools, tables, i32([length]), i32([0, n]), 0.09, window=window, splits=1,
                                      reading=pkv.PKV_READING_VALUES, workspace=ws, error_flag=err, **cache.planes, **fmt)
    ref, tol = reference(q, cache, [n], 0.09, window)
    assert int(err) == 0 and bool(((got.double() - ref).abs() <= tol).all())
    values = ws[-plan.value_blocks * hk * 128 * 2 * D * 2:].view(2, plan.value_blocks, hk, 128, 2 * D)
    made = (values != 0xAB).any(-1).any(0).any(1).flatten()  # rows of the sequence, from the first block's on
    lowest = max(0, length - n - window + 1)
    first = lowest // 128 * 128
    t = torch.arange(first, first + made.numel(), device=DEV)
    assert torch.equal(made, (t >= lowest) & (t < length))
