"""Prompt attention over pages of every format against float64, within the bounds that test_prompt_reference.py tries out."""

import math

import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv
from prompt_reference import E4M3, Pages, affine, attention, complaint

pytestmark = pytest.mark.gpu
DEV = "cuda"
DIMS = [(64, 64), (128, 128), (256, 256), (192, 128), (256, 128), (128, 256)]
AFFINE = [(128, 128), (256, 256), (256, 128), (128, 256)]
DIRECT, VALUES = pkv.PKV_READING_DIRECT, pkv.PKV_READING_VALUES
# every way that a format's pages are read
WAYS = [(dict(), 0), (E4M3, DIRECT), (E4M3, VALUES), (dict(bits=8), 0), (dict(bits=4), 0)]
WITH_DIMS = [(f, r, d) for f, r in WAYS for d in (AFFINE if affine(f) else DIMS)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def check(pages, hq, news, scale, *, seed=5, tables=None, flag=0, hidden=None, window=0, repeats=1, **kw):
    T, d = sum(news), pages.values[0].shape[-1]
    q = torch.randn(T, hq, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)
    ref, tol = attention(q, pages, news, scale, window, hidden)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    first = None
    for _ in range(repeats):
        err = i32([0])
        got = pkv.paged_prefill_attention(q, *pages.pools, pages.tables if tables is None else tables, i32(pages.lens), i32(starts),
                                          scale, error_flag=err, window=window, **pages.planes, **pages.fmt, **kw)
        assert int(err) == flag
        first = got if first is None else first
        assert torch.equal(got, first)
    assert (why := complaint(first, ref, tol, pages.fmt)) is None, why


@pytest.mark.parametrize("fmt,reading,dims", WITH_DIMS)
@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("any_scale", [False, True])
def test_formats_dims_and_splits(fmt, reading, dims, splits, any_scale):
    if any_scale and fmt is not E4M3:
        return  # e4m3 blocks alone have a scale that need not be a power of two
    pages = Pages([1, 700, 33, 129, 1000, 64, 130], 2, dims, 32, fmt, seed=splits, any_scale=any_scale, device=DEV)
    check(pages, 6, [1, 200, 0, 129, 3, 64, 2], 1 / math.sqrt(dims[0]), splits=splits, reading=reading)


@pytest.mark.parametrize("fmt,reading", WAYS)
@pytest.mark.parametrize("window", [1, 2, 31, 100, 128, 500])
@pytest.mark.parametrize("splits", [1, 3])
def test_windows(fmt, reading, window, splits):
    for dims in ((128, 128), (256, 256)):
        pages = Pages([900, 260, 5, 2000, 129], 2, dims, 32, fmt, seed=7, device=DEV)
        check(pages, 4, [300, 260, 5, 0, 129], 0.09, window=window, splits=splits, reading=reading)


@pytest.mark.parametrize("fmt,reading", WAYS)
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 96, 128, 256])
def test_block_sizes(fmt, reading, bs):
    for dims in ((128, 128), (256, 128)):
        check(Pages([517, 130], 2, dims, bs, fmt, seed=bs, device=DEV), 4, [300, 130], 0.09, splits=1, reading=reading)


@pytest.mark.parametrize("fmt,reading", WAYS)
@pytest.mark.parametrize("splits", [1, 2])
def test_bad_blocks_are_skipped(fmt, reading, splits):
    for dims in ((128, 128), (256, 256)):
        pages = Pages([300, 200], 2, dims, 32, fmt, seed=3, device=DEV)
        tables = pages.tables.clone()
        tables[0, 3], tables[1, 0], tables[1, 5] = -1, 10 ** 6, pages.pools[0].shape[0]
        gone = {0: [3], 1: [0, 5]}
        hidden = lambda b: torch.tensor([t // 32 in gone[b] for t in range(512)], device=DEV)
        check(pages, 4, [150, 200], 0.09, tables=tables, flag=1, hidden=hidden, splits=splits, reading=reading)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("splits", [0, 1])
def test_short_chunks_over_long_pages_read_directly(D, bs, splits):
    """Every slot of the ring of codes many times over, by many CTAs at once, again and again: the same bits each time."""
    lens = [700 + 953 * b for b in range(16)]
    news = [1 + b for b in range(16)]
    pages = Pages(lens, 4, (D, D), bs, E4M3, seed=D + bs, device=DEV)
    check(pages, 16, news, 1 / math.sqrt(D), splits=splits, reading=DIRECT, repeats=10)
