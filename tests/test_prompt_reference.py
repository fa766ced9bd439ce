"""The bounds for prompt attention over pages of codes, on the CPU: they let a model of the kernels' roundings pass and reject
outputs with a gain, a window one off, a lost block, a block under another scale, rows of another head."""

import pytest
import torch

from prompt_reference import E4M3, Pages, affine, attention, complaint

FORMATS = [dict(), E4M3, dict(bits=8), dict(bits=4)]
LENS, NEWS, SCALE = [900, 260, 5], [100, 80, 5], 0.09


def case(fmt, D, window, any_scale=False):
    pages = Pages(LENS, 2, (D, D), 32, fmt, seed=1, any_scale=any_scale)
    q = torch.randn(sum(NEWS), 4, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    return pages, q, *attention(q, pages, NEWS, SCALE, window)


def model(pages, q, window, **kw):
    """The kernel's roundings: 16-bit weights, for affine pages 16-bit keys and values, outputs in bf16."""
    half = lambda x: x.float().to(torch.float16).double()
    values = pages.values
    if affine(pages.fmt):
        pages.values = [half(x * 2.0 ** 8) / 2.0 ** 8 for x in values]
        out, _ = attention(q, pages, NEWS, SCALE, window, rounded=lambda p: half(p * 2.0 ** 7) / 2.0 ** 7, **kw)
        pages.values = values
    else:
        out, _ = attention(q, pages, NEWS, SCALE, window, rounded=lambda p: p.to(torch.bfloat16).double(), **kw)
    return out.to(torch.bfloat16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window", [0, 1, 100, 500])
@pytest.mark.parametrize("any_scale", [False, True])
def test_roundings_pass_and_mistakes_do_not(fmt, D, window, any_scale):
    pages, q, ref, tol = case(fmt, D, window, any_scale)
    good = model(pages, q, window)
    assert complaint(good, ref, tol, fmt) is None
    for gain in (1.01, 0.99, 1.1):
        assert complaint((good.double() * gain).to(torch.bfloat16), ref, tol, fmt)
    for other in [n for n in (window - 1, window + 1) if window and n]:
        assert complaint(model(pages, q, other), ref, tol, fmt)
    for late in (-1, 1):
        assert complaint(model(pages, q, window, late=late), ref, tol, fmt)
    if window == 0 or window == 500:
        lost = lambda b: (torch.arange(1024) // 32 == 20) if b == 0 else torch.zeros(1024, dtype=torch.bool)
        assert complaint(model(pages, q, window, hidden=lost), ref, tol, fmt)
    assert complaint(good.roll(1, 1), ref, tol, fmt)  # another head's
    assert complaint(good.roll(1, 0), ref, tol, fmt)  # another token's
    for which in (0, 1):  # one block's keys or values under twice its scale, where it is seen
        block = int(pages.tables[0, 26])
        pages.values[which][block] *= 2.0
        assert complaint(model(pages, q, window), ref, tol, fmt) or window == 1 and which == 0
        pages.values[which][block] /= 2.0
