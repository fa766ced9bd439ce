"""CPU checks of the C ABI of prompt attention: plans, and what is refused before any CUDA call."""

import ctypes
import math

import pytest

from quantized_kv_decode_partial_gb300 import binding as B
from quantized_kv_decode_partial_gb300 import build as pkv_build

FAKE = 1 << 20  # aligned, never dereferenced: checks come before any CUDA call


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return B.load_library()


def layout(**kw):
    lay = B.PoolLayout(100, 2, 32, 128, 16, 64)
    for k, v in kw.items():
        setattr(lay, k, v)
    return lay


def params(**kw):
    par = B.PrefillParams(2, 100, 8, 10, 0, 0, 0)
    for k, v in kw.items():
        setattr(par, k, v)
    return par


def plan(lib, lay, par, sms=152):
    out = B.PrefillPlan()
    return lib.pkv_make_prefill_plan(ctypes.byref(lay), ctypes.byref(par), sms, ctypes.byref(out)), out


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 256), (192, 128), (256, 128), (128, 256)])
@pytest.mark.parametrize("rep", [1, 3, 4, 64])
def test_plans(lib, dk, dv, rep):
    rc, p = plan(lib, layout(head_dim=dk, v_head_dim=dv), params(num_q_heads=2 * rep))
    assert rc == B.PKV_OK
    assert p.unit_tokens in (128 // rep, 2 * (128 // rep)) and p.smem_bytes <= 227 * 1024
    # units hold every way of dealing 100 tokens to 2 sequences
    for n in range(101):
        starts = [0, n, 100]
        first = [starts[b] // p.unit_tokens + b for b in range(2)]
        need = [-(-(starts[b + 1] - starts[b]) // p.unit_tokens) for b in range(2)]
        assert first[0] + need[0] <= first[1] or need[0] == 0 and first[1] >= first[0]
        assert first[1] + need[1] <= p.units
    assert (p.workspace_bytes == 0) == (p.splits == 1)


def test_values_are_written_where_many_tokens_share_keys(lib):
    e4m3 = dict(bits=8, group_size=B.PKV_GROUP_BLOCK)
    few, many = params(num_tokens=30, num_q_heads=32, splits=1), params(num_tokens=1000, num_q_heads=32, splits=1)
    lay = layout(num_kv_heads=8, **e4m3)
    assert plan(lib, lay, few)[1].value_blocks == 0 and plan(lib, lay, few)[1].workspace_bytes == 0
    p = plan(lib, lay, many)[1]
    assert p.value_blocks == 2 * 3 and p.workspace_bytes == 6 * 8 * 128 * 256 * 2  # tables of 320 rows
    for reading, blocks in ((1, 0), (2, 6)):
        few.reading = many.reading = reading
        assert plan(lib, lay, few)[1].value_blocks == plan(lib, lay, many)[1].value_blocks == blocks
    # a window bounds them by the tokens; more than 8 GB are written for the asking alone
    lay, wide = layout(num_kv_heads=8, num_blocks=70000, **e4m3), dict(num_tokens=1000, num_q_heads=32, max_blocks_per_seq=33000)
    assert plan(lib, lay, params(window=300, **wide))[1].value_blocks == 1000 // 128 + 1 + 2 * (300 // 128 + 3)
    assert plan(lib, lay, params(**wide))[1].value_blocks == 0
    assert plan(lib, lay, params(reading=2, **wide))[1].value_blocks == 2 * 8250
    # rows beyond 31 bits are never written
    assert plan(lib, lay, params(num_seqs=300, reading=2, **wide))[0] == B.PKV_ERR_UNSUPPORTED_SHAPE  # 300 * 8250 * 8 * 128
    assert plan(lib, layout(), params(reading=2))[1].value_blocks == 0  # bf16 pages are read as they are


@pytest.mark.parametrize("bits", [4, 8])
def test_affine_pages_are_read_by_values(lib, bits):
    lay = layout(num_kv_heads=8, bits=bits)
    for n in (30, 1000):
        p = plan(lib, lay, params(num_tokens=n, num_q_heads=32, splits=1))[1]
        assert p.value_blocks == 6 and p.workspace_bytes == 6 * 8 * 128 * 256 * 2 + 256  # and the factors
    assert plan(lib, lay, params(num_q_heads=32, reading=1))[0] == B.PKV_ERR_UNSUPPORTED_SHAPE


def test_splits_fill_the_gpu_and_can_be_set(lib):
    # one tile of queries over a long cache; many tiles
    assert plan(lib, layout(), params(num_seqs=1, num_tokens=16, max_blocks_per_seq=2000))[1].splits > 8
    assert plan(lib, layout(num_kv_heads=8), params(num_seqs=1, num_tokens=100000, num_q_heads=32, max_blocks_per_seq=3200))[1].splits == 1
    rc, p = plan(lib, layout(), params(splits=5))
    assert rc == B.PKV_OK and p.splits == 5 and p.workspace_bytes == 5 * 100 * 8 * 130 * 4


@pytest.mark.parametrize("lay,par,code", [
    (dict(block_size=4), dict(), B.PKV_ERR_BAD_LAYOUT), (dict(head_dim=96), dict(), B.PKV_ERR_BAD_LAYOUT),
    (dict(head_dim=64, v_head_dim=128), dict(), B.PKV_ERR_UNSUPPORTED_SHAPE),
    (dict(), dict(num_seqs=0), B.PKV_ERR_BAD_PARAMS), (dict(), dict(num_seqs=65536), B.PKV_ERR_BAD_PARAMS),
    (dict(), dict(num_tokens=-1), B.PKV_ERR_BAD_PARAMS), (dict(), dict(num_q_heads=3), B.PKV_ERR_BAD_PARAMS),
    (dict(), dict(num_q_heads=0), B.PKV_ERR_BAD_PARAMS), (dict(), dict(num_q_heads=130), B.PKV_ERR_UNSUPPORTED_SHAPE),
    (dict(), dict(max_blocks_per_seq=0), B.PKV_ERR_BAD_PARAMS), (dict(), dict(max_blocks_per_seq=1 << 26), B.PKV_ERR_BAD_PARAMS),
    (dict(), dict(max_blocks_per_seq=(1 << 26) - 8), B.PKV_ERR_BAD_PARAMS),
    (dict(), dict(window=-1), B.PKV_ERR_BAD_PARAMS), (dict(), dict(splits=-1), B.PKV_ERR_BAD_PARAMS),
    (dict(), dict(splits=65), B.PKV_ERR_BAD_PARAMS), (dict(), dict(reading=3), B.PKV_ERR_BAD_PARAMS), (dict(), dict(reading=-1), B.PKV_ERR_BAD_PARAMS), (dict(), dict(num_tokens=1 << 28), B.PKV_ERR_BAD_PARAMS),
])
def test_shapes_that_are_refused(lib, lay, par, code):
    assert plan(lib, layout(**lay), params(**par))[0] == code


def attend(lib, lay=None, par=None, q=FAKE, strides=(0, 1024, 128), k=FAKE, tables=FAKE, starts=FAKE, scale=0.1, out=FAKE,
           ks=None, ws=FAKE):
    s = B.RowStrides(*strides)
    return lib.pkv_paged_prefill_attention(
        ctypes.byref(lay or layout()), ctypes.byref(par or params()), q, ctypes.byref(s), k, FAKE, ks, None, None, None, tables,
        FAKE, starts, scale, out, ws, 0, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(par=params(num_tokens=0)), B.PKV_OK),
    (dict(q=None), B.PKV_ERR_NULL_POINTER), (dict(k=None), B.PKV_ERR_NULL_POINTER), (dict(tables=None), B.PKV_ERR_NULL_POINTER),
    (dict(starts=None), B.PKV_ERR_NULL_POINTER), (dict(out=None), B.PKV_ERR_NULL_POINTER),
    (dict(q=FAKE + 8), B.PKV_ERR_MISALIGNED), (dict(k=FAKE + 8), B.PKV_ERR_MISALIGNED), (dict(out=FAKE + 2), B.PKV_ERR_MISALIGNED),
    (dict(starts=FAKE + 2), B.PKV_ERR_MISALIGNED), (dict(ws=FAKE + 4), B.PKV_ERR_MISALIGNED),
    (dict(strides=(0, 1020, 128)), B.PKV_ERR_MISALIGNED), (dict(strides=(0, 0, 128)), B.PKV_ERR_BAD_PARAMS),
    (dict(strides=(0, 1024, 0)), B.PKV_ERR_BAD_PARAMS), (dict(strides=(0, 1 << 38, 128)), B.PKV_ERR_BAD_PARAMS),
    (dict(scale=math.nan), B.PKV_ERR_BAD_PARAMS), (dict(scale=-math.inf), B.PKV_ERR_BAD_PARAMS),
])
def test_calls_that_are_refused(lib, kw, code):
    assert attend(lib, **kw) == code
