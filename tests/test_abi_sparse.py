"""CPU checks of the sparse entry points' C ABI: structures, plans and refusals."""

import ctypes
import os
import re

import pytest

from quantized_kv_decode_partial_gb300 import binding as B
from quantized_kv_decode_partial_gb300 import build as pkv_build

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "pkv_decode.h")
FAKE = 1 << 20  # aligned, never dereferenced: checks come before any CUDA call


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return B.load_library()


def test_struct_layouts_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for cname, cls in (("pkv_sparse_params", B.SparseParams), ("pkv_sparse_plan", B.SparsePlan)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (cname, cname), text, re.S).group(1)
        names = [d.strip().split()[-1] for d in body.split(";") if d.strip()]
        assert names == [f for f, _ in cls._fields_], cname


def layout(**kw):
    d = dict(num_blocks=1000, num_kv_heads=4, block_size=32, head_dim=128, bits=16, group_size=64, v_head_dim=0)
    d.update(kw)
    return B.PoolLayout(*(d[n] for n, _ in B.PoolLayout._fields_))


def test_plan_sizes(lib):
    par = B.DecodeParams(3, 16, 2, 200)
    plan = B.make_sparse_plan(layout(), par, B.SparseParams(64, 1, 2), sm_count=152)
    units = 12
    up = lambda x: -(-x // 256) * 256
    select = up(units * 200 * 4) + up(units * 13 * 4) + up(units * 200 * 8)
    assert plan.select_bytes == select
    att = B.make_plan(layout(num_blocks=4000, num_kv_heads=1), B.DecodeParams(12, 4, 2, 64), sm_count=152)
    assert plan.attention.workspace_bytes == att.workspace_bytes
    assert plan.attention.partition_tokens == att.partition_tokens
    assert plan.workspace_bytes == select + up(units * 64 * 4) + up(units * 4) + att.workspace_bytes
    # no scores where the table holds no more than top_k blocks
    assert B.make_sparse_plan(layout(), par, B.SparseParams(200, 1, 2), sm_count=152).select_bytes == 0


@pytest.mark.parametrize("width,seqs,fmt", [(4, 8, 16), (4, 8, 8), (64, 64, 8), (3, 1, 4), (300, 2, 16)])
@pytest.mark.parametrize("top_k", [300, 1000, 16384, 1 << 20])
def test_a_budget_beyond_the_table_is_planned_as_the_table(lib, width, seqs, fmt, top_k):
    # no unit has more blocks than its table: neither grid nor workspace grow with the budget
    lay = layout(bits=fmt, num_kv_heads=8, group_size=B.PKV_GROUP_BLOCK if fmt == 8 else 64)
    par = B.DecodeParams(seqs, 32, 1, width)
    plan = lambda k: B.make_sparse_plan(lay, par, B.SparseParams(k, 1, 1), sm_count=152)
    assert plan(top_k).workspace_bytes == plan(width).workspace_bytes
    # a choice of the caller's own may name top_k blocks: partitions in proportion, not as many as
    # the table's few rows would take
    own = plan(top_k).attention
    assert own.max_partitions * own.partition_tokens >= top_k * 32
    assert own.partition_tokens >= 256 or own.max_partitions <= 16


@pytest.mark.parametrize("par,sparse,code", [
    ((1, 16, 1, 50, 0, 0), (8, 1, 1), B.PKV_OK),
    ((1, 16, 1, 50, 0, 0), (1, 0, 1), B.PKV_OK),
    ((1, 16, 1, 50, 0, 0), (0, 0, 1), B.PKV_ERR_BAD_PARAMS),
    ((1, 16, 1, 50, 0, 0), (8, -1, 1), B.PKV_ERR_BAD_PARAMS),
    ((1, 16, 1, 50, 0, 0), (8, 1, 0), B.PKV_ERR_BAD_PARAMS),
    ((1, 16, 1, 50, 0, 0), (8, 4, 5), B.PKV_ERR_BAD_PARAMS),
    ((1, 16, 1, 50, 0, 0), (8, 2**31 - 1, 2**31 - 1), B.PKV_ERR_BAD_PARAMS),
    ((1, 16, 1, 50, 0, 0), (1 << 27, 1, 1), B.PKV_ERR_BAD_PARAMS),      # 2^32 rows
    ((1, 16, 2, 50, 0, 0), (8, 1, 1), B.PKV_ERR_BAD_PARAMS),            # two new rows may lie in two blocks
    ((1, 16, 2, 50, 0, 0), (8, 1, 2), B.PKV_OK),
    ((1, 16, 1, 50, 0, 64), (8, 1, 1), B.PKV_ERR_BAD_PARAMS),           # windows
    ((16384, 16, 1, 50, 0, 0), (8, 1, 1), B.PKV_ERR_BAD_PARAMS),        # 65536 units
    ((16383, 16, 1, 50, 0, 0), (8, 1, 1), B.PKV_OK),
    ((1, 15, 1, 50, 0, 0), (8, 1, 1), B.PKV_ERR_BAD_PARAMS),
    ((1, 260, 1, 50, 0, 0), (8, 1, 1), B.PKV_ERR_UNSUPPORTED_SHAPE),
])
def test_parameters(lib, par, sparse, code):
    rc = lib.pkv_make_sparse_plan(ctypes.byref(layout()), ctypes.byref(B.DecodeParams(*par)),
                                  ctypes.byref(B.SparseParams(*sparse)), 152, ctypes.byref(B.SparsePlan()))
    assert rc == code


def refs(lay=None, par=None, sparse=None):
    return (ctypes.byref(lay or layout()), ctypes.byref(par or B.DecodeParams(1, 16, 1, 50)),
            ctypes.byref(sparse or B.SparseParams(8, 1, 1)))


def test_select_validates_before_cuda(lib):
    def call(q=FAKE, bounds=FAKE, tables=FAKE, lens=FAKE, blocks=None, ct=FAKE, cl=FAKE, ws=FAKE, n=1 << 30, **kw):
        return lib.pkv_select_blocks(*refs(**kw), q, bounds, tables, lens, blocks, ct, cl, ws, n, None, None)

    for name in ("q", "bounds", "tables", "lens", "ct", "cl"):
        assert call(**{name: None}) == B.PKV_ERR_NULL_POINTER, name
    for name in ("q", "bounds", "ws"):
        assert call(**{name: FAKE + 8}) == B.PKV_ERR_MISALIGNED, name
    for name in ("tables", "lens", "blocks", "ct", "cl"):
        assert call(**{name: FAKE + 2}) == B.PKV_ERR_MISALIGNED, name
    assert call(ws=None) == B.PKV_ERR_WORKSPACE_TOO_SMALL and call(n=100) == B.PKV_ERR_WORKSPACE_TOO_SMALL
    assert call(lay=layout(head_dim=96)) == B.PKV_ERR_BAD_LAYOUT


def test_sparse_attention_validates_before_cuda(lib):
    def call(q=FAKE, k=FAKE, ks=FAKE, bounds=FAKE, tables=FAKE, blocks=None, out=FAKE, ws=FAKE, n=1 << 30, **kw):
        return lib.pkv_sparse_decode_attention(*refs(**kw), q, k, FAKE, ks, None, ks, None, bounds, tables, FAKE, 0.1,
                                               blocks, out, ws, n, None, None)

    for name in ("q", "k", "bounds", "tables", "out"):
        assert call(**{name: None}) == B.PKV_ERR_NULL_POINTER, name
    assert call(bounds=FAKE + 8) == B.PKV_ERR_MISALIGNED and call(blocks=FAKE + 1) == B.PKV_ERR_MISALIGNED
    assert call(ws=FAKE + 8) == B.PKV_ERR_MISALIGNED
    assert call(ws=None) == B.PKV_ERR_WORKSPACE_TOO_SMALL and call(n=100) == B.PKV_ERR_WORKSPACE_TOO_SMALL
    e4m3 = layout(bits=8, group_size=B.PKV_GROUP_BLOCK)
    assert call(lay=e4m3, ks=None) == B.PKV_ERR_NULL_POINTER
    assert call(lay=layout(bits=8)) == B.PKV_ERR_NULL_POINTER  # affine pages without biases
    rc = lib.pkv_selected_decode_attention(*refs(), FAKE, FAKE, FAKE, None, None, None, None, None, FAKE, 0.1, FAKE, FAKE,
                                           1 << 30, None, None)
    assert rc == B.PKV_ERR_NULL_POINTER


def test_bounds_validate_before_cuda(lib):
    def call(lay=None, seqs=1, width=50, n=1, k=FAKE, ks=None, kb=None, tables=FAKE, lens=FAKE, bounds=FAKE):
        return lib.pkv_update_block_bounds(ctypes.byref(lay or layout()), seqs, width, n, k, ks, kb, tables, lens, bounds,
                                           None, None)

    assert call(n=0) == B.PKV_OK  # nothing to do
    for name in ("k", "tables", "lens", "bounds"):
        assert call(**{name: None}) == B.PKV_ERR_NULL_POINTER, name
    assert call(bounds=FAKE + 8) == B.PKV_ERR_MISALIGNED and call(k=FAKE + 8) == B.PKV_ERR_MISALIGNED
    for bad in (dict(seqs=0), dict(seqs=65536), dict(width=0), dict(n=-1), dict(width=1 << 27)):
        assert call(**bad) == B.PKV_ERR_BAD_PARAMS, bad
    assert call(lay=layout(bits=8)) == B.PKV_ERR_NULL_POINTER
    assert call(lay=layout(bits=8), ks=FAKE) == B.PKV_ERR_NULL_POINTER
    assert call(lay=layout(bits=8, group_size=B.PKV_GROUP_BLOCK)) == B.PKV_ERR_NULL_POINTER
    assert call(lay=layout(bits=8, group_size=B.PKV_GROUP_BLOCK), ks=FAKE + 2) == B.PKV_ERR_MISALIGNED
