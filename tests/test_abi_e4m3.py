"""CPU checks of the C ABI for e4m3 pages: which layouts are planned, what is refused."""

import ctypes

import pytest

from quantized_kv_decode_partial_gb300 import binding as B
from quantized_kv_decode_partial_gb300 import build as pkv_build

FAKE = 1 << 20  # aligned, never dereferenced: checks come before any CUDA call


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return B.load_library()


def plan_rc(lib, lay, par):
    return lib.pkv_make_plan(ctypes.byref(lay), ctypes.byref(par), 152, ctypes.byref(B.Plan()))


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 256), (192, 128), (256, 128), (128, 256)])
@pytest.mark.parametrize("bs", [8, 16, 32, 96])
def test_layouts_and_query_rows(lib, dk, dv, bs):
    for nq in (1, 8, 9, 33, 64, 65):
        lay = B.PoolLayout(100, 2, bs, dk, 8, B.PKV_GROUP_BLOCK, dv)
        rc = plan_rc(lib, lay, B.DecodeParams(3, 2 * nq, 1, 8))
        assert rc == (B.PKV_OK if nq <= 64 else B.PKV_ERR_UNSUPPORTED_SHAPE)


@pytest.mark.parametrize("lay,code", [
    (B.PoolLayout(100, 2, 32, 128, 4, B.PKV_GROUP_BLOCK), B.PKV_ERR_BAD_LAYOUT),  # 4-bit codes are affine
    (B.PoolLayout(100, 2, 32, 96, 8, B.PKV_GROUP_BLOCK), B.PKV_ERR_BAD_LAYOUT),
    (B.PoolLayout(100, 2, 4, 128, 8, B.PKV_GROUP_BLOCK), B.PKV_ERR_BAD_LAYOUT),
    (B.PoolLayout(100, 2, 48, 128, 8, B.PKV_GROUP_BLOCK), B.PKV_ERR_BAD_LAYOUT),
    (B.PoolLayout(100, 2, 32, 128, 8, -2), B.PKV_ERR_BAD_LAYOUT),
    (B.PoolLayout(100, 2, 32, 128, 8, 0), B.PKV_ERR_BAD_LAYOUT),
    (B.PoolLayout(100, 2, 32, 64, 8, 64), B.PKV_ERR_BAD_LAYOUT),  # affine pages have no 64-dim heads
    (B.PoolLayout(100, 2, 32, 64, 8, B.PKV_GROUP_BLOCK, 128), B.PKV_ERR_UNSUPPORTED_SHAPE),
])
def test_layouts_that_are_refused(lib, lay, code):
    assert plan_rc(lib, lay, B.DecodeParams(1, 4, 1, 4)) == code


def test_the_cuda_core_contraction_is_refused(lib):
    lay = B.PoolLayout(100, 2, 32, 128, 8, B.PKV_GROUP_BLOCK)
    assert plan_rc(lib, lay, B.DecodeParams(1, 4, 1, 4, 0, 0, B.PKV_CONTRACTION_CUDA_CORE)) == B.PKV_ERR_UNSUPPORTED_SHAPE


def test_scale_planes_are_required_and_biases_are_not(lib):
    lay, par = B.PoolLayout(100, 2, 32, 128, 8, B.PKV_GROUP_BLOCK), B.DecodeParams(1, 4, 1, 4)

    def attend(ks, vs, k=FAKE):
        return lib.pkv_paged_decode_attention(ctypes.byref(lay), ctypes.byref(par), FAKE, k, FAKE, ks, None, vs, None,
                                              FAKE, FAKE, 0.1, FAKE, FAKE, 1 << 30, None, None)

    assert attend(None, FAKE) == B.PKV_ERR_NULL_POINTER and attend(FAKE, None) == B.PKV_ERR_NULL_POINTER
    assert attend(FAKE + 2, FAKE) == B.PKV_ERR_MISALIGNED and attend(FAKE, FAKE + 1) == B.PKV_ERR_MISALIGNED
    assert attend(FAKE, FAKE, FAKE + 8) == B.PKV_ERR_MISALIGNED

    def append(ks, vs, n=1):
        return lib.pkv_paged_append(ctypes.byref(lay), 1, 4, n, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ks, None, vs, None,
                                    None, None)

    assert append(None, FAKE) == B.PKV_ERR_NULL_POINTER and append(FAKE, FAKE + 2) == B.PKV_ERR_MISALIGNED
    assert append(FAKE, FAKE, -1) == B.PKV_ERR_BAD_PARAMS


def test_the_fused_call_is_refused(lib):
    lay, par = B.PoolLayout(100, 2, 32, 128, 8, B.PKV_GROUP_BLOCK), B.DecodeParams(1, 4, 1, 4)
    rc = lib.pkv_paged_decode_append_attention(ctypes.byref(lay), ctypes.byref(par), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                               None, FAKE, None, FAKE, FAKE, 0.1, FAKE, FAKE, 1 << 30, None, None)
    assert rc == B.PKV_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("seqs,rows,d,rep,parts", [
    (4, 60000, 128, 4, 42),   # 512 CTAs, a little over one wave of 456: three waves
    (32, 8000, 128, 4, 5),
    (32, 16000, 64, 4, 7),    # four CTAs per SM
    (2, 8192, 128, 4, 26),    # CTAs of 256 KB would not fill a wave: one wave of shorter ones
    (8, 40003, 128, 4, 16),   # over two waves: as it was
    (1, 8192, 256, 4, 16),    # half a wave or less: one cluster per KV head
])
def test_partitions_fill_whole_waves(lib, seqs, rows, d, rep, parts):
    hk = 4 if seqs == 1 else 8
    blocks = -(-rows // 32)
    plan = B.make_plan(B.PoolLayout(seqs * blocks, hk, 32, d, 8, B.PKV_GROUP_BLOCK),
                       B.DecodeParams(seqs, hk * rep, 1, blocks, 0, 0, 0, B.PKV_SCHEDULE_PARTITIONS), 152)
    assert plan.max_partitions == parts
    assert plan.partition_tokens * plan.max_partitions >= rows


@pytest.mark.parametrize("d,nq,units,rows,balanced", [
    # runs of a unit that the merge would read one after the other: 1824 runs over few units
    (128, 16, 1, 16416, 0), (128, 16, 1, 131072, 0), (128, 16, 4, 32768, 0), (128, 32, 8, 131072, 0),
    (256, 16, 1, 8224, 0), (256, 16, 16, 32768, 0), (64, 32, 2, 131072, 0), (64, 32, 16, 131072, 0),
    # runs too short
    (128, 16, 64, 16416, 0), (256, 16, 32, 16416, 0), (128, 32, 64, 8224, 0),
    # many units of many rows
    (128, 16, 64, 32768, 1), (128, 32, 64, 16416, 1), (128, 32, 16, 131072, 1), (256, 16, 32, 32768, 1),
    (64, 32, 64, 16416, 1), (128, 16, 512, 32768, 1),
])
def test_balanced_schedule_where_units_have_few_runs(lib, d, nq, units, rows, balanced):
    hk = 8 if units % 8 == 0 else 1
    lay = B.PoolLayout(units // hk * rows // 32, hk, 32, d, 8, B.PKV_GROUP_BLOCK)
    plan = B.make_plan(lay, B.DecodeParams(units // hk, hk * nq, 1, rows // 32), sm_count=152)
    assert plan.balanced == balanced


@pytest.mark.parametrize("d,nq,hk,rows,cluster", [
    (256, 4, 4, 6144, True), (256, 8, 1, 8192, True), (256, 4, 4, 8704, False), (256, 4, 2, 12288, False),
    (128, 4, 2, 8192, True), (128, 8, 2, 12288, True), (128, 4, 2, 16384, False), (64, 4, 2, 16384, True),
    (64, 4, 2, 24576, False), (128, 16, 1, 6144, False), (64, 9, 1, 12288, False)])
def test_sixteen_partitions_in_a_cluster(lib, d, nq, hk, rows, cluster):
    lay = B.PoolLayout(rows // 32, hk, 32, d, 8, B.PKV_GROUP_BLOCK)
    plan = B.make_plan(lay, B.DecodeParams(1, hk * nq, 1, rows // 32), sm_count=152)
    assert (plan.merge_in_cluster, plan.max_partitions == 16, plan.workspace_bytes == 0) == (cluster,) * 3
