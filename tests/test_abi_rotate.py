"""CPU checks of the C ABI of norm and rotation: what is refused before any CUDA call."""

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


def rotation(**kw):
    r = B.Rotation(128, 128, 0, 1, 0)
    r.eps, r.amplitude = 1e-6, 1.0
    for k, v in kw.items():
        if k == "sections":
            r.sections[:len(v)] = v
        else:
            setattr(r, k, v)
    return r


def strides(heads, dim=128, **kw):
    s = B.RowStrides(0, heads * dim, dim)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def rotate(lib, r=None, seqs=0, tokens=4, hq=8, hk=2, q=FAKE, qs=None, k=FAKE, wq=None, positions=FAKE, freq=FAKE, q_out=FAKE,
           qos=None):
    """With seqs = 0 nothing is launched whatever passes the checks; with 1 the call must be refused."""
    ref = ctypes.byref
    r = r or rotation()
    return lib.pkv_norm_rotate(ref(r), seqs, tokens, hq, hk, q, ref(qs or strides(hq)), k, ref(strides(hk)), wq, None,
                               positions, freq, q_out, ref(qos or strides(hq)), FAKE, ref(strides(hk)), None)


@pytest.mark.parametrize("r", [
    rotation(), rotation(rot_dims=8), rotation(head_dim=64, rot_dims=64), rotation(head_dim=192, rot_dims=64),
    rotation(head_dim=256, rot_dims=256), rotation(pairing=1),
    rotation(num_axes=3, sections=[24, 20, 20]), rotation(num_axes=3, sections=[24, 20, 20], section_order=1),
    rotation(num_axes=4, sections=[16] * 4, section_order=1), rotation(num_axes=2, sections=[0, 64]),
    rotation(num_axes=3, sections=[22, 21, 21], section_order=1), rotation(eps=0.0),
])
def test_rotations_that_pass(lib, r):
    assert rotate(lib, r) == B.PKV_OK


@pytest.mark.parametrize("r,code", [
    (rotation(head_dim=96, rot_dims=96), B.PKV_ERR_BAD_LAYOUT),
    (rotation(rot_dims=0), B.PKV_ERR_BAD_PARAMS),
    (rotation(rot_dims=136), B.PKV_ERR_BAD_PARAMS),
    (rotation(rot_dims=60), B.PKV_ERR_BAD_PARAMS),
    (rotation(pairing=2), B.PKV_ERR_BAD_PARAMS),
    (rotation(num_axes=0), B.PKV_ERR_BAD_PARAMS),
    (rotation(num_axes=5), B.PKV_ERR_BAD_PARAMS),
    (rotation(num_axes=2, sections=[32, 31]), B.PKV_ERR_BAD_PARAMS),
    (rotation(num_axes=2, sections=[65, -1]), B.PKV_ERR_BAD_PARAMS),
    (rotation(num_axes=2, sections=[0, 64], section_order=1), B.PKV_ERR_BAD_PARAMS),
    (rotation(num_axes=2, sections=[32, 32], section_order=2), B.PKV_ERR_BAD_PARAMS),
    (rotation(eps=-1.0), B.PKV_ERR_BAD_PARAMS),
    (rotation(eps=math.nan), B.PKV_ERR_BAD_PARAMS),
    (rotation(amplitude=math.inf), B.PKV_ERR_BAD_PARAMS),
    (rotation(weight_offset=math.nan), B.PKV_ERR_BAD_PARAMS),
])
def test_rotations_that_are_refused(lib, r, code):
    assert rotate(lib, r) == code


@pytest.mark.parametrize("kw,code", [
    (dict(hq=0), B.PKV_ERR_BAD_PARAMS), (dict(hk=-1), B.PKV_ERR_BAD_PARAMS), (dict(tokens=-1), B.PKV_ERR_BAD_PARAMS),
    (dict(seqs=65536, tokens=65536), B.PKV_ERR_BAD_PARAMS),
    (dict(q=None), B.PKV_ERR_NULL_POINTER), (dict(k=None), B.PKV_ERR_NULL_POINTER),
    (dict(positions=None), B.PKV_ERR_NULL_POINTER), (dict(freq=None), B.PKV_ERR_NULL_POINTER),
    (dict(q_out=None), B.PKV_ERR_NULL_POINTER),
    (dict(q=FAKE + 8), B.PKV_ERR_MISALIGNED), (dict(q_out=FAKE + 2), B.PKV_ERR_MISALIGNED),
    (dict(positions=FAKE + 2), B.PKV_ERR_MISALIGNED), (dict(wq=FAKE + 1), B.PKV_ERR_MISALIGNED),
    (dict(qs=strides(8, token=1028)), B.PKV_ERR_MISALIGNED),
    (dict(qs=strides(8, token=-1024)), B.PKV_ERR_BAD_PARAMS),
    (dict(qos=strides(8, token=0)), B.PKV_ERR_BAD_PARAMS),  # output rows that overlap
    (dict(qos=strides(8, head=64)), B.PKV_ERR_BAD_PARAMS),
    (dict(qos=strides(8, token=1016)), B.PKV_ERR_BAD_PARAMS),
])
def test_arguments_that_are_refused(lib, kw, code):
    assert rotate(lib, **{"seqs": 1, **kw}) == code


def append(lib, lay=None, r=None, seqs=2, tokens=4, per=2, hq=8, starts=None, positions=FAKE, tables=FAKE, v=FAKE, ks=None,
           vs=None, width=4):
    ref = ctypes.byref
    return lib.pkv_norm_rotate_append(
        ref(lay or B.PoolLayout(10, 2, 32, 128, 16, 64)), ref(r or rotation()), seqs, tokens, per, hq, width, FAKE,
        ref(strides(hq)), FAKE, ref(strides(2)), v, ref(strides(2)), None, None, positions, FAKE, starts, tables, FAKE, FAKE,
        FAKE, ks, None, vs, None, FAKE, ref(strides(hq, seq=2048)), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0, per=0), B.PKV_OK),
    (dict(seqs=0), B.PKV_ERR_BAD_PARAMS), (dict(seqs=65536), B.PKV_ERR_BAD_PARAMS),
    (dict(tokens=5), B.PKV_ERR_BAD_PARAMS), (dict(per=-1), B.PKV_ERR_BAD_PARAMS), (dict(hq=0), B.PKV_ERR_BAD_PARAMS),
    (dict(width=0), B.PKV_ERR_BAD_PARAMS), (dict(width=1 << 26), B.PKV_ERR_BAD_PARAMS),
    (dict(per=0), B.PKV_ERR_NULL_POINTER),  # packed tokens need their starts
    (dict(tables=None), B.PKV_ERR_NULL_POINTER), (dict(v=None), B.PKV_ERR_NULL_POINTER),
    (dict(per=0, starts=FAKE + 2), B.PKV_ERR_MISALIGNED),
    (dict(v=FAKE + 8), B.PKV_ERR_MISALIGNED),
    (dict(positions=None, r=rotation(num_axes=2, sections=[32, 32])), B.PKV_ERR_BAD_PARAMS),
    (dict(r=rotation(head_dim=64, rot_dims=64)), B.PKV_ERR_BAD_LAYOUT),
    (dict(lay=B.PoolLayout(10, 2, 32, 96, 16, 64)), B.PKV_ERR_BAD_LAYOUT),
    (dict(lay=B.PoolLayout(10, 2, 32, 128, 8, B.PKV_GROUP_BLOCK)), B.PKV_ERR_NULL_POINTER),
    (dict(lay=B.PoolLayout(10, 2, 32, 128, 8, B.PKV_GROUP_BLOCK), ks=FAKE, vs=FAKE + 2), B.PKV_ERR_MISALIGNED),
    (dict(lay=B.PoolLayout(10, 2, 32, 128, 8, 64), ks=FAKE, vs=FAKE), B.PKV_ERR_NULL_POINTER),
])
def test_appends_that_are_refused(lib, kw, code):
    assert append(lib, **kw) == code
