"""CPU checks of prompt attention's plans over wide tables of affine pages: the workspace does not grow with the batch."""

import pytest

from quantized_kv_decode_partial_gb300 import binding as B
from test_abi_prefill import layout, lib, params, plan  # noqa: F401  (lib is a fixture)

GB8 = 8 << 30


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("seqs,width,group", [(64, 4096, 16), (256, 32768, 2), (65535, 64, 1024), (15, 4096, 15), (17, 4096, 16),
                                              (3, 200000, 1)])
def test_values_of_a_group_fit_8_gb(lib, bits, seqs, width, group):  # noqa: F811
    lay = layout(num_kv_heads=8, bits=bits)
    for n, q_heads in ((seqs, 32), (100000, 8)):
        rc, p = plan(lib, lay, params(num_seqs=seqs, num_tokens=n, num_q_heads=q_heads, max_blocks_per_seq=width, splits=1))
        assert rc == B.PKV_OK
        per_seq = -(-width * 32 // 128)
        assert p.value_blocks == per_seq * group and p.units == n // p.unit_tokens + group
        assert p.workspace_bytes == p.value_blocks * 8 * 128 * 256 * 2 + -(-2 * group * 8 * 4 // 256) * 256
        assert group == 1 or p.value_blocks * 8 * 128 * 256 * 2 <= GB8
        assert group == seqs or per_seq * (group + 1) * 8 * 128 * 256 * 2 > GB8


def test_a_window_bounds_the_groups_too(lib):  # noqa: F811
    lay = layout(num_kv_heads=8, bits=8)
    wide = dict(num_seqs=2000, num_tokens=4000, num_q_heads=32, max_blocks_per_seq=32768, splits=1)
    p = plan(lib, lay, params(window=300, **wide))[1]
    assert p.value_blocks == 4000 // 128 + 1 + 2000 * 5
    p = plan(lib, lay, params(window=100000, **wide))[1]
    part = 100000 // 128 + 3
    group = (p.value_blocks - 4000 // 128 - 1) // part
    assert p.value_blocks == 4000 // 128 + 1 + group * part and p.value_blocks * 8 * 128 * 256 * 2 <= GB8
    assert (p.value_blocks + part) * 8 * 128 * 256 * 2 > GB8


def test_rows_of_one_sequence_past_31_bits_are_refused(lib):  # noqa: F811
    lay = layout(num_kv_heads=1024, num_blocks=100, bits=8)
    assert plan(lib, lay, params(num_q_heads=1024, max_blocks_per_seq=65536))[0] == B.PKV_ERR_UNSUPPORTED_SHAPE
    assert plan(lib, lay, params(num_q_heads=1024, max_blocks_per_seq=65535 - 3))[0] == B.PKV_OK
