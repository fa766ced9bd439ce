"""The choice of blocks and the block bounds at the edges of their numbers."""

import numpy as np
import pytest
import torch

from oracle import sparse as S
from quantized_kv_decode_partial_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("n,seqs", [(40, 1), (400, 30), (1500, 1)])  # one launch, and two
def test_addends_that_a_matrix_instruction_cuts(d, n, seqs):
    # Block `high`: 1 and addends just under what its sums keep beside 1 (2^-25, and 2^-23 of
    # their total); block `low`: 1 less such addends, and a step in between. Each f32 sum is off
    # in its own direction, by more together than the step: only the exact sums tell them apart.
    bs, low, high = 16, 3, 17
    q = np.full(d, 2.0 ** -13)
    q[0] = 1.0
    cut = 1.9921875 * 2.0 ** -26
    k = np.zeros((n, d))
    k[low, 0], k[high, 0] = 1.0, 1.0
    k[high, 1:], k[low, 1:] = cut * 2.0 ** 13, -cut * 2.0 ** 13
    for at in range(0, d, 32):  # one larger addend in each instruction
        k[high, at + 4] = k[high, at + 8] = 4 * cut * 2.0 ** 13
    below = float((q * k[high]).sum() - (q * k[low])[2:].sum() - 1.0)  # the step that makes them equal
    unit = 2.0 ** -25
    step = (np.ceil(below / unit) - 2) // 4 * 4 * unit  # a little less, in whole steps of an f32 sum above 1
    k[low, 1] = step / q[1]
    bounds = torch.from_numpy(np.stack([k, k], 1)[:, None]).to(torch.bfloat16)
    assert np.array_equal(bounds[:, 0, 0].double().numpy()[[low, high]], k[[low, high]])  # bf16 values all
    qt = torch.from_numpy(np.tile(q, (seqs, 1, 1, 1))).to(torch.bfloat16)
    assert 0 < float((q * k[high]).sum() - (q * k[low]).sum()) < 8 * unit
    tables = [list(range(n))] * seqs
    ref = S.choose_blocks(qt.double().numpy(), bounds.double().numpy(), tables, [n * bs] * seqs, bs, 3, 1, 1)
    assert ref[0][0] == [0, high, n - 1]
    sel = B.select_blocks(qt.to(DEV), bounds.to(DEV), i32(tables), i32([n * bs] * seqs), block_size=bs, top_k=3)
    assert sel.blocks.tolist() == ref
