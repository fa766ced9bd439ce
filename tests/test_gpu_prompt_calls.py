"""What the binding remembers of a prompt's calls, whose shapes change with every step's token count."""

import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv
from quantized_kv_decode_partial_gb300 import binding
from test_gpu_rotate import DEV, freqs, randn

pytestmark = pytest.mark.gpu


def test_many_token_counts_leave_the_decode_calls_alone():
    D, bs, n = 64, 32, 1100
    pools = [randn(n // bs + 1, 1, bs, D, seed=i) for i in (1, 2)]
    tables = torch.arange(pools[0].shape[0], dtype=torch.int32, device=DEV)[None]
    lens, f, x = torch.tensor([n], dtype=torch.int32, device=DEV), freqs(D // 2), randn(n, 1, D, seed=3)
    zero = torch.zeros_like(lens)
    pos, starts = torch.arange(n, dtype=torch.int32, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    decode = lambda: pkv.paged_decode_attention(x[:1, :, None], *pools, tables, lens, 0.125)
    decode()
    held = set(binding._calls)
    first = {}
    for t in range(1, n):
        q = x[:t]
        got = (pkv.norm_rotate(q, None, pos[:t], f)[0], pkv.norm_rotate_append(q, q, q, None, f, tables, zero, *pools, query_starts=starts),
               pkv.paged_prefill_attention(q, *pools, tables, lens, starts, 0.125))
        if t == 5:
            first = [y.clone() for y in got]
    assert held <= set(binding._calls) and len(binding._prompt_calls) <= 1025
    again = (pkv.norm_rotate(x[:5], None, pos[:5], f)[0], pkv.norm_rotate_append(x[:5], x[:5], x[:5], None, f, tables, zero, *pools,
                                                                                  query_starts=starts))
    assert torch.equal(again[0], first[0]) and torch.equal(again[1][:1], first[1][:1])
