"""The choice of blocks and the block bounds at the edges of their numbers."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import block_scaled as O
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


@pytest.mark.parametrize("n,seqs", [(300, 1), (300, 40), (1500, 1)])
@pytest.mark.parametrize("bad", [float("nan"), -float("nan")])
def test_a_query_row_with_a_nan_scores_lowest(n, seqs, bad):
    # one launch and two; a row with a NaN has no score, the block's is that of the other rows
    rng = np.random.default_rng(n + seqs)
    hk, rep, d, bs, top_k = 2, 4, 128, 16, 20
    mid = rng.normal(size=(n, hk, d))
    bounds = torch.from_numpy(np.stack([mid - 0.3, mid + 0.3], 2)).to(torch.bfloat16)
    q = torch.from_numpy(rng.normal(size=(seqs, hk * rep, 1, d))).to(torch.bfloat16)
    q[:, 1] *= 4  # a row that would decide the choice
    clean = q.clone()
    q[:, 1, 0, 5] = bad      # KV head 0: one of its rows
    q[:, rep:, 0, 77] = bad  # KV head 1: all of them
    tables = [[int(x) for x in rng.permutation(n)] for _ in range(seqs)]
    sel = B.select_blocks(q.to(DEV), bounds.to(DEV), i32(tables), i32([n * bs] * seqs), block_size=bs, top_k=top_k)
    rows = [0, 2, 3]
    want = S.choose_blocks(clean[:, rows].double().numpy(), bounds[:, :1].double().numpy(), tables, [n * bs] * seqs, bs,
                           top_k, 1, 1)
    for b in range(seqs):
        assert sel.blocks[b, 0].tolist() == want[b][0], b
        assert sel.blocks[b, 1].tolist() == list(range(top_k - 1)) + [n - 1], b


def test_bounds_of_e4m3_keys_next_to_a_bf16_value():
    # scale * code lies within 2^-25 of a bf16 value (on either side), and rounds to it in f32
    hk, bs, d = 2, 32, 64
    ks = []
    for c in (1.125, 1.25, 1.375, 1.625, 1.75, 1.875):
        for f in range(128, 256):
            target = f * 2.0 ** -8
            for step in (-1, 0, 1):
                s = np.nextafter(np.float32(target / c), np.float32(np.inf if step > 0 else -np.inf)) if step else \
                    np.float32(target / c)
                exact = float(s) * c
                if exact != target and float(np.float32(exact)) == target:
                    ks.append((s, c))
    assert len(ks) > 100
    nb = -(-len(ks) // hk)
    scales = np.ones((nb, hk), np.float32)
    vals = np.zeros((nb, hk, bs, d))
    for i, (s, c) in enumerate(ks):
        scales[i // hk, i % hk] = s
        vals[i // hk, i % hk] = np.where(np.arange(d) % 2 == 0, c, -c)
    pool = O.e4m3_codes(vals)
    keys = O.block_values(pool, scales)
    tables = [list(range(nb))]
    ref = S.update_bounds(np.zeros((nb, hk, 2, d)), keys, tables, [nb * bs], nb * bs, True)
    got = torch.zeros((nb, hk, 2, d), dtype=torch.bfloat16, device=DEV)
    B.update_block_bounds(torch.from_numpy(pool).to(DEV), i32(tables), i32([nb * bs]), got, n_new=nb * bs,
                          k_scales=torch.from_numpy(scales).to(DEV), bits=8, group_size=B.PKV_GROUP_BLOCK)
    assert np.array_equal(got.double().cpu().numpy(), ref)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [128, 256])
def test_bounds_of_affine_keys_next_to_a_bf16_value(bits, d):
    # a bias of 1 and codes times scales far below half an f32 step of it, above and below
    rng = np.random.default_rng(bits + d)
    nb, hk, bs = 6, 2, 32
    words = rng.integers(-2 ** 31, 2 ** 31, size=(nb, hk, bs, d * bits // 32)).astype(np.int32)
    scale = rng.choice([-1.0, 1.0], size=(nb, hk, 1, d // 64)) * 2.0 ** -38 * np.ones((1, 1, bs, 1))
    bias = rng.choice([-1.0, 1.0, 1.5], size=(nb, hk, 1, d // 64)) * np.ones((1, 1, bs, 1))
    per = 32 // bits
    codes = (words.view(np.uint32)[..., None] >> (bits * np.arange(per, dtype=np.uint32))) & np.uint32(2 ** bits - 1)
    codes = codes.reshape(nb, hk, bs, d).astype(np.float64)
    keys = codes * np.repeat(scale, 64, -1) + np.repeat(bias, 64, -1)  # 53 bits hold them exactly
    tables = [[3, 0, 5, 1, 4, 2]]
    ref = S.update_bounds(np.zeros((nb, hk, 2, d)), keys, tables, [nb * bs - 7], nb * bs, False)
    dev = [torch.from_numpy(x).to(torch.bfloat16).to(DEV) for x in (scale, bias)]
    got = torch.zeros((nb, hk, 2, d), dtype=torch.bfloat16, device=DEV)
    B.update_block_bounds(torch.from_numpy(words).to(DEV), i32(tables), i32([nb * bs - 7]), got, n_new=nb * bs,
                          k_scales=dev[0], k_biases=dev[1], bits=bits)
    assert np.array_equal(got.double().cpu().numpy(), ref)


@pytest.mark.parametrize("bits", [16, "e4m3"])
@pytest.mark.parametrize("width,top_k", [(4, 64), (10, 11), (10, 2000)])
def test_a_budget_beyond_the_table(bits, width, top_k):
    # every block is taken: the dense decode's sums in another order, and places past the table's -1
    g = torch.Generator(device=DEV).manual_seed(width + top_k)
    seqs, hk, hq, d, bs = 3, 2, 8, 128, 32
    nb = seqs * width
    lens = i32([width * bs, 1, width * bs - 37])
    tables = torch.randperm(nb, generator=g, device=DEV, dtype=torch.int32).view(seqs, width)
    rows = torch.randn((2, nb, hk, bs, d), generator=g, device=DEV, dtype=torch.bfloat16)
    q = torch.randn((seqs, hq, 1, d), generator=g, device=DEV, dtype=torch.bfloat16)
    kw = {}
    if bits == "e4m3":
        rows = rows.to(torch.float8_e4m3fn)
        kw = dict(bits=8, group_size=B.PKV_GROUP_BLOCK, k_scales=torch.ones((nb, hk), device=DEV),
                  v_scales=torch.ones((nb, hk), device=DEV))
    bounds = torch.zeros((nb, hk, 2, d), dtype=torch.bfloat16, device=DEV)
    blocks = torch.full((seqs, hk, top_k), 7, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = B.sparse_decode_attention(q, rows[0], rows[1], bounds, tables, lens, 0.1, top_k=top_k, blocks=blocks,
                                    error_flag=err, **kw)
    sel = B.select_blocks(q, bounds, tables, lens, block_size=bs, top_k=top_k, error_flag=err)
    apart = B.selected_decode_attention(q, rows[0], rows[1], sel, 0.1, error_flag=err, **kw)
    dense = B.paged_decode_attention(q, rows[0], rows[1], tables, lens, 0.1, error_flag=err, **kw)
    assert int(err) == 0
    held = [width, 1, -(-(width * bs - 37) // bs)]
    for b in range(seqs):
        for h in range(hk):
            pad = [-1] * (top_k - held[b])
            assert blocks[b, h].tolist() == sel.blocks[b, h].tolist() == list(range(held[b])) + pad
            assert sel.tables[b, h].tolist() == [int(t) * hk + h for t in tables[b, :held[b]]] + pad
    # bf16 weights round by 2^-8 of each on both sides, outputs by 2^-8 of the value
    vmax = float(rows[1].float().abs().max())
    for o in (out, apart):
        assert ((o.float() - dense.float()).abs() <= 2.0 ** -7 * dense.float().abs() + 2.0 ** -7 * vmax).all()


@pytest.mark.parametrize("hk,pages", [(2, 60), (8, 1200)])  # one launch of the choice, and two
def test_choices_that_change_from_step_to_step_in_one_workspace(hk, pages):
    # the attention starts beside the choice whose tables it reads, in the memory of the last step's
    g = torch.Generator(device=DEV).manual_seed(pages)
    seqs, hq, d, bs, top_k, steps = 3, 2 * hk, 128, 16, 24, 60
    rows = torch.randn((2, seqs * pages, hk, bs, d), generator=g, device=DEV, dtype=torch.bfloat16)
    tables = torch.randperm(seqs * pages, generator=g, device=DEV, dtype=torch.int32).view(seqs, pages)
    lens = i32([pages * bs, pages * bs - 5, (pages - 7) * bs])
    bounds = torch.empty((seqs * pages, hk, 2, d), dtype=torch.bfloat16, device=DEV)
    B.update_block_bounds(rows[0], tables, lens, bounds, n_new=pages * bs)
    q = torch.randn((steps, seqs, hq, 1, d), generator=g, device=DEV, dtype=torch.bfloat16)
    call = lambda i, **kw: B.sparse_decode_attention(q[i], rows[0], rows[1], bounds, tables, lens, 0.3, top_k=top_k, **kw)
    want = []
    for i in range(steps):
        want.append(call(i))
        torch.cuda.synchronize()
    got = torch.empty_like(q)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    for i in range(steps):
        call(i, out=got[i], workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(got[i], want[i]) for i in range(steps))
    got.zero_()
    with torch.cuda.graph(graph):
        for i in range(steps):
            call(i, out=got[i], workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[i], want[i]) for i in range(steps))


def test_bounds_rebuilt_in_tables_of_nearly_2_31_rows():
    # "at least every length" said with the largest number there is; the rows past the length are not there
    d, bs, length = 128, 2 ** 30 - 32, 40
    k = torch.randn((1, 1, 64, d), device=DEV).to(torch.bfloat16)
    bounds = torch.zeros((1, 1, 2, d), dtype=torch.bfloat16, device=DEV)
    tables, lens, lib = i32([[0, 0]]), i32([length]), B.load_library()
    layout = B.PoolLayout(1, 1, bs, d, 16, 64, 0)
    rc = lib.pkv_update_block_bounds(ctypes.byref(layout), 1, 2, 2 ** 31 - 1, k.data_ptr(), None, None, tables.data_ptr(),
                                     lens.data_ptr(), bounds.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    rows = k[0, 0, :length].float()
    assert torch.equal(bounds[0, 0].float(), torch.stack([rows.amin(0), rows.amax(0)]))
