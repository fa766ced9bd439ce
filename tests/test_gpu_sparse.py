"""GPU parity of sparse decode attention: block bounds bit for bit, the choice of blocks
exactly (near ties and ties included), attention over the chosen rows within the decode's
bound.

Attention tolerance: weights round to bf16 (bf16 pages, 2^-8 of each) or fp16 (the others,
2^-11), so the weighted mean is off by at most 2^-8 max|V|; the f32 scores add under 2^-16 of
it, the output's rounding 2^-8 of the value. Bound: 2^-8 |ref| + 2^-8 max|V| + 2^-12 max|V|.
"""

import math
import threading

import numpy as np
import pytest
import torch

import oracle
from oracle import block_scaled as O
from oracle import paged_write
from oracle import sparse as S
from quantized_kv_decode_partial_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Plane:
    """One plane of pages in a format: device tensors, their keyword arguments and float64 values."""

    def __init__(self, rng, fmt, nb, hk, bs, d, drift=1.0):
        x = rng.normal(size=(nb, hk, bs, d)) + drift * rng.normal(size=(nb, hk, 1, d))
        self.fmt, self.scales, self.biases = fmt, None, None
        if fmt == 16:
            self.pool = bf16(x).to(DEV)
            self.values = self.pool.double().cpu().numpy()
        elif fmt == "e4m3":
            s = (2.0 ** rng.integers(-8, -6, size=(nb, hk)) * rng.uniform(0.6, 1, size=(nb, hk))).astype(np.float32)
            codes = O.e4m3_codes(np.clip(x / s[:, :, None, None], -448, 448))
            self.pool = torch.from_numpy(codes).to(DEV).view(torch.float8_e4m3fn)
            self.scales = torch.from_numpy(s).to(DEV)
            self.values = O.block_values(codes, s)
        else:
            codes, s, z = paged_write.quantize_groups(bf16(x).float().numpy(), fmt)
            words = paged_write.pack_codes(codes, fmt).view(np.int32)
            self.pool = torch.from_numpy(words).to(DEV)
            self.scales, self.biases = bf16(s).to(DEV), bf16(z).to(DEV)
            self.values = oracle.dequantize(words, s, z, fmt, 64)

    @property
    def kw(self):
        return dict(bits=8 if self.fmt == "e4m3" else self.fmt,
                    group_size=B.PKV_GROUP_BLOCK if self.fmt == "e4m3" else 64)


def make_tables(rng, lens, bs, extra=2):
    pages = [-(-max(n, 0) // bs) for n in lens]
    perm = rng.permutation(sum(pages) + extra)
    width, at, rows = max(max(pages), 1), 0, []
    for p in pages:
        rows.append([int(x) for x in perm[at:at + p]] + [-1] * (width - p))
        at += p
    return rows, len(perm)


# ------------------------------------------------------------------------------------------ bounds
@pytest.mark.parametrize("fmt,d", [(16, 64), (16, 128), (16, 192), (16, 256), (8, 128), (8, 256), (4, 128), (4, 256),
                                   ("e4m3", 64), ("e4m3", 128), ("e4m3", 192), ("e4m3", 256)])
@pytest.mark.parametrize("bs,lens,n_new", [(32, [1, 32, 33, 100], 1), (32, [7, 64, 90, 300], 40), (8, [30, 9, 8], 5),
                                           (96, [250, 96, 1], 1000), (16, [17, 0, 40], 16)])
def test_bounds_match_the_oracle(fmt, d, bs, lens, n_new):
    rng = np.random.default_rng(d + bs + n_new)
    tables, nb = make_tables(rng, lens, bs)
    k = Plane(rng, fmt, nb, 3, bs, d)
    held = bf16(rng.normal(size=(nb, 3, 2, d))).to(DEV)
    ref = S.update_bounds(held.double().cpu().numpy(), k.values, tables, lens, n_new, whole_blocks=fmt == "e4m3")
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = B.update_block_bounds(k.pool, i32(tables), i32(lens), held, n_new=n_new, k_scales=k.scales,
                                k_biases=k.biases, error_flag=err, **k.kw)
    assert got is held and int(err) == 0
    got = got.double().cpu().numpy()
    if fmt in (4, 8):
        # scale * code is exact in f32 and its sum with the bias rounds once, half a step of
        # 2^-24 relative, before the outward rounding: a bound may sit one bf16 step inside
        # only where the exact value is that close to it
        step = np.ldexp(1.0, np.frexp(ref)[1] - 8)
        bad = got != ref
        assert bad.mean() < 1e-3 and (np.abs(got - ref) <= step)[bad].all()
    else:
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("fmt", [16, 8, 4, "e4m3"])
def test_bounds_token_by_token_are_those_at_once(fmt):
    rng = np.random.default_rng(5)
    lens, bs = [70, 31], 32
    tables, nb = make_tables(rng, lens, bs)
    k = Plane(rng, fmt, nb, 2, bs, 128)
    args = dict(k_scales=k.scales, k_biases=k.biases, **k.kw)
    at_once = torch.zeros((nb, 2, 2, 128), dtype=torch.bfloat16, device=DEV)
    B.update_block_bounds(k.pool, i32(tables), i32(lens), at_once, n_new=70, **args)
    step = torch.full_like(at_once, 7.0)
    for j in range(1, 71):
        B.update_block_bounds(k.pool, i32(tables), i32([j, min(j, 31)]), step, n_new=1, **args)
    used = [x for row, n in zip(tables, lens) for x in row[:-(-n // bs)]]
    assert torch.equal(step[used], at_once[used])
    rest = [x for x in range(nb) if x not in used]
    assert (step[rest] == 7.0).all()


def test_bounds_bad_blocks_and_lengths():
    rng = np.random.default_rng(6)
    k = Plane(rng, 16, 4, 2, 32, 128)
    held = torch.full((4, 2, 2, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.update_block_bounds(k.pool, i32([[0, 9], [1, 2], [3, 3]]), i32([40, 65, -2]), held, n_new=100, error_flag=err)
    assert int(err) == B.PKV_DEVERR_BAD_BLOCK | B.PKV_DEVERR_BAD_SEQ_LEN
    assert (held[1:] == 3.0).all() and (held[0] != 3.0).any()


# ------------------------------------------------------------------------------------------ choice
def run_choice(rng, bounds, q, tables, lens, bs, top_k, first, last, want_err=0):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sel = B.select_blocks(q.to(DEV), bounds.to(DEV), i32(tables), i32(lens), block_size=bs, top_k=top_k,
                          first_blocks=first, last_blocks=last, error_flag=err)
    torch.cuda.synchronize()
    assert int(err) == want_err
    return sel


def check_choice(rng, bounds, q, tables, lens, bs, top_k, first, last):
    sel = run_choice(rng, bounds, q, tables, lens, bs, top_k, first, last)
    ref = S.choose_blocks(q.double().numpy(), bounds.double().numpy(), tables, lens, bs, top_k, first, last)
    hk = bounds.shape[1]
    for b, length in enumerate(lens):
        n = -(-length // bs)
        for h in range(hk):
            want = ref[b][h]
            pad = [-1] * (top_k - len(want))
            assert sel.blocks[b, h].tolist() == want + pad, (b, h)
            assert sel.tables[b, h].tolist() == [tables[b][j] * hk + h for j in want] + pad
            assert int(sel.lens[b, h]) == (len(want) - 1) * bs + length - (n - 1) * bs
    return sel


def random_bounds(rng, nb, hk, d, width=0.5):
    mid = rng.normal(size=(nb, hk, d))
    half = np.abs(rng.normal(size=(nb, hk, d))) * width
    return bf16(np.stack([mid - half, mid + half], 2))


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("rep,n", [(1, 1), (4, 2), (3, 3), (16, 4)])
def test_choice_matches_the_oracle(d, rep, n):
    rng = np.random.default_rng(d + rep + n)
    bs, lens = 16, [n, 16 * 20, 16 * 20 + 1, 1000, 333]
    tables, nb = make_tables(rng, lens, bs)
    bounds = random_bounds(rng, nb, 2, d)
    q = bf16(rng.normal(size=(len(lens), 2 * rep, n, d)))
    for top_k, first, last in ((20, 1, 2), (5, 0, 2), (3, 1, 2), (40, 7, 9)):
        check_choice(rng, bounds, q, tables, lens, bs, top_k, first, last)


def test_near_ties_are_decided_as_by_exact_sums():
    # Blocks whose exact scores differ by a few units in 2^-30 of the sum, far below an f32
    # sum's error, in an order unrelated to their place; and among them equal ones.
    rng = np.random.default_rng(8)
    n, d, bs = 400, 128, 16
    base = rng.normal(size=d) * 4
    lo = np.tile(base, (n, 1))
    perm = rng.permutation(n)
    q = rng.normal(size=(1, 1, 1, d)) * 4
    q[..., 0] = 2.0 ** -14
    lo[:, 0] = 0.5 + (perm // 2) * 2.0 ** -8  # pairs of equal blocks; bf16-exact steps
    bounds = bf16(np.stack([lo, lo], 1)[:, None])
    q = bf16(q)
    tables = [[int(x) for x in rng.permutation(n)]]
    for top_k in (3, 50, 51, 200, 399):
        check_choice(rng, bounds, q, tables, [n * bs - 3], bs, top_k, 1, 1)


def test_equal_blocks_and_zero_queries():
    rng = np.random.default_rng(9)
    n, d, bs = 300, 128, 16
    tables = [list(range(n)), list(range(n))]
    same = random_bounds(rng, 1, 2, d).expand(n, 2, 2, d).contiguous()
    q = bf16(rng.normal(size=(2, 8, 1, d)))
    q[1] = 0
    sel = check_choice(rng, same, q, tables, [n * bs, n * bs - 5], bs, 20, 2, 3)
    assert sel.blocks[0, 0].tolist() == list(range(17)) + [n - 3, n - 2, n - 1]
    check_choice(rng, random_bounds(rng, n, 2, d), q, tables, [n * bs, n * bs - 5], bs, 20, 2, 3)


def test_more_blocks_than_shared_memory_holds():
    rng = np.random.default_rng(10)
    n, d, bs = 20011, 64, 16
    bounds = random_bounds(rng, n, 1, d)
    bounds[5000:5040] = bounds[0]
    bounds[19000] = bounds[0]
    q = bf16(rng.normal(size=(1, 2, 1, d)))
    tables = [[int(x) for x in rng.permutation(n)]]
    for top_k in (2, 64, 8300):
        check_choice(rng, bounds, q, tables, [n * bs - 7], bs, top_k, 1, 1)


@pytest.mark.parametrize("n,seqs,hk,width", [(17, 1, 3, 40), (129, 3, 2, 129), (300, 4, 2, 300), (1000, 1, 8, 1000),
                                             (1024, 1, 1, 1024), (1025, 1, 1, 1025), (257, 3, 2, 9000), (129, 100, 2, 129)])
def test_one_kernel_and_two(n, seqs, hk, width):
    # clusters of 1, 2, 4 and 8 CTAs, tables on both sides of 1024 blocks, more clusters than SMs
    rng = np.random.default_rng(n + seqs + hk)
    bs, d = 16, 64
    lens = [max(1, n - 11 * b) * bs - b % bs for b in range(seqs)]
    tables, nb = make_tables(rng, lens, bs)
    tables = [t + [-1] * (width - len(t)) for t in tables]
    bounds = random_bounds(rng, nb, hk, d)
    q = bf16(rng.normal(size=(seqs, hk, 1, d)))
    check_choice(rng, bounds, q, tables, lens, bs, 16, 1, 1)


def test_infinite_and_nan_bounds_and_bad_blocks():
    rng = np.random.default_rng(11)
    n, d, bs, top_k = 200, 128, 16, 30
    bounds = random_bounds(rng, n, 1, d)
    bounds[10] = float("nan")
    bounds[11, 0, 1] = float("inf")
    bounds[12, 0, 0] = float("-inf")
    q = bf16(rng.normal(size=(1, 4, 1, d)))
    tables = [list(range(n))]
    tables[0][20], tables[0][21] = -5, n + 3
    sel = run_choice(rng, bounds, q, tables, [n * bs], bs, top_k, 1, 1, B.PKV_DEVERR_BAD_BLOCK)
    got = sel.blocks[0, 0].tolist()
    assert got == sorted(set(got)) and len(got) == top_k and got[0] == 0 and got[-1] == n - 1
    assert 11 in got and 12 in got and not {10, 20, 21} & set(got)
    # too few good blocks: bad ones fill the places, as -1 for the attention to skip and flag
    tables = [[0] + [-1] * 198 + [5]]
    sel = run_choice(rng, bounds, q, tables, [n * bs], bs, top_k, 1, 1, B.PKV_DEVERR_BAD_BLOCK)
    assert sel.blocks[0, 0].tolist() == list(range(29)) + [199]
    assert sel.tables[0, 0].tolist() == [0] + [-1] * 28 + [5]


def test_bad_lengths():
    rng = np.random.default_rng(12)
    bounds = random_bounds(rng, 40, 2, 128)
    q = bf16(rng.normal(size=(3, 4, 2, 128)))
    tables = [list(range(40))] * 3
    sel = run_choice(rng, bounds, q, tables, [1, 641, -3], 16, 8, 1, 2, B.PKV_DEVERR_BAD_SEQ_LEN)
    assert (sel.lens == 0).all() and (sel.blocks == -1).all() and (sel.tables == -1).all()


# --------------------------------------------------------------------------------------- attention
def run_sparse(rng, fmt, lens, hq, hk, d, dv, n, bs, top_k, first, last, **kw):
    tables, nb = make_tables(rng, lens, bs)
    k, v = Plane(rng, fmt, nb, hk, bs, d), Plane(rng, fmt, nb, hk, bs, dv)
    full = [list(range(nb))]
    bounds = torch.zeros((nb, hk, 2, d), dtype=torch.bfloat16, device=DEV)
    B.update_block_bounds(k.pool, i32(full), i32([nb * bs]), bounds, n_new=nb * bs, k_scales=k.scales,
                          k_biases=k.biases, **k.kw)
    q = bf16(rng.normal(size=(len(lens), hq, n, d)) * 1.5)
    scale = 1 / math.sqrt(d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    blocks = torch.empty((len(lens), hk, top_k), dtype=torch.int32, device=DEV)
    out = B.sparse_decode_attention(q.to(DEV), k.pool, v.pool, bounds, i32(tables), i32(lens), scale, top_k=top_k,
                                    first_blocks=first, last_blocks=last, k_scales=k.scales, k_biases=k.biases,
                                    v_scales=v.scales, v_biases=v.biases, blocks=blocks, error_flag=err, **k.kw, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    chosen = S.choose_blocks(q.double().numpy(), bounds.double().cpu().numpy(), tables, lens, bs, top_k, first, last)
    for b in range(len(lens)):
        for h in range(hk):
            assert blocks[b, h].tolist() == chosen[b][h] + [-1] * (top_k - len(chosen[b][h]))
    ref = S.sparse_attention(q.double().numpy(), k.values, v.values, tables, lens, scale, chosen)
    vmax = np.abs(v.values).max()
    diff = np.abs(out.double().cpu().numpy() - ref)
    worst = np.max(diff - 2.0 ** -8 * np.abs(ref) - (2.0 ** -8 + 2.0 ** -12) * vmax)
    assert worst <= 0, worst
    return q, k, v, bounds, tables, out, blocks


@pytest.mark.parametrize("fmt,d,dv", [(16, 64, 64), (16, 128, 128), (16, 192, 128), (16, 256, 256), (8, 128, 128),
                                      (8, 256, 256), (4, 128, 128), (4, 256, 256), (4, 256, 128), ("e4m3", 64, 64),
                                      ("e4m3", 128, 128), ("e4m3", 256, 256), ("e4m3", 192, 128)])
@pytest.mark.parametrize("n,bs", [(1, 32), (3, 32), (2, 16), (4, 8)])
def test_sparse_attention_matches_the_oracle(fmt, d, dv, n, bs):
    run_sparse(np.random.default_rng(d + dv + n + bs), fmt, [n, 5 * bs, 40 * bs + 1, 777], 8, 2, d, dv, n, bs, 9, 1, 2)


@pytest.mark.parametrize("fmt,lens,hq,hk,n,bs,top_k,first,last,kw", [
    (16, [2000], 8, 2, 1, 16, 64, 0, 1, {}),
    (16, [3000, 2, 1500], 32, 8, 2, 16, 33, 3, 4, {"partition_tokens": 64}),   # states through the workspace
    (4, [1500] * 9, 16, 4, 1, 32, 20, 1, 1, {"schedule": B.PKV_SCHEDULE_BALANCED}),
    ("e4m3", [1500, 40], 64, 1, 1, 32, 1, 0, 1, {}),                           # one block of 64 query heads
    (16, [1023, 1024, 1025], 2, 2, 1, 32, 32, 1, 1, {"contraction": B.PKV_CONTRACTION_CUDA_CORE}),
])
def test_schedules_and_budgets(fmt, lens, hq, hk, n, bs, top_k, first, last, kw):
    run_sparse(np.random.default_rng(sum(lens)), fmt, lens, hq, hk, 128, 128, n, bs, top_k, first, last, **kw)


@pytest.mark.parametrize("fmt", [16, "e4m3"])
def test_a_budget_for_every_block_is_the_dense_decode(fmt):
    q, k, v, bounds, tables, out, _ = run_sparse(np.random.default_rng(3), fmt, [500, 64, 33], 8, 2, 128, 128, 1, 32,
                                                 16, 1, 1, partition_tokens=512)
    dense = B.paged_decode_attention(q.to(DEV), k.pool, v.pool, i32(tables), i32([500, 64, 33]), 1 / math.sqrt(128),
                                     k_scales=k.scales, v_scales=v.scales, partition_tokens=512, **k.kw)
    assert torch.equal(out, dense)


def test_choice_and_attention_apart_are_the_one_call():
    rng = np.random.default_rng(21)
    q, k, v, bounds, tables, out, blocks = run_sparse(rng, 16, [900, 1600], 8, 2, 128, 128, 2, 16, 12, 1, 2)
    sel = B.select_blocks(q.to(DEV), bounds, i32(tables), i32([900, 1600]), block_size=16, top_k=12, last_blocks=2)
    again = B.selected_decode_attention(q.to(DEV), k.pool, v.pool, sel, 1 / math.sqrt(128))
    assert torch.equal(sel.blocks, blocks) and torch.equal(again, out)


def test_bad_block_and_length_in_the_sparse_call():
    rng = np.random.default_rng(22)
    q, k, v, bounds, tables, _, _ = run_sparse(rng, 16, [900, 800], 8, 2, 128, 128, 1, 16, 12, 1, 1)
    t = i32(tables)
    t[0, 0] = -7  # a block that is always taken
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = B.sparse_decode_attention(q.to(DEV), k.pool, v.pool, bounds, t, i32([900, 5000]), 0.1, top_k=12,
                                    error_flag=err)
    assert int(err) == B.PKV_DEVERR_BAD_BLOCK | B.PKV_DEVERR_BAD_SEQ_LEN
    assert (out[1] == 0).all() and torch.isfinite(out.float()).all() and (out[0] != 0).any()


def test_two_streams_and_a_captured_graph():
    rng = np.random.default_rng(23)
    q, k, v, bounds, tables, out, _ = run_sparse(rng, 16, [900, 1600], 8, 2, 128, 128, 1, 16, 12, 1, 1)
    args = (q.to(DEV), k.pool, v.pool, bounds, i32(tables), i32([900, 1600]), 1 / math.sqrt(128))
    plan = B.make_sparse_plan(B.layout_for(k.pool, 128, 16), B.DecodeParams(2, 8, 1, len(tables[0])),
                              B.SparseParams(12, 1, 1))
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        with torch.cuda.stream(st):
            ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
            for _ in range(20):
                o = B.sparse_decode_attention(*args, top_k=12, workspace=ws)
            outs.append(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)
    got = torch.zeros_like(out)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sparse_decode_attention(*args, top_k=12, workspace=ws, out=got)
    ws.fill_(0xFF)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out)


def test_a_run_of_steps_over_e4m3_pages():
    # as a server runs them: a prompt, then tokens, each appended, its bounds kept, and attended sparsely
    rng = np.random.default_rng(31)
    bs, hk, hq, d, steps, prompt = 32, 2, 8, 128, 6, [290, 63]
    lens = [0, 0]
    tables, nb = make_tables(rng, [p + steps for p in prompt], bs)
    kc = np.full((nb, hk, bs, d), 0x7F, np.uint8)  # an unused pool: NaN codes and scales
    vc, ks, vs = kc.copy(), np.full((nb, hk), np.nan, np.float32), np.full((nb, hk), np.nan, np.float32)
    dev = [torch.from_numpy(x).to(DEV) for x in (kc, vc, ks, vs)]
    bounds = torch.full((nb, hk, 2, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    ref_bounds = np.zeros((nb, hk, 2, d))
    fmt = dict(bits=8, group_size=B.PKV_GROUP_BLOCK)
    top_k, dt = 4, i32(tables)
    for step in range(steps + 1):
        # the prompts differ in length: each is appended by a call of its own
        for b in ([0, 1] if step == 0 else [None]):
            which = slice(None) if b is None else slice(b, b + 1)
            n = 1 if b is None else prompt[b]
            new = [bf16(rng.normal(size=(len(lens[which]), hk, n, d)) * (1 + step)) for _ in range(2)]
            at = lens[which]
            B.paged_append(new[0].to(DEV), new[1].to(DEV), dt[which], i32(at), dev[0], dev[1], k_scales=dev[2],
                           v_scales=dev[3], **fmt)
            kc, ks = O.append_blocks(new[0].float().numpy(), tables[which], at, kc, ks)
            vc, vs = O.append_blocks(new[1].float().numpy(), tables[which], at, vc, vs)
            lens[which] = [l + n for l in at]
            B.update_block_bounds(dev[0], dt[which], i32(lens[which]), bounds, n_new=n, k_scales=dev[2], **fmt)
            ref_bounds = S.update_bounds(ref_bounds, O.block_values(kc, ks), tables[which], lens[which], n, True)
        q = bf16(rng.normal(size=(2, hq, 1, d)))
        blocks = torch.empty((2, hk, top_k), dtype=torch.int32, device=DEV)
        out = B.sparse_decode_attention(q.to(DEV), dev[0], dev[1], bounds, dt, i32(lens), 0.1, top_k=top_k,
                                        k_scales=dev[2], v_scales=dev[3], blocks=blocks, **fmt)
        chosen = S.choose_blocks(q.double().numpy(), ref_bounds, tables, lens, bs, top_k, 1, 1)
        assert [[x for x in blocks[b, h].tolist() if x >= 0] for b in range(2) for h in range(hk)] == \
            [c for per in chosen for c in per]
        K, V = O.block_values(kc, ks), O.block_values(vc, vs)
        ref = S.sparse_attention(q.double().numpy(), K, V, tables, lens, 0.1, chosen)
        vmax = max(float(np.abs(oracle.gather_pages(V, t, l)).max()) for t, l in zip(tables, lens))
        diff = np.abs(out.double().cpu().numpy() - ref)
        assert (diff <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * vmax).all(), step
    assert np.array_equal(dev[0].cpu().numpy(), kc) and np.array_equal(dev[3].cpu().numpy(), vs, equal_nan=True)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("shape", ["normal", "cancelling", "one large", "growing"])
def test_score_errors_are_far_within_the_bound_the_choice_uses(d, shape):
    # E = D 2^-25 |q|_1 max|bound|; for wide tables the f32 scores lie at the start of the
    # choice's workspace, as integers of the same order
    rng = np.random.default_rng(d)
    n, bs, rep, width = 128, 16, 4, 8193
    bounds, q = rng.normal(size=(n, 1, 2, d)), rng.normal(size=(1, rep, 1, d))
    if shape == "cancelling":
        bounds[..., 1::2] = -bounds[..., ::2] * np.sign(q[0, 0, 0, 1::2] * q[0, 0, 0, ::2])
        q[..., 1::2] = np.abs(q[..., ::2]) * np.sign(q[..., 1::2])
    elif shape == "one large":
        bounds[..., 0] *= 300
    elif shape == "growing":
        bounds *= 2.0 ** np.linspace(-6, 6, d)
    bounds = bf16(np.sort(bounds, 2))
    q = bf16(q)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    tables = [list(range(n)) + [-1] * (width - n)]
    B.select_blocks(q.to(DEV), bounds.to(DEV), i32(tables), i32([n * bs]), block_size=bs, top_k=8, workspace=ws)
    keys = ws[:4 * n].cpu().numpy().view(np.uint32)
    got = np.where(keys >> 31, keys ^ np.uint32(0x80000000), ~keys).astype(np.uint32).view(np.float32).astype(np.float64)
    bd, qd = bounds.double().numpy(), q.double().numpy()
    ref = S.block_scores(qd[0, :, 0], bd[:, 0, 0], bd[:, 0, 1])
    e = d * 2.0 ** -25 * np.abs(qd).sum(-1).max() * np.abs(bd).max()
    worst = np.abs(got - ref).max() / e
    assert worst < 0.1, worst


@pytest.mark.parametrize("width", [400, 1500])
def test_products_near_the_smallest_normal_number(width):
    # scores around 2^-118, where the error bound of an f32 score would leave the normal range
    rng = np.random.default_rng(41)
    n, bs, d = 400, 16, 128
    bounds = bf16(random_bounds(rng, n, 2, d).double().numpy() * 2.0 ** -61)
    q = bf16(rng.normal(size=(1, 8, 1, d)) * 2.0 ** -60)
    bounds[100:110] = bounds[50]  # equal scores among them
    tables = [[int(x) for x in rng.permutation(n)] + [-1] * (width - n)]
    for top_k in (3, 40, 399):
        check_choice(rng, bounds, q, tables, [n * bs - 3], bs, top_k, 1, 1)


@pytest.mark.parametrize("fmt", [16, "e4m3"])
def test_nearly_as_many_units_as_a_call_takes(fmt):
    # 8191 sequences of 8 KV heads; all blocks chosen is the dense decode, two are the ends
    g = torch.Generator(device=DEV).manual_seed(5)
    seqs, hk, hq, d, bs = 8191, 8, 8, 64, 32
    lens = torch.randint(1, 3 * bs + 1, (seqs,), generator=g, device=DEV, dtype=torch.int32)
    tables = torch.randperm(3 * seqs, generator=g, device=DEV, dtype=torch.int32).view(seqs, 3)
    rows = torch.randn((2, 3 * seqs, hk, bs, d), generator=g, device=DEV, dtype=torch.bfloat16)
    q = torch.randn((seqs, hq, 1, d), generator=g, device=DEV, dtype=torch.bfloat16)
    kw, sc = {}, {}
    if fmt == "e4m3":
        rows = rows.to(torch.float8_e4m3fn)
        kw = dict(bits=8, group_size=B.PKV_GROUP_BLOCK)
        sc = dict(k_scales=torch.ones((3 * seqs, hk), device=DEV), v_scales=torch.ones((3 * seqs, hk), device=DEV))
    k, v = rows[0], rows[1]
    bounds = torch.empty((3 * seqs, hk, 2, d), dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.update_block_bounds(k, tables, lens, bounds, n_new=3 * bs, k_scales=sc.get("k_scales"), error_flag=err, **kw)
    blocks = torch.empty((seqs, hk, 2), dtype=torch.int32, device=DEV)
    dense = B.paged_decode_attention(q, k, v, tables, lens, 0.125, error_flag=err, **sc, **kw)
    every = B.sparse_decode_attention(q, k, v, bounds, tables, lens, 0.125, top_k=3, error_flag=err, **sc, **kw)
    ends = B.sparse_decode_attention(q, k, v, bounds, tables, lens, 0.125, top_k=2, blocks=blocks, error_flag=err, **sc, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    # the same sums in another order, then a rounding to bf16 on each side
    vmax = float(v.float().abs().max())
    assert ((every.float() - dense.float()).abs() <= 2.0 ** -7 * dense.float().abs() + 2.0 ** -7 * vmax).all()
    n = (lens + bs - 1) // bs
    last = torch.where(n > 1, n - 1, -1)
    assert (blocks[:, :, 0] == 0).all() and (blocks[:, :, 1] == last[:, None]).all()
    assert ((ends.float() - every.float())[n <= 2].abs() <= 2.0 ** -7 * every.float()[n <= 2].abs() + 2.0 ** -7 * vmax).all()


def test_two_threads_on_the_default_stream_and_on_one_side_stream():
    # each thread holds its own workspace of the default stream; other streams' are each call's own
    rng = np.random.default_rng(43)
    cases = [run_sparse(rng, fmt, lens, 8, 2, 128, 128, 1, 16, 12, 1, 1)
             for fmt, lens in ((16, [9000, 1600]), ("e4m3", [700, 5000, 64]))]
    lengths = ([9000, 1600], [700, 5000, 64])
    side = torch.cuda.Stream()
    wrong, gate = [], threading.Barrier(2)

    def work(case, lens):
        q, k, v, bounds, tables, want, _ = case
        qd, dt, dl = q.to(DEV), i32(tables), i32(lens)
        torch.cuda.synchronize()
        for stream in (torch.cuda.default_stream(), side):
            with torch.cuda.stream(stream):
                gate.wait()
                got = [B.sparse_decode_attention(qd, k.pool, v.pool, bounds, dt, dl, 1 / math.sqrt(128), top_k=12,
                                                 k_scales=k.scales, v_scales=v.scales, **k.kw) for _ in range(40)]
                stream.synchronize()
                wrong.extend(1 for o in got if not torch.equal(o, want))

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, lengths)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_scores_read_again_from_memory_and_marks_in_two_segments():
    # more blocks than the choice keeps scores of in shared memory (24576) and marks at once (32768)
    rng = np.random.default_rng(47)
    n, d, bs = 33001, 64, 16
    bounds = random_bounds(rng, n, 1, d)
    bounds[5000:5040] = bounds[0]
    bounds[32990] = bounds[0]
    q = bf16(rng.normal(size=(1, 2, 1, d)))
    tables = [[int(x) for x in rng.permutation(n)]]
    for top_k in (2, 300, 25000):
        check_choice(rng, bounds, q, tables, [n * bs - 7], bs, top_k, 1, 1)
    same = bounds[:1].expand(n, 1, 2, d).contiguous()  # ties everywhere: every block is ambiguous
    check_choice(rng, same, q, tables, [n * bs - 7], bs, 40, 1, 2)


@pytest.mark.parametrize("n", [400, 1800, 9000])
def test_more_ambiguous_blocks_than_are_ranked_in_shared_memory(n):
    # 300 blocks within an f32 sum's error of one another, in no order, and equal ones among them
    rng = np.random.default_rng(n)
    d, bs = 128, 16
    base = rng.normal(size=d) * 4
    lo = rng.normal(size=(n, d)) * 0.1
    near = rng.permutation(np.arange(1, n - 1))[:300]
    lo[near] = base
    lo[near, 0] = 0.5 + (np.arange(300) // 3) * 2.0 ** -8
    q = np.tile(base, (1, 2, 1, 1))
    q[..., 0] = 2.0 ** -14
    bounds, q = bf16(np.stack([lo, lo], 1)[:, None]), bf16(q)
    tables = [[int(x) for x in rng.permutation(n)]]
    for top_k in (20, 152, 301):
        check_choice(rng, bounds, q, tables, [n * bs - 3], bs, top_k, 1, 1)


@pytest.mark.parametrize("fmt", [16, "e4m3"])
def test_bounds_after_a_sequence_gave_up_rows(fmt):
    # four proposed tokens, three given up, two others appended in their place: the bounds still hold every key
    rng = np.random.default_rng(53)
    hk, bs, d = 2, 32, 128
    tables = i32([[2, 0, 1]])
    kw = {} if fmt == 16 else dict(bits=8, group_size=B.PKV_GROUP_BLOCK)
    pools = [torch.zeros((3, hk, bs, d), dtype=torch.bfloat16 if fmt == 16 else torch.uint8, device=DEV) for _ in range(2)]
    sc = {} if fmt == 16 else {s: torch.zeros((3, hk), device=DEV) for s in ("k_scales", "v_scales")}
    bounds = torch.full((3, hk, 2, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    for at, n, size in ((0, 40, 1.0), (40, 4, 9.0), (41, 2, 1.0), (43, 30, 1.0)):
        new = [bf16(rng.normal(size=(1, hk, n, d)) * size).to(DEV) for _ in range(2)]
        B.paged_append(*new, tables, i32([at]), *pools, **sc, **kw)
        B.update_block_bounds(pools[0], tables, i32([at + n]), bounds, n_new=n, k_scales=sc.get("k_scales"), **kw)
        keys = pools[0].double() if fmt == 16 else torch.from_numpy(
            O.block_values(pools[0].cpu().numpy(), sc["k_scales"].cpu().numpy())).to(DEV)
        rows = keys[tables[0].long()].transpose(0, 1).reshape(hk, 3 * bs, d)[:, :at + n]
        for j in range(-(-(at + n) // bs)):
            lo, hi = bounds[int(tables[0, j])].double().unbind(1)
            held = rows[:, j * bs:(j + 1) * bs]
            assert (lo <= held.amin(1)).all() and (hi >= held.amax(1)).all()
            if fmt == "e4m3":  # read whole: no looser than the rounding
                assert (lo >= held.amin(1) - held.amin(1).abs() * 2.0 ** -7).all()
                assert (hi <= held.amax(1) + held.amax(1).abs() * 2.0 ** -7).all()
