"""GPU parity of e4m3 pages (one f32 scale per block and KV head): append against the
bit-exact write oracle, decode attention against the float64 oracle.

Attention tolerance. Codes and queries enter the products exactly (an e4m3 value is an fp16
value; queries are prescaled by powers of two), sums are f32. What is rounded: each weight to
fp16 (2^-11 relative, or 2^-25 of the row's largest weight), so the weighted mean is off by at
most 2^-11 max|V| for the relative part; the f32 scores and exponentials add under 2^-16 of
max|V| for scores below 2^6; and the output's rounding to bf16, 2^-8 of the value. The bound
is 2^-8 |ref| + 2^-10 max|V|.
"""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import block_scaled as O
from quantized_kv_decode_partial_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FMT = dict(bits=8, group_size=B.PKV_GROUP_BLOCK)


def make_pool(rng, nb, hk, bs, d, tables, lens, spread=2):
    """Codes and scales of one plane; rows at or past each length and blocks of no sequence hold NaN."""
    codes = O.e4m3_codes(np.clip(rng.normal(size=(nb, hk, bs, d)) * 96, -448, 448))
    scales = 2.0 ** rng.integers(-8, -8 + spread, size=(nb, hk))
    scales = (scales * rng.uniform(0.5, 1.0, size=(nb, hk))).astype(np.float32)  # any scale may be read
    used = set()
    for t, n in zip(tables, lens):
        pages = -(-n // bs)
        used |= set(t[:pages])
        if n % bs:
            codes[t[pages - 1], :, n % bs:] = 0x7F
    for i in set(range(nb)) - used:
        codes[i], scales[i] = 0xFF, np.nan
    return codes, scales


def make_tables(rng, lens, bs, extra=3):
    pages = [-(-n // bs) for n in lens]
    perm = rng.permutation(sum(pages) + extra)
    width, at, rows = max(max(pages), 1), 0, []
    for p in pages:
        rows.append([int(x) for x in perm[at:at + p]] + [-1] * (width - p))
        at += p
    return rows, len(perm)


def e4m3(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).to(DEV).view(torch.float8_e4m3fn)


def run_attend(rng, lens, hq, hk, d, dv, n, bs, *, window=0, partition=0, schedule=0, spread=2, edit=None):
    tables, nb = make_tables(rng, lens, bs)
    kc, ks = make_pool(rng, nb, hk, bs, d, tables, lens, spread)
    vc, vs = make_pool(rng, nb, hk, bs, dv, tables, lens, spread)
    if edit:
        edit(kc, ks, vc, vs, tables)
    q = torch.from_numpy(rng.normal(size=(len(lens), hq, n, d)).astype(np.float32)).to(torch.bfloat16)
    scale = 1 / math.sqrt(d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = B.paged_decode_attention(q.to(DEV), e4m3(kc), e4m3(vc), torch.tensor(tables, dtype=torch.int32, device=DEV),
                                   torch.tensor(lens, dtype=torch.int32, device=DEV), scale,
                                   k_scales=torch.from_numpy(ks).to(DEV), v_scales=torch.from_numpy(vs).to(DEV),
                                   window=window, partition_tokens=partition, schedule=schedule, error_flag=err, **FMT)
    torch.cuda.synchronize()
    assert int(err) == 0
    V = O.block_values(vc, vs)
    ref = oracle.paged_decode_attention(q.double().numpy(), O.block_values(kc, ks), V, tables, lens, scale, n,
                                        window=window)
    vmax = 0.0
    for t, l in zip(tables, lens):
        rows = oracle.gather_pages(V, t, l)
        vmax = max(vmax, float(np.abs(rows).max()))
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - ref) - 2.0 ** -8 * np.abs(ref) - 2.0 ** -10 * vmax)
    assert worst <= 0, f"beyond the bound by {worst:.3e} (max|V| {vmax:.3e})"


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (256, 256), (192, 128), (256, 128), (128, 256)])
@pytest.mark.parametrize("rep,n", [(1, 1), (4, 2), (5, 3), (8, 4), (16, 4)])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_head_dims_rows_and_block_sizes(d, dv, rep, n, bs):
    rng = np.random.default_rng(d + dv + 7 * rep + n + bs)
    run_attend(rng, [n, 333, 70], 2 * rep, 2, d, dv, n, bs)


@pytest.mark.parametrize("lens,hq,hk,d,n,bs,kw", [
    ([8192], 16, 4, 256, 1, 32, {}),                                   # one CTA per SM, clusters
    ([1], 4, 4, 128, 1, 32, {}),                                       # one row
    ([31, 32, 33, 64, 65], 4, 1, 64, 1, 32, {}),                       # around a block's end
    ([4000, 17, 2500], 8, 2, 128, 2, 64, {"partition": 96}),           # workspace and merge
    ([2000] * 24, 16, 4, 128, 1, 32, {"partition": 128}),              # several waves
    ([1500, 3, 900], 8, 4, 128, 1, 32, {"schedule": B.PKV_SCHEDULE_BALANCED}),
    ([1500, 4, 901], 32, 4, 256, 3, 32, {"schedule": B.PKV_SCHEDULE_BALANCED}),
    ([1500, 3, 900], 8, 4, 64, 1, 96, {"schedule": B.PKV_SCHEDULE_BALANCED, "window": 100}),
    ([3000, 40, 41], 8, 2, 128, 4, 32, {"window": 37}),                # windows ending inside blocks
    ([3000, 40, 41], 8, 2, 256, 4, 16, {"window": 1}),
    ([3000, 40, 41], 8, 2, 128, 2, 8, {"window": 300}),
])
def test_schedules_windows_and_lengths(lens, hq, hk, d, n, bs, kw):
    run_attend(np.random.default_rng(sum(lens) + d), lens, hq, hk, d, d, n, bs, **kw)


@pytest.mark.parametrize("bs", [8, 16, 32])
def test_scales_far_apart(bs):
    # value scales over 2^40 from block to block, within one chunk where blocks are small
    run_attend(np.random.default_rng(bs), [200, 129], 4, 2, 128, 128, 1, bs, spread=40)


@pytest.mark.parametrize("rep,d,bs,schedule", [(1, 128, 32, 1), (16, 128, 32, 1), (16, 128, 32, 2), (4, 256, 16, 1),
                                               (12, 64, 8, 1)])
@pytest.mark.parametrize("rising", [True, False])
def test_scores_rising_and_falling_along_the_cache(rep, d, bs, schedule, rising):
    # the running maximum follows a row's scores in steps, whatever their order
    def edit(kc, ks, vc, vs, tables):
        for t in tables:
            held = [b for b in t if b >= 0]
            for i, b in enumerate(held if rising else held[::-1]):
                ks[b] *= 0.02 * 500.0 ** (i / len(held))

    run_attend(np.random.default_rng(rep + d), [2500, 700], 2 * rep, 2, d, d, 1, bs, schedule=schedule, edit=edit)


@pytest.mark.parametrize("bs", [8, 32])
def test_zero_scales(bs):
    def edit(kc, ks, vc, vs, tables):
        ks[tables[0][0]] = 0.0
        vs[tables[0][0]] = 0.0
        for b in tables[1]:
            if b >= 0:
                ks[b], vs[b] = 0.0, 0.0

    run_attend(np.random.default_rng(bs), [100, 60], 4, 2, 128, 128, 1, bs, edit=edit)


def test_long_cache_offsets_past_32_bits():
    # a pool of 4.5 GB per plane: byte offsets of its last blocks exceed 2^32
    bs, hk, d, nb = 32, 8, 128, 140000
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.zeros((nb, hk, bs, d), dtype=torch.uint8, device=DEV)
    v = torch.zeros((nb, hk, bs, d), dtype=torch.uint8, device=DEV)
    ks = torch.full((nb, hk), 2.0 ** -7, device=DEV)
    vs = torch.full((nb, hk), 2.0 ** -7, device=DEV)
    last = list(range(nb - 4, nb))
    lens, n_new = [0], 100
    tables = torch.tensor([last], dtype=torch.int32, device=DEV)
    k_new = torch.randn((1, hk, n_new, d), generator=g, device=DEV).to(torch.bfloat16)
    v_new = torch.randn((1, hk, n_new, d), generator=g, device=DEV).to(torch.bfloat16)
    B.paged_append(k_new, v_new, tables, torch.tensor(lens, dtype=torch.int32, device=DEV), k, v, k_scales=ks,
                   v_scales=vs, **FMT)
    q = torch.randn((1, 32, 1, d), generator=g, device=DEV).to(torch.bfloat16)
    out = B.paged_decode_attention(q, k, v, tables, torch.tensor([n_new], dtype=torch.int32, device=DEV), 0.1,
                                   k_scales=ks, v_scales=vs, **FMT)
    kc, kss = O.append_blocks(k_new.float().cpu().numpy(), [[0, 1, 2, 3]], [0], np.zeros((4, hk, bs, d), np.uint8),
                              np.ones((4, hk), np.float32))
    assert np.array_equal(k[nb - 4:].cpu().numpy(), kc) and np.array_equal(ks[nb - 4:].cpu().numpy(), kss)
    vc, vss = O.append_blocks(v_new.float().cpu().numpy(), [[0, 1, 2, 3]], [0], np.zeros((4, hk, bs, d), np.uint8),
                              np.ones((4, hk), np.float32))
    V = O.block_values(vc, vss)
    ref = oracle.paged_decode_attention(q.double().cpu().numpy(), O.block_values(kc, kss), V, [[0, 1, 2, 3]], [n_new],
                                        0.1, 1)
    diff = np.abs(out.double().cpu().numpy() - ref)
    assert (diff <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * np.abs(V).max()).all()


# ------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (256, 256), (192, 128), (128, 256)])
@pytest.mark.parametrize("lens,n_new,bs", [([0, 5, 31, 32], 1, 32), ([0, 5, 60], 70, 32), ([3, 8, 15], 9, 8),
                                           ([0, 100], 200, 96), ([40, 1], 4, 64), ([7], 33, 16)])
def test_append_matches_the_oracle(d, dv, lens, n_new, bs):
    rng = np.random.default_rng(d + dv + n_new + bs)
    hk = 3
    tables, nb = make_tables(rng, [l + n_new for l in lens], bs)
    kc, ks = make_pool(rng, nb, hk, bs, d, tables, lens)
    vc, vs = make_pool(rng, nb, hk, bs, dv, tables, lens)
    ks = np.where(np.isnan(ks), ks, 2.0 ** np.ceil(np.log2(ks))).astype(np.float32)  # as the append leaves them
    mag = 10.0 ** rng.uniform(-3, 2, size=(len(lens), hk, 1, 1))  # some blocks' scales grow, some do not
    k_new = torch.from_numpy(rng.normal(size=(len(lens), hk, n_new, d)) * mag).to(torch.bfloat16)
    v_new = torch.from_numpy(rng.normal(size=(len(lens), hk, n_new, dv)) * mag).to(torch.bfloat16)
    v_new[0, 0] = 0  # a block of zeros
    dk, dv_, dks, dvs = e4m3(kc), e4m3(vc), torch.from_numpy(ks).to(DEV), torch.from_numpy(vs).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.paged_append(k_new.to(DEV), v_new.to(DEV), torch.tensor(tables, dtype=torch.int32, device=DEV),
                   torch.tensor(lens, dtype=torch.int32, device=DEV), dk, dv_, k_scales=dks, v_scales=dvs,
                   error_flag=err, **FMT)
    assert int(err) == 0
    for got, got_s, new, c, s in ((dk, dks, k_new, kc, ks), (dv_, dvs, v_new, vc, vs)):
        ref, ref_s = O.append_blocks(new.float().numpy(), tables, lens, c, s)
        assert np.array_equal(got_s.cpu().numpy(), ref_s, equal_nan=True)
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), ref)  # rows past the last one are as they were


def test_append_bad_blocks_and_lengths():
    bs, hk, d = 32, 2, 64
    k = torch.full((4, hk, bs, d), 0x11, dtype=torch.uint8, device=DEV)
    v = k.clone()
    ks = torch.full((4, hk), 0.5, device=DEV)
    vs = ks.clone()
    tables = torch.tensor([[0, 9], [1, 2], [3, 3]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([30, 60, -1], dtype=torch.int32, device=DEV)
    new = torch.ones((3, hk, 8, d), dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.paged_append(new, new, tables, lens, k, v, k_scales=ks, v_scales=vs, error_flag=err, **FMT)
    assert int(err) == B.PKV_DEVERR_BAD_BLOCK | B.PKV_DEVERR_BAD_SEQ_LEN
    assert (k[1:] == 0x11).all() and (v[1:] == 0x11).all() and (ks[1:] == 0.5).all()  # 60 + 8 rows exceed 64
    assert (k[0, :, :30] == 0x11).all() and (k[0, :, 30:] != 0x11).all()


def test_append_with_a_scale_of_the_callers():
    # a scale that is no power of two and large enough stays; codes divide by it
    bs, hk, d = 32, 1, 64
    rng = np.random.default_rng(2)
    kc = O.e4m3_codes(np.clip(rng.normal(size=(1, hk, bs, d)) * 96, -448, 448))
    ks = np.full((1, hk), 0.0123, np.float32)
    new = torch.from_numpy(rng.normal(size=(1, hk, 3, d))).to(torch.bfloat16)
    for mul in (1.0, 40.0):
        k, v = e4m3(kc), e4m3(kc)
        s, s2 = torch.from_numpy(ks).to(DEV), torch.from_numpy(ks).to(DEV)
        x = new * mul
        B.paged_append(x.to(DEV), x.to(DEV), torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                       torch.full((1,), 9, dtype=torch.int32, device=DEV), k, v, k_scales=s, v_scales=s2, **FMT)
        ref, ref_s = O.append_blocks(x.float().numpy(), [[0]], [9], kc, ks)
        assert np.array_equal(s.cpu().numpy(), ref_s) and np.array_equal(k.view(torch.uint8).cpu().numpy(), ref)


def test_append_then_attend_on_a_side_stream_and_in_a_graph():
    rng = np.random.default_rng(9)
    bs, hk, d, n = 32, 2, 128, 1
    lens = [63, 10, 200]
    tables, nb = make_tables(rng, [l + 8 for l in lens], bs)
    kc, ks = make_pool(rng, nb, hk, bs, d, tables, lens)
    vc, vs = make_pool(rng, nb, hk, bs, d, tables, lens)
    k, v, dks, dvs = e4m3(kc), e4m3(vc), torch.from_numpy(ks).to(DEV), torch.from_numpy(vs).to(DEV)
    q = torch.from_numpy(rng.normal(size=(3, 8, n, d))).to(torch.bfloat16).to(DEV)
    new = torch.from_numpy(rng.normal(size=(2, 3, hk, n, d))).to(torch.bfloat16).to(DEV)
    dt = torch.tensor(tables, dtype=torch.int32, device=DEV)
    before = torch.tensor(lens, dtype=torch.int32, device=DEV)
    after = before + 1
    out = torch.empty_like(q)
    plan = B.make_plan(B.layout_for(k, d, 8, B.PKV_GROUP_BLOCK, v), B.DecodeParams(3, 8, n, dt.shape[1]))
    ws = torch.empty(max(1, plan.workspace_bytes), dtype=torch.uint8, device=DEV)

    def step():
        B.paged_append(new[0], new[1], dt, before, k, v, k_scales=dks, v_scales=dvs, **FMT)
        B.paged_decode_attention(q, k, v, dt, after, 0.09, k_scales=dks, v_scales=dvs, out=out, workspace=ws, **FMT)
        before.add_(1)
        after.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    x = new.float().cpu().numpy()
    for j in range(6):  # the same rows appended six times
        at = [l + j for l in lens]
        kc, ks = O.append_blocks(x[0], tables, at, kc, ks)
        vc, vs = O.append_blocks(x[1], tables, at, vc, vs)
    assert np.array_equal(k.view(torch.uint8).cpu().numpy(), kc) and np.array_equal(v.view(torch.uint8).cpu().numpy(), vc)
    V = O.block_values(vc, vs)
    ref = oracle.paged_decode_attention(q.double().cpu().numpy(), O.block_values(kc, ks), V, tables,
                                        [l + 6 for l in lens], 0.09, 1)
    vmax = max(float(np.abs(oracle.gather_pages(V, t, l + 6)).max()) for t, l in zip(tables, lens))
    diff = np.abs(out.double().cpu().numpy() - ref)
    assert (diff <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * vmax).all()


def test_bad_blocks_and_lengths_are_flagged_and_zeroed():
    rng = np.random.default_rng(11)
    bs, hk, d = 32, 2, 128
    lens = [100, 64]
    tables, nb = make_tables(rng, lens, bs)
    kc, ks = make_pool(rng, nb, hk, bs, d, tables, lens)
    q = torch.from_numpy(rng.normal(size=(2, 4, 1, d))).to(torch.bfloat16).to(DEV)
    dt = torch.tensor(tables, dtype=torch.int32, device=DEV)
    dt[0, 1] = nb + 5
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    s = torch.from_numpy(ks).to(DEV)
    out = B.paged_decode_attention(q, e4m3(kc), e4m3(kc), dt, torch.tensor([100, 500], dtype=torch.int32, device=DEV),
                                   0.1, k_scales=s, v_scales=s, error_flag=err, **FMT)
    assert int(err) == B.PKV_DEVERR_BAD_BLOCK | B.PKV_DEVERR_BAD_SEQ_LEN
    assert (out[1] == 0).all() and torch.isfinite(out.float()).all() and (out[0] != 0).any()


def test_no_alloc_and_host_step_take_e4m3_pages():
    rng = np.random.default_rng(13)
    bs, hk, d, lens = 32, 2, 128, [150, 999]
    tables, nb = make_tables(rng, lens, bs)
    kc, ks = make_pool(rng, nb, hk, bs, d, tables, lens)
    vc, vs = make_pool(rng, nb, hk, bs, d, tables, lens)
    k, v, dks, dvs = e4m3(kc), e4m3(vc), torch.from_numpy(ks).to(DEV), torch.from_numpy(vs).to(DEV)
    q = torch.from_numpy(rng.normal(size=(2, 8, 1, d))).to(torch.bfloat16)
    t, l = torch.tensor(tables, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
    want = B.paged_decode_attention(q.to(DEV), k, v, t.to(DEV), l.to(DEV), 0.1, k_scales=dks, v_scales=dvs, **FMT)
    step = B.HostDecodeStep(q, t, l, k, v, 0.1, k_scales=dks, v_scales=dvs, **FMT)
    got = step()
    torch.cuda.synchronize()
    assert torch.equal(got, want.cpu())
    lib, out = B.load_library(), torch.empty_like(want)
    lay = B.layout_for(k, d, 8, B.PKV_GROUP_BLOCK, v)
    par = B.DecodeParams(2, 8, 1, t.shape[1])
    dq, dt, dl = q.to(DEV), t.to(DEV), l.to(DEV)
    rc = lib.pkv_paged_decode_attention_no_alloc(
        ctypes.byref(lay), ctypes.byref(par), dq.data_ptr(), k.data_ptr(), v.data_ptr(), dks.data_ptr(), None,
        dvs.data_ptr(), None, dt.data_ptr(), dl.data_ptr(), 0.1, out.data_ptr(), None,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(out, want)
