"""Arguments the binding refuses before a kernel sees them (no GPU needed)."""

import pytest
import torch

from quantized_kv_decode_partial_gb300 import binding as B

NB, HK, BS, D = 6, 2, 32, 128
E4M3 = dict(bits=8, group_size=B.PKV_GROUP_BLOCK)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def scales(*shape):
    return torch.ones(shape, dtype=torch.float32)


def decode(**kw):
    a = dict(q=bf16(3, 4, 1, D), k_pool=codes(NB, HK, BS, D), v_pool=codes(NB, HK, BS, D), block_tables=i32(3, 2),
             seq_lens=i32(3), scale=0.1, k_scales=scales(NB, HK), v_scales=scales(NB, HK), **E4M3)
    return {**a, **kw}


def append(**kw):
    a = dict(k_new=bf16(3, HK, 1, D), v_new=bf16(3, HK, 1, D), block_tables=i32(3, 2), seq_lens=i32(3),
             k_pool=codes(NB, HK, BS, D), v_pool=codes(NB, HK, BS, D), k_scales=scales(NB, HK), v_scales=scales(NB, HK),
             **E4M3)
    return {**a, **kw}


def sparse(**kw):
    return decode(k_bounds=bf16(NB, HK, 2, D), top_k=2, **kw)


def select(**kw):
    a = dict(q=bf16(3, 4, 1, D), k_bounds=bf16(NB, HK, 2, D), block_tables=i32(3, 4), seq_lens=i32(3), block_size=BS,
             top_k=2)
    return {**a, **kw}


def selected(**kw):
    a = decode(selection=B.BlockSelection(i32(3, HK, 2), i32(3, HK, 2), i32(3, HK)))
    del a["block_tables"], a["seq_lens"]
    return {**a, **kw}


def bounds(**kw):
    a = dict(k_pool=bf16(NB, HK, BS, D), block_tables=i32(3, 2), seq_lens=i32(3), k_bounds=bf16(NB, HK, 2, D), n_new=1)
    return {**a, **kw}


@pytest.mark.parametrize("scale,error", [(torch.ones(NB, HK, dtype=torch.float16), TypeError),
                                         (scales(NB, 1), ValueError), (scales(NB * HK), ValueError),
                                         (scales(NB, 2 * HK)[:, ::2], ValueError)])
@pytest.mark.parametrize("call,args", [(B.paged_decode_attention, decode), (B.paged_append, append),
                                       (B.sparse_decode_attention, sparse), (B.selected_decode_attention, selected)])
def test_scales_of_e4m3_pages(call, args, scale, error):
    for name in ("k_scales", "v_scales"):
        with pytest.raises(error, match="e4m3"):
            call(**args(**{name: scale}))


@pytest.mark.parametrize("scale,error", [(torch.ones(NB, HK, dtype=torch.bfloat16), TypeError),
                                         (scales(NB, HK, BS, 2), ValueError), (scales(NB - 1, HK), ValueError)])
@pytest.mark.parametrize("call,more", [(B.HostDecodeStep, {}), (B.paged_decode_passes, dict(passes="partial"))])
def test_scales_of_e4m3_pages_in_prepared_steps_and_single_passes(call, more, scale, error):
    # 16-bit planes, such as affine pages have, would be read as f32 past their end
    for name in ("k_scales", "v_scales"):
        with pytest.raises(error, match="e4m3"):
            call(**decode(**{name: scale}, **more))


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.int32])
@pytest.mark.parametrize("call,args,more", [
    (B.paged_decode_attention, decode, {}), (B.paged_append, append, {}), (B.HostDecodeStep, decode, {}),
    (B.paged_decode_passes, decode, dict(passes="partial")), (B.sparse_decode_attention, sparse, {}),
    (B.selected_decode_attention, selected, {}), (B.update_block_bounds, bounds, dict(k_scales=scales(NB, HK), **E4M3))])
def test_codes_of_another_float8_type(call, args, more, dtype):
    # their bytes would be read as e4m3fn codes
    for name in ("k_pool", "v_pool")[:1 if call is B.update_block_bounds else 2]:
        pool = torch.zeros(NB, HK, BS, D // (4 if dtype is torch.int32 else 1), dtype=dtype)
        with pytest.raises(TypeError, match="e4m3"):
            call(**{**args(**more), name: pool})


V_POOLS = [codes(NB - 1, HK, BS, D), codes(NB, HK, BS // 2, D), codes(NB, 1, BS, D), codes(NB + 1, HK, BS, D)]


@pytest.mark.parametrize("wrong,error", [(dict(v_pool=p), ValueError) for p in V_POOLS] + [
    (dict(q=torch.zeros(3, 4, 1, D)), TypeError), (dict(seq_lens=torch.zeros(3, dtype=torch.int64)), TypeError),
    (dict(block_tables=torch.zeros(3, 2, dtype=torch.int64)), TypeError), (dict(block_tables=i32(2, 2)), ValueError),
    (dict(seq_lens=i32(2)), ValueError)])
@pytest.mark.parametrize("call,more", [(B.paged_decode_attention, {}), (B.HostDecodeStep, {}),
                                       (B.paged_decode_passes, dict(passes="partial"))])
def test_shapes_and_types_of_decode_calls_over_e4m3_pages(call, more, wrong, error):
    with pytest.raises(error, match=next(iter(wrong))):
        call(**decode(**wrong, **more))


@pytest.mark.parametrize("wrong,error", [(dict(v_pool=p), ValueError) for p in V_POOLS] + [
    (dict(k_new=torch.zeros(3, HK, 1, D)), TypeError), (dict(v_new=torch.zeros(3, HK, 1, D)), TypeError),
    (dict(v_new=bf16(3, HK, 1, D // 2)), ValueError), (dict(v_new=bf16(3, HK, 2, D)), ValueError),
    (dict(v_new=bf16(2, HK, 1, D)), ValueError), (dict(k_new=bf16(3, 1, 1, D), v_new=bf16(3, 1, 1, D)), ValueError),
    (dict(seq_lens=torch.zeros(3, dtype=torch.int64)), TypeError), (dict(seq_lens=i32(4)), ValueError),
    (dict(block_tables=torch.zeros(3, 2, dtype=torch.int64)), TypeError), (dict(block_tables=i32(4, 2)), ValueError)])
def test_shapes_and_types_of_appends_into_e4m3_pages(wrong, error):
    with pytest.raises(error, match=next(iter(wrong))):
        B.paged_append(**append(**wrong))


@pytest.mark.parametrize("call,args,name,like", [
    (B.paged_append, append, "k_new", bf16(1, HK, 1, D).expand(3, HK, 1, D)),
    (B.paged_append, append, "v_new", bf16(3, HK, 1, 2 * D)[..., ::2]),
    (B.paged_append, append, "v_pool", codes(1, HK, BS, D).expand(NB, HK, BS, D)),
    (B.paged_append, append, "seq_lens", i32(1).expand(3)),
    (B.paged_decode_passes, decode, "q", bf16(1, 4, 1, D).expand(3, 4, 1, D)),
    (B.paged_decode_passes, decode, "block_tables", i32(3, 4)[:, ::2]),
    (B.HostDecodeStep, decode, "k_pool", codes(NB, HK, BS, 2 * D)[..., ::2])])
def test_strided_tensors_of_calls_over_e4m3_pages(call, args, name, like):
    # an expanded tensor holds fewer values than the kernel would read
    more = dict(passes="partial") if call is B.paged_decode_passes else {}
    with pytest.raises(ValueError, match="contiguous"):
        call(**args(**{name: like}, **more))


@pytest.mark.gpu
@pytest.mark.parametrize("call,args,name", [(B.paged_append, append, n) for n in ("v_new", "seq_lens", "k_scales", "v_pool")] +
                         [(B.paged_decode_attention, decode, n) for n in ("seq_lens", "v_scales", "v_pool", "block_tables")])
def test_e4m3_calls_with_a_tensor_on_the_host_or_strided(call, args, name):
    right = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in args().items()}
    call(**right)  # its shapes are remembered
    with pytest.raises(ValueError, match="one device"):
        call(**{**right, name: right[name].cpu()})
    if name != "seq_lens":
        wide = torch.stack([right[name], right[name]], -1)[..., 0]
        with pytest.raises(ValueError, match="contiguous"):
            call(**{**right, name: wide})
    with pytest.raises((TypeError, ValueError)):
        call(**{**right, "seq_lens": right["seq_lens"].long()})
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("wrong,error", [(dict(out=bf16(3, 4, 1, D // 2)), ValueError), (dict(out=torch.zeros(3, 4, 1, D)), TypeError)])
def test_outputs_of_e4m3_decode_calls(wrong, error):
    right = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in decode().items()}
    with pytest.raises(error, match="out"):
        B.paged_decode_attention(**right, **{k: v.cuda() for k, v in wrong.items()})


def affine(args, bits, **kw):
    words, d = lambda: i32(NB, HK, BS, D * bits // 32), D // 64
    a = args(k_pool=words(), bits=bits, group_size=64, k_scales=bf16(NB, HK, BS, d), k_biases=bf16(NB, HK, BS, d))
    if args is not bounds:
        a.update(v_pool=words(), v_scales=bf16(NB, HK, BS, d), v_biases=bf16(NB, HK, BS, d))
    return {**a, **kw}


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("plane,error", [(torch.zeros(NB, HK, BS, D // 64), TypeError), (bf16(NB, HK, BS, 1), ValueError),
                                         (bf16(NB, HK), ValueError), (bf16(NB - 1, HK, BS, D // 64), ValueError)])
@pytest.mark.parametrize("call,args", [(B.sparse_decode_attention, sparse), (B.selected_decode_attention, selected),
                                       (B.update_block_bounds, bounds)])
def test_planes_of_affine_pages_in_sparse_calls(call, args, plane, error, bits):
    for name in ("k_scales", "k_biases", "v_scales", "v_biases")[:2 if args is bounds else 4]:
        with pytest.raises(error, match=name):
            call(**affine(args, bits, **{name: plane}))


@pytest.mark.gpu
@pytest.mark.parametrize("call,args", [(B.sparse_decode_attention, sparse), (B.selected_decode_attention, selected),
                                       (B.update_block_bounds, bounds)])
def test_sparse_calls_over_affine_pages_with_remembered_shapes(call, args):
    right = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in affine(args, 4).items()}
    if "selection" in right:
        right["selection"] = B.BlockSelection(*(t.cuda() for t in right["selection"]))
    call(**right)
    with pytest.raises(ValueError, match="k_scales"):
        call(**{**right, "k_scales": bf16(NB, HK, BS, 1).cuda()})
    torch.cuda.synchronize()


def test_workspaces_are_held_up_to_a_bound():
    ws, cpu = B._Workspaces(), torch.device("cpu")
    small = ws.get(cpu, 0, 0, 1000)
    assert ws.get(cpu, 0, 0, 10) is small and ws.get(cpu, 0, 7, 10) is not small
    grown = ws.get(cpu, 0, 0, ws.MOST_HELD)
    assert grown.numel() == ws.MOST_HELD and ws.get(cpu, 0, 0, 1000) is grown
    large = ws.get(cpu, 0, 0, ws.MOST_HELD + 1)
    assert large.numel() == ws.MOST_HELD + 1 and ws.held == {0: grown}


@pytest.mark.gpu
def test_a_large_step_gives_its_workspace_back():
    # 64 sequences whose tables could hold 262144 blocks of scores: about 200 MB for this one call
    call = lambda width: B.select_blocks(bf16(64, 4, 1, 64).cuda(), bf16(4, 1, 2, 64).cuda(), i32(64, width).cuda(),
                                         torch.ones(64, dtype=torch.int32, device="cuda"), block_size=32, top_k=4)
    call(8)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    call(1 << 18)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() <= before + B._Workspaces.MOST_HELD


def test_pools_of_another_format():
    # a pool whose rows hold fewer bytes than the format's would be read past its end
    with pytest.raises(ValueError, match="k_pool"):
        B.layout_for(codes(NB, HK, BS, D), D, 16)
    with pytest.raises(ValueError, match="k_pool"):
        B.layout_for(torch.zeros(NB, HK, BS, D // 8, dtype=torch.int32), D, 8)
    assert B.layout_for(torch.zeros(NB, HK, BS, D // 8, dtype=torch.int32), D, 4).head_dim == D


@pytest.mark.gpu
@pytest.mark.parametrize("call,args,wrong,error", [
    (B.sparse_decode_attention, sparse, dict(q=torch.zeros(3, 4, 1, D)), TypeError),
    (B.sparse_decode_attention, sparse, dict(seq_lens=torch.zeros(3, dtype=torch.int64)), TypeError),
    (B.sparse_decode_attention, sparse, dict(seq_lens=i32(2)), ValueError),
    (B.sparse_decode_attention, sparse, dict(k_bounds=bf16(NB, HK, D, 2)), ValueError),
    (B.sparse_decode_attention, sparse, dict(v_pool=codes(NB - 1, HK, BS, D)), ValueError),
    (B.sparse_decode_attention, sparse, dict(blocks=i32(3, HK, 3)), ValueError),
    (B.sparse_decode_attention, sparse, dict(out=bf16(3, 4, 1, D // 2)), ValueError),
    (B.sparse_decode_attention, sparse, dict(out=torch.zeros(3, 4, 1, D)), TypeError),
    (B.sparse_decode_attention, sparse, dict(q=bf16(3, D, 1, 4).transpose(1, 3)), ValueError),
    (B.select_blocks, select, dict(k_bounds=torch.zeros(NB, HK, 2, D)), TypeError),
    (B.select_blocks, select, dict(block_tables=i32(2, 4)), ValueError),
    (B.select_blocks, select, dict(out=B.BlockSelection(i32(3, HK, 2), i32(3, HK, 1), i32(3, HK))), ValueError),
    (B.selected_decode_attention, selected, dict(selection=B.BlockSelection(i32(3, HK, 2), i32(3, 1, 2), i32(3, HK))),
     ValueError),
    (B.selected_decode_attention, selected, dict(v_pool=codes(NB, HK, BS // 2, D)), ValueError),
    (B.update_block_bounds, bounds, dict(k_bounds=torch.zeros(NB, HK, 2, D)), TypeError),
    (B.update_block_bounds, bounds, dict(k_bounds=bf16(NB, HK, 2, 2 * D)), ValueError),
    (B.update_block_bounds, bounds, dict(seq_lens=i32(4)), ValueError),
])
def test_types_and_shapes(call, args, wrong, error):
    def on_gpu(x):
        if isinstance(x, tuple):
            return B.BlockSelection(*map(on_gpu, x))
        return x.cuda() if isinstance(x, torch.Tensor) else x

    right = {k: on_gpu(v) for k, v in args().items()}
    for _ in range(2):  # the second time with the right call's shapes remembered
        with pytest.raises(error):
            call(**{**right, **{k: on_gpu(v) for k, v in wrong.items()}})
        call(**right)
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("call,args,name", [(B.sparse_decode_attention, sparse, "seq_lens"),
                                            (B.sparse_decode_attention, sparse, "k_bounds"),
                                            (B.select_blocks, select, "block_tables"),
                                            (B.selected_decode_attention, selected, "v_pool"),
                                            (B.update_block_bounds, bounds, "seq_lens")])
def test_tensors_on_the_host(call, args, name):
    right = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in args().items()}
    if "selection" in right:
        right["selection"] = B.BlockSelection(*(t.cuda() for t in right["selection"]))
    with pytest.raises(ValueError, match="one device"):
        call(**{**right, name: right[name].cpu()})
