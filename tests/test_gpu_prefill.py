"""Prompt attention over pages against float64 softmax attention over the same values."""

import math

import pytest
import torch

import quantized_kv_decode_partial_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = dict(bits=8, group_size=pkv.PKV_GROUP_BLOCK)


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


class Cache:
    """Pages of a format with tables in no order; ``values`` are what the pages stand for, in float64."""

    def __init__(self, lens, hk, dk, dv, bs, fmt, seed=0, poison=True):
        self.lens, self.hk, self.bs, self.fmt = lens, hk, bs, fmt
        bits = fmt.get("bits", 16)
        pages = [-(-l // bs) for l in lens]
        nb = sum(pages) + 2
        g = torch.Generator().manual_seed(seed)
        perm = torch.randperm(nb, generator=g).tolist()
        self.tables = torch.full((len(lens), max(1, max(pages)) + 1), -5, dtype=torch.int32)
        for b, n in enumerate(pages):
            for j in range(n):
                self.tables[b, j] = perm.pop()
        self.planes, self.values, self.pools = {}, [], []
        for name, d in (("k", dk), ("v", dv)):
            if bits == 16:
                pool = torch.randn(nb, hk, bs, d, generator=g).to(torch.bfloat16)
                self.values.append(pool.double().to(DEV))
                if poison:  # rows past the lengths and blocks of nobody
                    used = torch.zeros(nb, bs, dtype=torch.bool)
                    for b, l in enumerate(lens):
                        for t in range(l):
                            used[self.tables[b, t // bs], t % bs] = True
                    pool[~used[:, None, :, None].expand_as(pool)] = float("nan")
            elif fmt is E4M3:
                pool = (torch.randn(nb, hk, bs, d, generator=g) * 96).clamp(-448, 448).to(torch.float8_e4m3fn)
                s = torch.rand(nb, hk, generator=g) * 0.02 + 0.002
                if seed % 2 == 0:
                    s = torch.exp2(torch.floor(torch.log2(s)))
                self.planes[name + "_scales"] = s.to(DEV)
                self.values.append((pool.double() * s.double()[..., None, None]).to(DEV))
                used = torch.zeros(nb, bs, dtype=torch.bool)
                for b, l in enumerate(lens):
                    for t in range(l):
                        used[self.tables[b, t // bs], t % bs] = True
                pool.view(torch.uint8)[~used[:, None, :, None].expand_as(pool)] = 0x7F  # not a number
            else:
                codes = torch.randint(0, 2 ** bits, (nb, hk, bs, d), generator=g)
                s = ((torch.rand(nb, hk, bs, d // 64, generator=g) + 0.5) * 4 / 2 ** bits).to(torch.bfloat16)
                z = (torch.randn(nb, hk, bs, d // 64, generator=g) * 0.3 - 2.0).to(torch.bfloat16)
                self.planes[name + "_scales"], self.planes[name + "_biases"] = s.to(DEV), z.to(DEV)
                x = codes.unflatten(-1, (-1, 64)).double() * s.double()[..., None] + z.double()[..., None]
                self.values.append(x.flatten(-2).to(DEV))
                per = 32 // bits
                w = (codes.unflatten(-1, (-1, per)) << (torch.arange(per) * bits)).sum(-1)
                pool = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
            self.pools.append(pool.to(DEV))
        self.tables = self.tables.to(DEV)

    def rows(self, b, which):
        """[HK, len, D] in float64."""
        n = -(-self.lens[b] // self.bs)
        x = self.values[which][self.tables[b, :n].long()]
        return x.transpose(0, 1).flatten(1, 2)[:, :self.lens[b]]


def reference(q, cache, news, scale, window=0, hidden=None):
    """Outputs [T, HQ, Dv] and what an error may reach, in float64. hidden(b) -> mask of keys not seen."""
    T, hq, d = q.shape
    rep, dv = hq // cache.hk, cache.values[1].shape[-1]
    out = torch.zeros(T, hq, dv, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    first = 0
    for b, n in enumerate(news):
        if n == 0:
            continue
        L = cache.lens[b]
        k, v = cache.rows(b, 0), cache.rows(b, 1)
        x = q[first:first + n].double().view(n, cache.hk, rep, d).permute(1, 2, 0, 3)
        s = x @ k[:, None].transpose(-1, -2) * scale
        size = (x.abs() @ k[:, None].abs().transpose(-1, -2) * abs(scale)).amax().item()
        at = L - n + torch.arange(n, device=DEV)[:, None]
        t = torch.arange(L, device=DEV)[None]
        seen = t <= at
        if window:
            seen = seen & (t > at - window)
        if hidden is not None:
            seen = seen & ~hidden(b)[None, :L]
        p = torch.exp(s - s.masked_fill(~seen, -math.inf).amax(-1, keepdim=True).clamp(min=-1e300)).masked_fill(~seen, 0.0)
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
        o, a = p @ v[:, None], p @ v[:, None].abs()
        # weights: rounded to bf16 (2^-8); scores: d products of 16 at a time into f32, each step off by
        # 17 * 2^-24 of the sum of magnitudes; the exponential and its argument 2^-20; sums over L keys in f32
        rel = 2.0 ** -8 + 2 * (1.1 * d * 2.0 ** -24 * size + 2.0 ** -20) + L * 2.0 ** -24
        if cache.fmt.get("bits", 16) != 16:  # keys and values rounded to bf16 (affine: fp16) on their way in, unless they fit
            rel = rel + 2.0 ** -8 + 2 * 2.0 ** -8 * size
        out[first:first + n] = o.permute(2, 0, 1, 3).reshape(n, hq, dv)
        tol[first:first + n] = (2.0 ** -8 * o.abs() + rel * a).permute(2, 0, 1, 3).reshape(n, hq, dv)
        first += n
    return out, tol


def run(q, cache, news, scale, tables=None, lens=None, starts=None, **kw):
    if starts is None:
        starts = [0]
        for n in news:
            starts.append(starts[-1] + n)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    out = pkv.paged_prefill_attention(q, *cache.pools, cache.tables if tables is None else tables,
                                      i32(cache.lens if lens is None else lens), i32(starts), scale, error_flag=err,
                                      **cache.planes, **cache.fmt, **kw)
    return out, int(err)


def check(q, cache, news, scale, **kw):
    got, err = run(q, cache, news, scale, **kw)
    ref, tol = reference(q, cache, news, scale, kw.get("window", 0))
    assert err == 0
    n = sum(news)
    diff = (got.double() - ref).abs()[:n]
    assert bool((diff <= tol[:n]).all()), f"beyond by {(diff - tol[:n]).max().item():.3e}, max diff {diff.max().item():.3e}"
    return got


DIMS = [(64, 64), (128, 128), (256, 256), (192, 128), (256, 128), (128, 256)]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("splits", [1, 3])
def test_one_prompt(dk, dv, splits):
    cache = Cache([150], 2, dk, dv, 32, dict())
    check(randn(150, 8, dk, seed=1), cache, [150], 1 / math.sqrt(dk), splits=splits)


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("splits", [0, 1, 2, 7])
def test_ragged_chunks(dk, dv, splits):
    lens, news = [1, 700, 33, 129, 1000, 64], [1, 200, 0, 129, 3, 64]
    cache = Cache(lens, 2, dk, dv, 16, dict(), seed=1)
    check(randn(sum(news), 6, dk, seed=2), cache, news, 1 / math.sqrt(dk), splits=splits)


@pytest.mark.parametrize("bs", [8, 16, 32, 48, 64, 96, 128, 256])
def test_block_sizes(bs):
    lens, news = [517, 130], [300, 130]
    for dk, dv in ((128, 128), (256, 256)):
        check(randn(sum(news), 4, dk, seed=3), Cache(lens, 2, dk, dv, bs, dict(), seed=bs), news, 0.09, splits=1)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (2, 1), (3, 1), (10, 2), (7, 1), (8, 1), (33, 1), (64, 1), (128, 2)])
def test_head_groups(hq, hk):
    lens, news = [300, 77], [140, 77]
    check(randn(sum(news), hq, 128, seed=4), Cache(lens, hk, 128, 128, 32, dict()), news, 0.09)


@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 128, 500, 10 ** 6])
@pytest.mark.parametrize("dk,dv,splits", [(128, 128, 1), (128, 128, 3), (256, 256, 1), (64, 64, 0)])
def test_windows(window, dk, dv, splits):
    lens, news = [900, 260, 5], [300, 260, 5]
    check(randn(sum(news), 4, dk, seed=5), Cache(lens, 2, dk, dv, 32, dict()), news, 0.09, window=window, splits=splits)


@pytest.mark.parametrize("fmt", [dict(), E4M3, dict(bits=8)])
def test_blocks_below_the_window_may_be_gone(fmt):
    """Their table entries are none, or those of blocks whose scales are not numbers."""
    lens, news, window = [900, 300], [20, 140], 100
    cache = Cache(lens, 2, 128, 128, 32, fmt)
    q = randn(160, 4, 128, seed=17)
    ref, tol = reference(q, cache, news, 0.09, window)
    spare = (set(range(cache.pools[0].shape[0])) - set(cache.tables.flatten().tolist())).pop()
    for t in cache.planes.values():
        t[spare] = math.nan
    tables = cache.tables.clone()
    tables[0, :(900 - 20 - window + 1) // 32 - 1] = -1
    tables[0, (900 - 20 - window + 1) // 32 - 1] = spare
    tables[1, :(300 - 140 - window + 1) // 32] = spare
    got, err = run(q, cache, news, 0.09, tables=tables, window=window)
    assert err == 0 and bool(((got.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("scale", [0.0, -0.09, 1.0, 3.0, 1e-8])
def test_scales(scale):
    lens, news = [300, 200], [300, 7]
    check(randn(sum(news), 4, 128, seed=6), Cache(lens, 2, 128, 128, 32, dict()), news, scale)


AFFINE = [(128, 128), (256, 256), (256, 128), (128, 256)]
CODES = [(E4M3, d) for d in DIMS] + [(dict(bits=b), d) for b in (4, 8) for d in AFFINE]


def allowed(fmt, reading):
    """Affine pages have one way of being read."""
    return reading if fmt is E4M3 else 0


@pytest.mark.parametrize("fmt,dims", CODES)
@pytest.mark.parametrize("splits,reading", [(0, 0), (1, 1), (3, 1), (1, 2), (3, 2)])
def test_pages_of_codes(fmt, dims, splits, reading):
    lens, news = [1, 700, 33, 129, 1000, 64, 130], [1, 200, 0, 129, 3, 64, 2]
    cache = Cache(lens, 2, *dims, 32, fmt, seed=splits)
    check(randn(sum(news), 6, dims[0], seed=2), cache, news, 1 / math.sqrt(dims[0]), splits=splits, reading=allowed(fmt, reading))


@pytest.mark.parametrize("fmt", [E4M3, dict(bits=8), dict(bits=4)])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 96, 128, 256])
@pytest.mark.parametrize("reading", [1, 2])
def test_block_sizes_of_codes(fmt, bs, reading):
    lens, news = [517, 130], [300, 130]
    for dims in ((128, 128), (256, 256)):
        check(randn(sum(news), 4, dims[0], seed=3), Cache(lens, 2, *dims, bs, fmt, seed=bs + 1), news, 0.09, splits=1,
              reading=allowed(fmt, reading))


@pytest.mark.parametrize("fmt", [E4M3, dict(bits=8), dict(bits=4)])
@pytest.mark.parametrize("window", [1, 100, 500])
@pytest.mark.parametrize("reading", [1, 2])
def test_windows_of_codes(fmt, window, reading):
    lens, news = [900, 260, 5, 2000, 129], [300, 260, 5, 0, 129]
    for dims in ((128, 128), (256, 256)):
        check(randn(sum(news), 4, dims[0], seed=5), Cache(lens, 2, *dims, 32, fmt), news, 0.09, window=window, reading=allowed(fmt, reading))
    # tables so wide that the values lie by tokens
    cache = Cache(lens, 2, 128, 128, 32, fmt)
    cache.tables = torch.nn.functional.pad(cache.tables, (0, 400), value=-1)
    check(randn(sum(news), 4, 128, seed=5), cache, news, 0.09, window=window, reading=allowed(fmt, reading))


@pytest.mark.parametrize("fmt", [E4M3, dict(bits=8), dict(bits=4)])
@pytest.mark.parametrize("dims", [(128, 128), (256, 256)])
@pytest.mark.parametrize("reading", [1, 2])
def test_bad_blocks_of_codes_are_skipped(fmt, dims, reading):
    lens, news = [300, 200], [150, 200]
    cache = Cache(lens, 2, *dims, 32, fmt)
    q = randn(350, 4, dims[0], seed=10)
    tables = cache.tables.clone()
    tables[0, 3], tables[1, 0], tables[1, 5] = -1, 10 ** 6, cache.pools[0].shape[0]
    got, err = run(q, cache, news, 0.09, tables=tables, reading=allowed(fmt, reading))
    assert err == 1
    gone = {0: [3], 1: [0, 5]}
    ref, tol = reference(q, cache, news, 0.09, hidden=lambda b: torch.tensor([t // 32 in gone[b] for t in range(512)], device=DEV))
    assert bool(((got.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("reading", [1, 2])
def test_block_scales_of_zero_and_far_apart(reading):
    cache = Cache([300], 2, 128, 128, 32, E4M3)
    for name, scale, row in (("k_scales", 0.0, 2), ("v_scales", 0.0, 3), ("v_scales", 2.0 ** 30, 4), ("v_scales", 2.0 ** -40, 5),
                             ("k_scales", 2.0 ** -40, 6)):
        at = cache.tables[0, row].long()
        which = 0 if name[0] == "k" else 1
        cache.values[which][at] *= scale / cache.planes[name][at].double()[:, None, None]
        cache.planes[name][at] = scale
    check(randn(300, 4, 128, seed=14), cache, [300], 0.09, reading=reading)


@pytest.mark.parametrize("fmt", [dict(), E4M3, dict(bits=8), dict(bits=4)])
@pytest.mark.parametrize("D", [128, 256])
def test_error_beside_the_outputs_own_rounding(fmt, D):
    """Root mean square over the output: bf16 weights cost as much as the output's rounding to bf16 does (independent, so
    sqrt(2) of it, with a tenth for the sample); affine pages, whose values have more bits, get fp16 and next to nothing."""
    lens, news = [2000, 700], [300, 200]
    cache = Cache(lens, 2, D, D, 32, fmt, seed=2)
    q = randn(500, 8, D, seed=15)
    got, _ = run(q, cache, news, 1 / math.sqrt(D))
    ref, _ = reference(q, cache, news, 1 / math.sqrt(D))
    own = (ref.to(torch.bfloat16).double() - ref).norm()
    assert (got.double() - ref).norm() <= (1.1 if fmt.get("bits") in (4, 8) and fmt is not E4M3 else 1.1 * math.sqrt(2)) * own


@pytest.mark.parametrize("key,value,query", [(1e-6, 1e-6, 1.0), (1e5, 1e5, 1e-5), (1e-20, 1e20, 1e20), (1.0, 0.0, 1.0),
                                             (0.0, 1.0, 1.0), (1.0, 1.0, 0.0)])
def test_affine_pages_of_any_size(key, value, query):
    """Values far beyond and below fp16's range, per sequence and head: powers of two bring them in."""
    lens, news = [300, 50], [120, 50]
    cache = Cache(lens, 2, 128, 128, 32, dict(bits=8))
    for name, by in (("k", key), ("v", value)):
        for plane in ("_scales", "_biases"):
            t = cache.planes[name + plane]
            ratio = (t.float() * by).to(torch.bfloat16)
            blocks = cache.tables[0, :10].long()  # the first sequence's alone
            t[blocks] = ratio[blocks]
        which = 0 if name == "k" else 1
        pool = cache.pools[which].view(torch.uint8).double().unflatten(-1, (-1, 64))
        s, z = cache.planes[name + "_scales"].double(), cache.planes[name + "_biases"].double()
        cache.values[which] = (pool * s[..., None] + z[..., None]).flatten(-2)
    q = (randn(170, 4, 128, seed=16).float() * query).to(torch.bfloat16)
    check(q, cache, news, 0.09)


def test_rising_maxima_are_followed():
    # keys that grow along the sequence: every tile raises the maximum by far more than the slack
    cache = Cache([1000], 1, 128, 128, 32, dict(), poison=False)
    ramp = (torch.arange(1024, device=DEV) / 40).view(-1, 1, 32, 1)
    order = cache.tables[0, :32].long()
    base = torch.ones(32, 1, 32, 128, device=DEV) * ramp
    cache.pools[0][order] = base.to(torch.bfloat16)
    cache.values[0][order] = cache.pools[0][order].double()
    q = (torch.ones(500, 2, 128, device=DEV) * 0.5).to(torch.bfloat16)
    check(q, cache, [500], 0.09)
    check(-q, cache, [500], 0.09)


def test_strided_queries_and_given_outputs():
    lens, news = [100, 90], [60, 90]
    cache = Cache(lens, 2, 128, 128, 32, dict())
    qkv = randn(150, (8 + 4) * 128, seed=7)
    q = qkv.view(150, 12, 128)[:, :8]
    want = check(q.contiguous(), cache, news, 0.09)
    out = torch.full((150, 8, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    got, _ = run(q, cache, news, 0.09, out=out)
    assert got is out and torch.equal(got, want)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(run(heads_first, cache, news, 0.09)[0], want)


@pytest.mark.parametrize("splits", [1, 4])
def test_tokens_of_no_sequence_stay_as_they_were(splits):
    lens, news = [200, 150], [100, 50]
    cache = Cache(lens, 2, 128, 128, 32, dict())
    q = randn(170, 4, 128, seed=8)
    out = torch.full((170, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    run(q, cache, news, 0.09, starts=[10, 110, 160], out=out, splits=splits)
    assert (out[:10] == 5.0).all() and (out[160:] == 5.0).all()
    ref, tol = reference(q[10:160], cache, news, 0.09)
    assert bool(((out[10:160].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("splits", [1, 3])
def test_bad_lengths_write_zeros(splits):
    lens, news = [200, 150, 90], [100, 50, 90]
    cache = Cache(lens, 2, 128, 128, 32, dict())
    q = randn(240, 4, 128, seed=9)
    for bad in (49, -1, 10 ** 6, 2 ** 31 - 1):
        got, err = run(q, cache, news, 0.09, lens=[200, bad, 90], splits=splits)
        assert err == 2 and not got[100:150].any()
        ref, tol = reference(q, cache, news, 0.09)
        diff = (got.double() - ref).abs()
        assert bool((diff <= tol)[:100].all()) and bool((diff <= tol)[150:].all())


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("dk,dv", [(128, 128), (256, 256)])
def test_bad_blocks_are_skipped(splits, dk, dv):
    lens, news = [300, 200], [150, 200]
    cache = Cache(lens, 2, dk, dv, 32, dict())
    q = randn(350, 4, dk, seed=10)
    tables = cache.tables.clone()
    tables[0, 3], tables[1, 0], tables[1, 5] = -1, 10 ** 6, cache.pools[0].shape[0]
    got, err = run(q, cache, news, 0.09, tables=tables, splits=splits)
    assert err == 1
    gone = {0: [3], 1: [0, 5]}
    hidden = lambda b: torch.tensor([t // 32 in gone[b] for t in range(512)], device=DEV)
    ref, tol = reference(q, cache, news, 0.09, hidden=hidden)
    assert bool(((got.double() - ref).abs() <= tol).all())
    assert not got[150:182].any()  # their only block is none


@pytest.mark.parametrize("reading", [1, 2])
def test_bad_lengths_and_starts_over_codes(reading):
    lens, news = [200, 150, 90], [100, 50, 90]
    cache = Cache(lens, 2, 128, 128, 32, E4M3)
    q = randn(240, 4, 128, seed=9)
    ref, tol = reference(q, cache, news, 0.09)
    for bad in (49, -1, 10 ** 6, 2 ** 31 - 1):
        got, err = run(q, cache, news, 0.09, lens=[200, bad, 90], reading=reading, window=1000)
        assert err == 2 and not got[100:150].any()
        diff = (got.double() - ref).abs()
        assert bool((diff <= tol)[:100].all()) and bool((diff <= tol)[150:].all())
    for starts in ([0, 160, 140, 240], [0, 50, 100, 241], [-3, 50, 100, 240], [0, 2 ** 31 - 1, 100, 240], [240, 50, 0, 0]):
        out = torch.full((242, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV)
        _, err = run(q, cache, news, 0.09, starts=starts, out=out[1:241], reading=reading)
        assert err & 2 and (out[0] == 5.0).all() and (out[241] == 5.0).all()


def test_starts_that_fall_or_leave_the_tokens_touch_nothing_else():
    q = randn(100, 4, 128, seed=11)
    for starts in ([0, 60, 40], [0, 50, 101], [-3, 50, 100], [0, 2 ** 31 - 1, 100], [100, 50, 0], [0, 100, 50, 100]):
        cache = Cache([200, 150, 90][:len(starts) - 1], 2, 128, 128, 32, dict())
        for splits in (1, 2):
            out = torch.full((102, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV)
            _, err = run(q, cache, [0, 0], 0.09, starts=starts, out=out[1:101], splits=splits)
            assert err & 2 and (out[0] == 5.0).all() and (out[101] == 5.0).all()


def test_no_tokens():
    cache = Cache([40], 2, 128, 128, 32, dict())
    got, err = run(randn(0, 4, 128), cache, [0], 0.09)
    assert got.shape == (0, 4, 128) and err == 0
    out = torch.full((5, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    run(randn(5, 4, 128), cache, [0], 0.09, starts=[2, 2], out=out)
    assert (out == 5.0).all()


def test_one_token_agrees_with_decode():
    lens = [1, 500, 77, 1300]
    cache = Cache(lens, 2, 128, 128, 32, dict())
    q = randn(4, 8, 128, seed=12)
    got = check(q, cache, [1] * 4, 0.09)
    want = pkv.paged_decode_attention(q[:, :, None].contiguous(), *cache.pools, cache.tables,
                                      torch.tensor(lens, dtype=torch.int32, device=DEV), 0.09)
    assert (got.double() - want[:, :, 0].double()).abs().max() < 2e-2


def test_repeats_give_the_same_bits_and_graphs_replay():
    lens, news = [700, 333], [400, 333]
    cache = Cache(lens, 2, 128, 128, 32, dict())
    q = randn(sum(news), 8, 128, seed=13)
    for splits in (1, 3):
        want, _ = run(q, cache, news, 0.09, splits=splits)
        assert torch.equal(run(q, cache, news, 0.09, splits=splits)[0], want)
        out, err = torch.empty_like(want), torch.zeros(1, dtype=torch.int32, device=DEV)
        starts = torch.tensor([0, 400, 733], dtype=torch.int32, device=DEV)
        sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_prefill_attention(q, *cache.pools, cache.tables, sl, starts, 0.09, splits=splits, out=out, error_flag=err)
        out.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    cache = Cache([100], 2, 128, 128, 32, dict())
    q = randn(50, 4, 128)
    starts, lens = torch.tensor([0, 50], dtype=torch.int32, device=DEV), torch.tensor([100], dtype=torch.int32, device=DEV)
    good = dict(q=q, k_pool=cache.pools[0], v_pool=cache.pools[1], block_tables=cache.tables, seq_lens=lens,
                query_starts=starts, scale=0.09)
    pkv.paged_prefill_attention(**good)
    for bad in (dict(q=q.float()), dict(q=q[None]), dict(q=q[..., :64]), dict(q=q[:, :3]), dict(seq_lens=lens.long()),
                dict(query_starts=starts[:1]), dict(query_starts=starts.cpu()), dict(k_pool=cache.pools[0].float()),
                dict(v_pool=cache.pools[1][:2]), dict(block_tables=cache.tables.long()), dict(window=-1), dict(splits=-1),
                dict(splits=65), dict(scale=math.nan), dict(scale=math.inf), dict(out=q[:49]), dict(out=q.float()),
                dict(q=q[:, :1].expand(50, 4, 128)), dict(splits=2, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
                dict(bits=8), dict(reading=3), dict(q=q.transpose(1, 2)), dict(q=randn(50, 130 * 2, 128))):
        with pytest.raises((TypeError, ValueError, pkv.PkvError)):
            pkv.paged_prefill_attention(**{**good, **bad})
