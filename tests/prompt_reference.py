"""Attention of packed new tokens over pages of every format in float64, and what the kernels' roundings may add, on any
device: for tests over pages whose values 16 bits hold exactly or nearly so."""

import math

import torch

import quantized_kv_decode_partial_gb300 as pkv

E4M3 = dict(bits=8, group_size=pkv.PKV_GROUP_BLOCK)


def affine(fmt):
    return fmt.get("bits", 16) != 16 and "group_size" not in fmt


class Pages:
    """Pages with tables in no order. ``values`` are the rows that attention sees, in float64: of e4m3 pages with any scales the
    products that bf16 rounds, of the others exactly what the pages say."""

    def __init__(self, lens, hk, dims, bs, fmt, seed=0, any_scale=False, device="cpu"):
        self.lens, self.hk, self.bs, self.fmt, self.device = lens, hk, bs, fmt, device
        bits = fmt.get("bits", 16)
        per = [-(-n // bs) for n in lens]
        nb = sum(per) + 2
        g = torch.Generator().manual_seed(seed)
        perm = torch.randperm(nb, generator=g).tolist()
        self.tables = torch.full((len(lens), max(1, max(per)) + 1), -5, dtype=torch.int32)
        for b, n in enumerate(per):
            for j in range(n):
                self.tables[b, j] = perm.pop()
        self.planes, self.values, self.pools = {}, [], []
        for name, d in zip("kv", dims):
            if bits == 16:
                pool = torch.randn(nb, hk, bs, d, generator=g).to(torch.bfloat16)
                x = pool.double()
            elif not affine(fmt):
                pool = (torch.randn(nb, hk, bs, d, generator=g) * 96).clamp(-448, 448).to(torch.float8_e4m3fn)
                s = torch.rand(nb, hk, generator=g) * 0.02 + 0.002
                if not any_scale:
                    s = torch.exp2(torch.floor(torch.log2(s)))
                self.planes[name + "_scales"] = s
                x = (pool.float() * s[..., None, None]).to(torch.bfloat16).double()
            else:
                codes = torch.randint(0, 2 ** bits, (nb, hk, bs, d), generator=g)
                s = ((torch.rand(nb, hk, bs, d // 64, generator=g) + 0.5) * 4 / 2 ** bits).to(torch.bfloat16)
                z = (torch.randn(nb, hk, bs, d // 64, generator=g) * 0.3 - 2.0).to(torch.bfloat16)
                self.planes[name + "_scales"], self.planes[name + "_biases"] = s, z
                x = (codes.unflatten(-1, (-1, 64)).double() * s.double()[..., None] + z.double()[..., None]).flatten(-2)
                n = 32 // bits
                w = (codes.unflatten(-1, (-1, n)) << (torch.arange(n) * bits)).sum(-1)
                pool = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
            self.pools.append(pool.to(device))
            self.values.append(x.to(device))
        self.planes = {n: t.to(device) for n, t in self.planes.items()}
        self.tables = self.tables.to(device)

    def rows(self, b, which):
        """[HK, len, D]"""
        n = -(-self.lens[b] // self.bs)
        x = self.values[which][self.tables[b, :n].long()]
        return x.transpose(0, 1).flatten(1, 2)[:, :self.lens[b]]


def attention(q, pages, news, scale, window=0, hidden=None, rounded=None, late=0):
    """Outputs [T, HQ, Dv] and each one's tolerance, in float64. hidden(b): mask of keys that nobody sees. rounded(x): what is
    done to the weights (relative to a row's largest) before they meet the values, for a model of the kernel; late: places by which
    its mask is off."""
    T, hq, d = q.shape
    rep, dv, dev = hq // pages.hk, pages.values[1].shape[-1], pages.device
    out = torch.zeros(T, hq, dv, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    first = 0
    for b, n in enumerate(news):
        if n == 0:
            continue
        L = pages.lens[b]
        k, v = pages.rows(b, 0)[:, None], pages.rows(b, 1)[:, None]
        x = q[first:first + n].double().view(n, pages.hk, rep, d).permute(1, 2, 0, 3)
        s = x @ k.transpose(-1, -2) * scale
        at, t = L - n + late + torch.arange(n, device=dev)[:, None], torch.arange(L, device=dev)[None]
        seen = (t <= at) & (t > at - window) if window else t <= at
        if hidden is not None:
            seen = seen & ~hidden(b)[None, :L]
        size = (x.abs() @ k.abs().transpose(-1, -2) * abs(scale)).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
        p = torch.exp(s - s.masked_fill(~seen, -math.inf).amax(-1, keepdim=True).clamp(min=-1e300)).masked_fill(~seen, 0.0)
        total = p.sum(-1, keepdim=True).clamp(min=1e-300)
        o, a = (p if rounded is None else rounded(p)) @ v / total, p @ v.abs() / total
        # Of the sum of weighted magnitudes: weights rounded to bf16 or fp16; scores in f32 (d products, 16 at a time, each step
        # off by 17 * 2^-24 of the magnitudes added up), twice, as numerator and sum; the exponential 2^-20; sums over L keys.
        # Affine keys and values are rounded to fp16, and fp16 weights below 2^-21 of the largest are off by 2^-32 of it.
        rel = (2.0 ** -11 if affine(pages.fmt) else 2.0 ** -8) + 2 * (1.1 * d * 2.0 ** -24 * size + 2.0 ** -20) + L * 2.0 ** -24
        if affine(pages.fmt):
            rel = rel + 2.0 ** -11 + 2 * 2.0 ** -11 * size
            a = a + 2.0 ** -21 * seen.double() @ v.abs() / total
        out[first:first + n] = o.permute(2, 0, 1, 3).reshape(n, hq, dv)
        tol[first:first + n] = (2.0 ** -8 * o.abs() + rel * a).permute(2, 0, 1, 3).reshape(n, hq, dv)
        first += n
    return out, tol


def complaint(got, ref, tol, fmt):
    """What is wrong with outputs, or None. Beside each one's tolerance the root mean square of all: weights rounded to bf16 cost
    as much as the rounding of the outputs does (independent of it and, for values about zero, as large: the square root of two
    together), fp16 next to nothing; a tenth more for the sample, and for the scores' f32 sums."""
    err = (got.double() - ref).abs()
    if not bool((err <= tol).all()):
        return f"{int((err > tol).sum())} of {err.numel()} beyond tolerance, by {(err - tol).max().item():.3e} at most"
    own = (ref.to(torch.bfloat16).double() - ref).norm().item()
    most = (1.1 if affine(fmt) else 1.1 * math.sqrt(2)) * own + 1e-12 * ref.norm().item()
    if not err.norm().item() <= most:
        return f"root mean square {err.norm().item() / own:.3f} of the outputs' own rounding"
    return None
