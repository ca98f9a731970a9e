"""Plain 64-bit implementations of the paged-cache operators (torch on the host) and
the inputs of their tests."""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float16: torch.finfo(torch.float16).eps / 2}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}    # half the least step


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, trained=4096.0, beta_fast=32.0,
                beta_slow=1.0):
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "parts":
        g = [min(1.0, max(0.0, (trained * x / math.tau - beta_slow) / (beta_fast - beta_slow))) for x in f]
        f = [x * (y + (1 - y) / factor) for x, y in zip(f, g)]
    return torch.tensor(f, dtype=torch.float64), 1 + 0.1 * math.log(factor) if scaling == "parts" else 1.0


def turn(x, positions, f, mag, interleaved, gradient=False):
    """[batch][heads][n][dh] float64 turned at positions [batch][n]."""
    rot = 2 * f.numel()
    angle = positions.double()[:, None, :, None] * f
    c, s = mag * angle.cos(), mag * angle.sin() * (-1 if gradient else 1)
    y = x.double().clone()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = x[..., ia].double(), x[..., ib].double()
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def turn_slack(x, rot, mag, interleaved):
    """The fp32 part of the rotation's error: cos and sin are off by at most 3e-7
    (argument rounded to 24 bits of half a turn, 2 ulp of the function, magnitude),
    three roundings of 2^-24: below 1e-6 (|x_a| + |x_b|) mag."""
    y = torch.zeros_like(x, dtype=torch.float64)
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    both = x[..., ia].double().abs() + x[..., ib].double().abs()
    y[..., ia] = y[..., ib] = 1e-6 * mag * both
    return y


def exponent(amax):
    """Least e in [-117, 120] with amax <= 448 2^e, for finite amax (float64 tensor)."""
    m, k = torch.frexp(amax)
    return torch.where(amax > 0, k - 9 + (m > 0.875).to(k.dtype), -200).clamp(-117, 120)


def quantise(x):
    """Rows of exact values -> (codes uint8, exponent bytes uint8)."""
    x = x.double()
    amax = x.abs().amax(-1)
    fine = torch.isfinite(amax)
    e = exponent(torch.where(fine, amax, 1.0))
    top = torch.where(e == 120, 240.0, 448.0)[..., None].double()
    q = torch.minimum(torch.maximum(torch.ldexp(x, -e[..., None].double()), -top), top)
    code = q.float().to(torch.float8_e4m3fn).view(torch.uint8)   # exact in fp32: 11 bits, scaled by 2^-e
    return torch.where(fine[..., None], code, 0x7f).to(torch.uint8), torch.where(fine, e + 127, 255).to(torch.uint8)


def dequantise(code, exp):
    v = code.view(torch.float8_e4m3fn).double() * torch.pow(2.0, exp.double() - 127)[..., None]
    return torch.where((exp == 255)[..., None], math.nan, v)


def pool_rows(cache, which, b, index):
    """Rows `index` (list) of request b: [Hkv][rows][dh] float64 on the host."""
    page = cache.k.shape[2]
    t = cache.table[b].cpu().long()
    idx = torch.as_tensor(index, dtype=torch.long)
    pages, slots = t[idx // page], idx % page
    x = getattr(cache, which).cpu()
    if x.dtype in HALF:
        return x[pages, :, slots].double().transpose(0, 1)
    e = getattr(cache, which + "_exp").cpu()
    return dequantise(x.view(torch.uint8)[pages, :, slots], e[pages, :, slots]).transpose(0, 1)


def make_cache(dt, kind, dtype, batch, rows, Hkv, page, dh, seed, spare=2, fill=True):
    """A cache on the GPU with shuffled pages; rows of N(0, 1) values (scaled a row), or
    NaN bits everywhere."""
    g = torch.Generator().manual_seed(seed)
    per = -(-rows // page)
    pages = batch * per + spare
    table = torch.randperm(pages, generator=g)[:batch * per].to(torch.int32).view(batch, per).contiguous().cuda()
    cdt = torch.float8_e4m3fn if kind == "e4m3" else dtype
    cache = dt.PagedCache.empty(pages, Hkv, page, dh, table, cdt)
    for which in "kv":
        p, e = getattr(cache, which), getattr(cache, which + "_exp")
        if not fill:
            p.view(torch.uint8).fill_(0x7f if kind == "e4m3" else 0xff)
            if e is not None:
                e.fill_(127)
            continue
        x = torch.randn(p.shape, generator=g) * torch.exp2(torch.randint(-2, 3, p.shape[:3], generator=g))[..., None]
        if kind == "e4m3":
            code, ex = quantise(x.to(torch.bfloat16))
            p.view(torch.uint8).copy_(code)
            e.copy_(ex)
        else:
            p.copy_(x.to(dtype))
    return cache


def poison_behind(cache, lengths):
    """NaN in every slot of the pool that is not one of the first lengths[b] rows."""
    page = cache.k.shape[2]
    keep = torch.zeros(cache.k.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lengths):
        for j in range(n):
            keep[int(cache.table[b, j // page]), j % page] = True
    gone = ~keep.cuda()[:, None, :].expand(cache.k.shape[:3])
    for which in "kv":
        p = getattr(cache, which)
        p.view(torch.uint8 if p.element_size() == 1 else torch.int16)[gone] = 0x7f if p.element_size() == 1 else 0x7fff


def attention(cache, q, prefix, mask, counts, scale):
    """(out, slack factor's mean of p |v|, A) in float64: q [batch][H][n][dh] host."""
    batch, H, n, dh = q.shape
    G = H // cache.Hkv
    out = torch.zeros(batch, H, n, dh, dtype=torch.float64)
    mass, big = torch.zeros_like(out), 0.0
    for b in range(batch):
        pre, cnt = int(prefix[b]), int(counts[b]) if counts is not None else n
        L = pre + cnt
        if L == 0:
            continue
        k, v = (pool_rows(cache, w, b, range(L)) for w in "kv")
        see = torch.ones(cnt, L, dtype=torch.bool)
        see[:, pre:] = mask[b, :cnt, :cnt].bool() if mask is not None else torch.ones(cnt, cnt).tril().bool()
        for h in range(H):
            kk, vv = k[h // G], v[h // G]
            for lo in range(0, cnt, 256):
                x = scale * q[b, h, lo:min(cnt, lo + 256)].double() @ kk.T
                s = see[lo:lo + 256]
                big = max(big, abs(scale) * float((q[b, h, lo:lo + 256].double().abs() @ torch.nan_to_num(kk.abs(), posinf=0.).T).max()) if cnt else 0.0)
                x = torch.where(s, x, -math.inf)
                m = x.amax(-1, keepdim=True)
                p = torch.where(s, torch.exp(x - torch.where(torch.isfinite(m), m, 0.0)), 0.0)
                z = p.sum(-1, keepdim=True)
                p = torch.where(z == 0, 0.0, p / z)      # NaN where a score that the row sees is NaN
                fine = torch.isfinite(vv)
                y = p @ torch.where(fine, vv, 0.0)
                if not fine.all():      # only to the rows that see the key
                    for j in (~fine).any(1).nonzero()[:, 0].tolist():
                        odd = torch.where(fine[j], 0.0, vv[j])
                        y[s[:, j]] = y[s[:, j]] + odd
                out[b, h, lo:lo + x.shape[0]] = y
                mass[b, h, lo:lo + x.shape[0]] = p @ torch.where(fine, vv.abs(), 0.0)
    return out, mass, big


def attention_slack(ref, mass, big, dtype, dh, keys):
    """Allowed error: the output's rounding; each weight's rounding to 16 bits; the
    relative error of a weight from its score (dh products accumulated in fp32, the
    exponent's argument rounded) and of the sums over the keys, all times sum p |v|."""
    u = 2.0 ** -23
    weight = 2 * (dh * u * big + 4 * u * (1 + big)) + 2 * keys * u
    return HALF[dtype] * ref.abs() + TINY[dtype] + (HALF[dtype] + weight) * mass
