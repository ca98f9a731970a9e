"""Plain 64-bit forms of the operators around the paged cache's attention, and bounds of what
the kernels' roundings may differ from them by (CPU tensors throughout)."""
from __future__ import annotations

import torch

BF, FP = torch.bfloat16, torch.float16
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -11}            # half a step, relative
TINY = {BF: 2.0 ** -133, FP: 2.0 ** -25}          # half a step of subnormal numbers


def norm(x, residual, weight, offset, eps):
    """(y, t) in 64 bits."""
    t = x.double() + (0 if residual is None else residual.double())
    g = offset + (torch.ones(t.shape[-1], dtype=torch.float64) if weight is None else weight.double())
    return t * g / torch.sqrt((t * t).mean(-1, keepdim=True) + eps), t


# fp32 roundings in y: t, t g, g itself, a sum of d squares in at most 8 * 4 steps a thread and 10
# across threads (half of its relative error), 1 / d, the root's 2 ulp, the product: below 64 * 2^-24
NORM_SLACK = 2.0 ** -18


def norm_slack(y, dtype):
    return (HALF[dtype] + NORM_SLACK) * y.abs() + TINY[dtype]


def exponent(most):
    """Least e in [-117, 120] with most <= 448 2^e (64-bit magnitudes)."""
    m, k = torch.frexp(most.double())
    return torch.where(most > 0, k - 9 + (m > 0.875).to(k.dtype), -117).clamp(-117, 120)


def from_rows8(codes, exps):
    v = codes.view(torch.float8_e4m3fn).double()
    v = torch.ldexp(v, exps.to(torch.int64)[..., None] - 127)
    return torch.where((exps == 255)[..., None], float("nan"), v)


def rows8_slack(y, exps, slack):
    """Half a step of e4m3 at the row's exponent, and `slack` of y itself."""
    step = torch.ldexp(torch.ones((), dtype=torch.float64), exps.to(torch.int64)[..., None] - 127)
    return torch.maximum(y.abs() * 2.0 ** -4, 2.0 ** -10 * step) + slack


def project(x, w, n, index=None, x16=None, down=None, up=None, scale=None):
    """x [batch n][K], w [O][K] (64-bit values): y in 64 bits."""
    y = x.double() @ w.double().t()
    if index is None:
        return y
    for b, a in enumerate(index.tolist()):
        if 0 <= a < down.shape[0]:
            r = slice(b * n, (b + 1) * n)
            u = x16[r].double() @ down[a].double().t() * (1.0 if scale is None else float(scale[a]))
            y[r] += u @ up[a].double().t()
    return y


def project_slack(x, w, n, y, dtype, index=None, x16=None, down=None, up=None, scale=None):
    """The result's rounding, K additions' of fp32 (each at most 2^-24 of the sum of magnitudes: a bound
    for any order, and for the tensor cores' fewer and coarser ones), and for an adapter the rounding
    of x A^T to 16 bits and its own sums."""
    u24 = 2.0 ** -24
    K = x.shape[1]
    over = K * u24 * (x.double().abs() @ w.double().abs().t())
    if index is not None:
        for b, a in enumerate(index.tolist()):
            if 0 <= a < down.shape[0]:
                r, s = slice(b * n, (b + 1) * n), 1.0 if scale is None else float(scale[a])
                d, v, z = down[a].double(), up[a].double(), x16[r].double()
                u = z @ d.t() * s
                off = HALF[dtype] * u.abs() + (K + 2) * u24 * abs(s) * (z.abs() @ d.abs().t()) + TINY[dtype]
                over[r] += off @ v.abs().t() + (K + down.shape[1]) * u24 * (u.abs() @ v.abs().t())
    return HALF[dtype] * (y.abs() + over) + over + TINY[dtype]


class Pool:
    """Pages as lists: what dt_cache_reserve does, request after request."""

    def __init__(self, pages, batch, width, page, order=None):
        self.page, self.width = page, width
        self.free = list(order) if order is not None else list(range(pages - 1, -1, -1))
        self.array = self.free + [-1] * (pages - len(self.free))
        self.table = [[] for _ in range(batch)]

    def reserve(self, lengths):
        """Status of each request: None, "over" or "none"."""
        said = [None] * len(self.table)
        need = [-(-max(n, 0) // self.page) for n in lengths]
        for b, k in enumerate(need):
            if k > self.width:
                need[b], said[b] = len(self.table[b]), "over"
        for b in reversed(range(len(need))):
            while len(self.table[b]) > need[b]:
                self.free.append(self.table[b].pop())
        there, asked = len(self.free), 0
        for b, k in enumerate(need):
            want = k - len(self.table[b])
            asked += max(want, 0)
            if want > 0 and asked > there:
                said[b] = "none"
                continue
            for _ in range(want):
                self.table[b].append(self.free.pop())
        self.array[:len(self.free)] = self.free
        return said

    def tables(self):
        return [row + [-1] * (self.width - len(row)) for row in self.table]
