"""Workloads of the paged-cache operators: rotary positions, cache write and read, attention over
the cache for trees, chains and single tokens, and the commit of an accepted path.

A case names an operator (``op``), its sizes and its types. ``run`` computes one pass, either in
plain 32-bit torch operations or (``own``) through the library's entry points.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
POISON = float("nan")        # what rows that nobody has written hold


def listed():
    return [
        # the next token of a few requests: one call per layer, latency counts
        dict(name="rotary-token", op="rotary", type="bf16", batch=8, n=1, H=32, Hkv=8, dh=128, rot=128,
             interleaved=False, scaling="none", factor=1.0, trained=4096, gradient=False, far=2000),
        # the gradient of a long prompt's queries and keys, a part of each head turned, positions far
        # past the trained length
        dict(name="rotary-prompt-gradient", op="rotary", type="fp16", batch=2, n=4099, H=32, Hkv=8, dh=128,
             rot=64, interleaved=True, scaling="parts", factor=16.0, trained=8192, gradient=True, far=100000),
        # the drafted trees of a serving batch (node budget 64, 8B shape): q and k turned, k and v
        # written into 16-bit pages; trees cut to different sizes
        dict(name="write-trees", op="write", type="bf16", cache="16", batch=32, n=65, H=32, Hkv=8, dh=128,
             page=64, prefix=1024, low=512, rotary=True, cut=True),
        # one new token of each of 128 requests into an 8-bit cache, and the row as the cache holds it
        dict(name="store-tokens-e4m3", op="write", type="bf16", cache="e4m3", batch=128, n=1, H=32, Hkv=8, dh=128,
             page=64, prefix=4096, low=1, rotary=False, cut=False),
        # a long prompt into an 8-bit cache (small pages), and the rows read back
        dict(name="store-prompt-e4m3", op="write", type="fp16", cache="e4m3", batch=3, n=5003, H=32, Hkv=8, dh=128,
             page=16, prefix=100, low=0, rotary=False, cut=False),
        # long 8-bit caches read back whole (moved to another runner, or for a layer that wants 16 bits)
        dict(name="read-long-e4m3", op="read", type="bf16", cache="e4m3", batch=8, n=16385, Hkv=8, dh=128,
             page=64, low=9000),
        # the accepted paths of a serving batch's trees (block of 16)
        dict(name="commit-trees", op="commit", type="bf16", cache="16", batch=32, n=65, depth=16, Hkv=8, dh=128,
             page=64, prefix=1024, low=512),
        # the same at the stress batch, 8-bit, trees of 257 rows, and the path's rows read back
        dict(name="commit-stress-e4m3", op="commit", type="bf16", cache="e4m3", batch=128, n=257, depth=16, Hkv=8,
             dh=128, page=32, prefix=2048, low=1024),
        # one request's small tree behind a short prompt, narrow heads: latency counts
        dict(name="attend-one-tree", op="attend", type="fp16", cache="16", batch=1, n=33, H=16, Hkv=2, dh=64, page=16,
             prefix=333, low=333, mask="tree", blank=False, cut=False),
        # single tokens of a serving batch, each at its own length, 8-bit cache
        dict(name="attend-tokens-e4m3", op="attend", type="bf16", cache="e4m3", batch=32, n=1, H=32, Hkv=8, dh=128,
             page=64, prefix=8192, low=512, mask="tree", blank=False, cut=False),
        # the serving batch's trees, 16-bit cache
        dict(name="attend-trees", op="attend", type="bf16", cache="16", batch=32, n=65, H=32, Hkv=8, dh=128, page=64,
             prefix=1024, low=512, mask="tree", blank=False, cut=True),
        # wide trees (node budget 128) of a few requests with long contexts, 8-bit cache
        dict(name="attend-long-e4m3", op="attend", type="bf16", cache="e4m3", batch=8, n=129, H=32, Hkv=8, dh=128,
             page=128, prefix=32768, low=16384, mask="tree", blank=False, cut=False),
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], its logarithm uniform."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(("rotary", "write", "read", "commit", "attend", "attend", "attend"))
    Hkv = rng.choice((1, 2, 4, 8))
    H = Hkv * rng.choice((1, 2, 4, 5, 8))
    dh = rng.choice((64, 128, 128, 128, 96, 80, 256))
    kind, cache = rng.choice(("bf16", "bf16", "fp16")), rng.choice(("16", "e4m3"))
    page = rng.choice((16, 32, 64, 128))
    if op == "rotary":
        rot = rng.choice((dh, dh, dh // 2, 32))
        scaling = rng.choice(("none", "linear", "base", "parts"))
        batch = _spread(rng, 1, 64)
        n = _spread(rng, 1, max(1, min(8192, 40 * 8198 * 128 // (batch * (H + Hkv) * dh))))
        return dict(op=op, type=kind, batch=batch, n=n, H=H, Hkv=Hkv, dh=dh, rot=rot, interleaved=rng.random() < 0.5,
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice((2.0, 4.5, 16.0, 40.0)),
                    trained=rng.choice((2048, 4096, 8192)), gradient=rng.random() < 0.5, far=_spread(rng, 100, 1000000))
    if op == "write":
        batch = _spread(rng, 1, 128)
        n = _spread(rng, 1, max(1, min(8192, 3 * 5003 * 8 * 128 // (batch * Hkv * dh))))
        prefix = _spread(rng, 1, 4096)
        return dict(op=op, type=kind, cache=cache, batch=batch, n=n, H=H, Hkv=Hkv, dh=dh, page=page, prefix=prefix,
                    low=rng.randrange(prefix + 1), rotary=rng.random() < 0.5, cut=rng.random() < 0.5)
    if op == "read":
        batch = _spread(rng, 1, 32)
        n = _spread(rng, 1, max(1, min(65536, 5 * 16385 * 8 * 128 // (batch * Hkv * dh))))
        return dict(op=op, type=kind, cache=cache, batch=batch, n=n, Hkv=Hkv, dh=dh, page=page,
                    low=rng.randrange(n + 1))
    if op == "commit":
        prefix = _spread(rng, 1, 2048)
        return dict(op=op, type=kind, cache=cache, batch=_spread(rng, 1, 128), n=_spread(rng, 2, 257),
                    depth=rng.choice((2, 8, 16)), Hkv=Hkv, dh=dh, page=page, prefix=prefix,
                    low=rng.randrange(prefix + 1))
    mask = rng.choice(("tree", "tree", "causal"))
    batch = _spread(rng, 1, 64)
    n = rng.choice((1, 1, _spread(rng, 2, 16), _spread(rng, 17, 300), _spread(rng, 17, 300)))
    if mask == "causal":
        n = rng.choice((n, _spread(rng, 300, 1500)))
    n = max(1, min(n, 80000000 // (batch * H * dh)))
    keys = int(min(65536, 8 * 24000 * 8 * 128 / (batch * Hkv * dh), 8 * 32 * 129 * 24000 * 128 / (batch * H * n * dh)))
    keys = _spread(rng, 1, max(1, keys))
    return dict(op=op, type=kind, cache=cache, batch=batch, n=n, H=H, Hkv=Hkv, dh=dh, page=page, prefix=keys,
                low=rng.randrange(keys + 1), mask=mask, blank=mask == "tree" and rng.random() < 0.3,
                cut=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _tree_parents(batch, n, g):
    """Parents of trees grown node by node, the earlier nodes likelier: [batch][n], the root's -1."""
    at = torch.arange(n, device="cuda")
    u = torch.rand(batch, n, generator=g, device="cuda") ** 2
    parent = (u * at).long().clamp(max=n - 1)
    parent = torch.minimum(parent, (at - 1).clamp(min=0))
    parent[:, 0] = -1
    return parent


def _ancestors(parent):
    """[batch][n][n] 1 where the column is the row itself or one of its ancestors."""
    batch, n = parent.shape
    step = torch.zeros(batch, n + 1, n + 1, device="cuda")
    step.scatter_(2, torch.cat([parent.clamp(min=-1) + 1, torch.zeros(batch, 1, dtype=torch.long, device="cuda")], 1)
                  .roll(1, 1)[:, :, None], 1.0)
    step[:, 0, 0] = 1.0
    reach = step + torch.eye(n + 1, device="cuda")
    for _ in range(max(1, math.ceil(math.log2(n + 1)))):
        reach = (reach @ reach).clamp(max=1.0)
    return (reach[:, 1:, 1:] > 0).to(torch.uint8)


def _power(e):
    """2^e in 32 bits, exactly, for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _values_to_cache(x):
    """Rows of values as e4m3 codes (uint8) and one power-of-two scale a row (uint8, biased by 127)."""
    x = x.float()
    most = x.abs().amax(-1)
    m, k = torch.frexp(most)
    e = (k.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)).clamp(-117, 120)
    q = x * _power(-e)[..., None]
    top = torch.where(e >= 120, 240.0, 448.0)[..., None]
    code = torch.minimum(torch.maximum(q, -top), top).to(torch.float8_e4m3fn).view(torch.uint8)
    fine = torch.isfinite(most)
    return torch.where(fine[..., None], code, 0x7f).to(torch.uint8), torch.where(fine, e + 127, 255).to(torch.uint8)


def _pool(case, g, batch, rows, kind):
    """Pages for `rows` rows of each request in a shuffled order, with spare pages, filled with `POISON`."""
    per = -(-rows // case["page"])
    pages = batch * per + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:batch * per].to(torch.int32).view(batch, per)
    shape = (pages, case["Hkv"], case["page"], case["dh"])
    if kind == "e4m3":
        code = lambda: torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda")
        exp = lambda: torch.full(shape[:3], 127, dtype=torch.uint8, device="cuda")
        return dict(k=code(), v=code(), k_exp=exp(), v_exp=exp(), table=table.contiguous())
    full = lambda: torch.full(shape, POISON, dtype=TYPES[case["type"]], device="cuda")
    return dict(k=full(), v=full(), k_exp=None, v_exp=None, table=table.contiguous())


def _slots(table, page, index):
    """Page and slot of each cache row `index` [batch][m]."""
    return table.long().gather(1, index // page), index % page


def _fill(case, g, cache, lengths, rows):
    """Values in the first `lengths` rows of each request, and poison behind them: [batch] lengths, `rows` the most."""
    per = cache["table"].shape[1]
    dh, page, batch = case["dh"], case["page"], lengths.numel()
    valid = torch.arange(per * page, device="cuda")[None] < lengths[:, None]
    valid = valid.view(batch, per, 1, page, 1)
    where = cache["table"].long().view(-1)
    for name in ("k", "v"):
        x = torch.randn(batch, per, case["Hkv"], page, dh, generator=g, device="cuda", dtype=torch.bfloat16)
        if name == "k":       # some channels carry larger keys, as trained models' do
            x = x * (1.0 + 3.0 * (torch.arange(dh, device="cuda") % 37 == 5)).to(torch.bfloat16)
        if case["cache"] == "e4m3":
            code, e = _values_to_cache(x)
            code, e = torch.where(valid, code, 0x7f), torch.where(valid[..., 0], e, 127)
            cache[name][where] = code.view(-1, *code.shape[2:])
            cache[name + "_exp"][where] = e.view(-1, *e.shape[2:])
        else:
            x = torch.where(valid, x.to(TYPES[case["type"]]), POISON)
            cache[name][where] = x.view(-1, *x.shape[2:])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    batch, op = case["batch"], case["op"]
    dt = TYPES[case["type"]]
    whole = lambda low, high: torch.randint(low, high + 1, (batch,), generator=g, device="cuda", dtype=torch.int32)
    s = dict(case=case)
    if op == "rotary" or op == "write":
        # heads as views of one projection's output: [batch][n][(H + 2 Hkv) dh]
        n, H, Hkv, dh = case["n"], case["H"], case["Hkv"], case["dh"]
        x = torch.randn(batch, n, H + 2 * Hkv, dh, generator=g, device="cuda", dtype=dt).transpose(1, 2)
        s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if op == "rotary":
        first = whole(0, case["far"])
        s["positions"] = (first[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)[None]).contiguous()
    elif op == "write":
        s["first"] = whole(case["low"], case["prefix"])
        s["counts"] = torch.maximum(whole(1, n), whole(1, n)) if case["cut"] else None
        depth = torch.randint(0, min(16, n), (batch, n), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = (s["first"][:, None] + depth).contiguous()
        s["cache"] = _pool(case, g, batch, case["prefix"] + n, case["cache"])
    elif op == "read":
        n = case["n"]
        s["counts"] = whole(case["low"], n)
        s["first"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        s["cache"] = _pool(case, g, batch, n, case["cache"])
        _fill(case, g, s["cache"], s["counts"], n)
    elif op == "commit":
        n, depth = case["n"], case["depth"]
        s["first"] = whole(case["low"], case["prefix"])
        s["cache"] = _pool(case, g, batch, case["prefix"] + n, case["cache"])
        _fill(case, g, s["cache"], s["first"] + n, case["prefix"] + n)
        # an accepted path: the root, then rows in rising order
        path = torch.rand(batch, n, generator=g, device="cuda").argsort(1)[:, :min(depth, n)].sort(1).values
        path[:, 0] = 0
        s["path"] = path.to(torch.int32).contiguous()
        s["lengths"] = torch.minimum(whole(1, path.shape[1]), whole(1, path.shape[1]))
    else:
        n, H, dh = case["n"], case["H"], case["dh"]
        s["prefix"] = whole(case["low"], case["prefix"])
        s["counts"] = torch.maximum(whole(1, n), whole(1, n)) if case["cut"] else None
        lengths = s["prefix"] + (n if s["counts"] is None else s["counts"])
        s["cache"] = _pool(case, g, batch, case["prefix"] + n, case["cache"])
        _fill(case, g, s["cache"], lengths, case["prefix"] + n)
        s["q"] = torch.randn(batch, n, H, dh, generator=g, device="cuda", dtype=dt).transpose(1, 2)
        s["mask"] = _ancestors(_tree_parents(batch, n, g)).contiguous() if case["mask"] == "tree" else None
        if case["blank"]:     # rows of the batch that hold no node: they see no tree row, themselves neither
            s["mask"][:, n // 2::8] = 0
    return s


# ------------------------------------------------------------- plain forms

def _frequencies(case, dtype):
    """Angle per position of each pair, and the factor on the turned values."""
    rot, base, factor = case["rot"], 10000.0, case["factor"]
    if case["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2))
    f = torch.tensor(base, dtype=dtype, device="cuda") ** (-torch.arange(0, rot, 2, dtype=dtype, device="cuda") / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":    # pairs that turn often in the trained length keep their speed
        turns = case["trained"] * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _turned(case, x, positions, gradient=False):
    """x [batch][heads][n][dh] in 32 bits, its first `rot` values turned (angles in 64 bits)."""
    rot = case["rot"]
    f, magnitude = _frequencies(case, torch.float64)
    angle = positions.double()[:, None, :, None] * f
    c, s = (magnitude * angle.cos()).to(x.dtype), (magnitude * angle.sin()).to(x.dtype)
    s = -s if gradient else s
    t, rest = x[..., :rot], x[..., rot:]
    a, b = (t[..., 0::2], t[..., 1::2]) if case["interleaved"] else (t[..., :rot // 2], t[..., rot // 2:])
    ya, yb = a * c - b * s, a * s + b * c
    y = torch.stack([ya, yb], -1).flatten(-2) if case["interleaved"] else torch.cat([ya, yb], -1)
    return torch.cat([y, rest], -1)


WRITE_ROTARY = dict(interleaved=False, scaling="none", factor=1.0, trained=4096)


def _dense(cache, name, dtype):
    """All rows of each request in order: [batch][Hkv][rows][dh]."""
    where = cache["table"].long()
    x = cache[name][where]
    if cache[name + "_exp"] is not None:
        e = cache[name + "_exp"][where]
        x = x.view(torch.float8_e4m3fn).to(dtype) * _power(e.int().clamp(1, 254) - 127)[..., None].to(dtype)
        x = torch.where((e == 255)[..., None], POISON, x)
    x = x.to(dtype).transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4])


def _rounded(x, dt):
    return x.clamp(-65504.0, 65504.0).to(dt) if dt == torch.float16 else x.to(dt)


def _plain_read(cache, n, first, counts, dt):
    at = torch.arange(n, device="cuda")[None]
    live = at < counts[:, None]
    index = torch.where(live, first[:, None] + at, 0).long()
    page, slot = _slots(cache["table"], cache["k"].shape[2], index)
    out = []
    for name in ("k", "v"):
        x = cache[name][page, :, slot]
        if cache[name + "_exp"] is not None:
            e = cache[name + "_exp"][page, :, slot]
            x = x.view(torch.float8_e4m3fn).float() * _power(e.int().clamp(1, 254) - 127)[..., None]
            x = torch.where((e == 255)[..., None], POISON, x)
        x = torch.where(live[..., None, None], x.float(), 0.0)
        out.append(_rounded(x, dt).transpose(1, 2).contiguous())
    return out


def _plain_write(s):
    case, cache = s["case"], s["cache"]
    n, dt = case["n"], TYPES[case["type"]]
    counts = s["counts"] if s["counts"] is not None else torch.full_like(s["first"], n)
    k, v, q = s["k"].float(), s["v"].float(), None
    if case["rotary"]:
        turn = dict(WRITE_ROTARY, rot=case["dh"])
        k, q = _turned(turn, k, s["positions"]), _turned(turn, s["q"].float(), s["positions"]).to(dt)
    at = torch.arange(n, device="cuda")[None]
    b, i = (at < counts[:, None]).nonzero(as_tuple=True)
    index = (s["first"][b] + i).long()
    page, slot = cache["table"].long()[b, index // case["page"]], index % case["page"]
    for name, x in (("k", k), ("v", v)):
        x = x.transpose(1, 2)[b, i]
        if case["cache"] == "e4m3":
            cache[name][page, :, slot], cache[name + "_exp"][page, :, slot] = _values_to_cache(x)
        else:
            cache[name][page, :, slot] = x.to(dt)
    if case["cache"] == "e4m3":
        return dict(q=q, rows=_plain_read(cache, n, s["first"], counts, dt))
    return dict(q=q, k=cache["k"], v=cache["v"])


def _plain_commit(s):
    case, cache = s["case"], s["cache"]
    at = torch.arange(s["path"].shape[1], device="cuda")[None]
    b, j = (at < s["lengths"][:, None]).nonzero(as_tuple=True)
    old, new = (s["first"][b] + s["path"][b, j]).long(), (s["first"][b] + j).long()
    page = lambda index: (cache["table"].long()[b, index // case["page"]], slice(None), index % case["page"])
    for name in ("k", "v", "k_exp", "v_exp"):
        if cache[name] is not None:
            cache[name][page(new)] = cache[name][page(old)]
    if case["cache"] == "e4m3":
        return _plain_read(cache, s["path"].shape[1], s["first"], s["lengths"], TYPES[case["type"]])
    return cache["k"], cache["v"]


def _attend(s, dtype):
    case, q = s["case"], s["q"]
    batch, H, n, dh = q.shape
    Hkv = case["Hkv"]
    k, v = _dense(s["cache"], "k", dtype), _dense(s["cache"], "v", dtype)
    rows = k.shape[2]
    t = torch.arange(rows, device="cuda")[None] - s["prefix"][:, None]          # tree row of each key
    counts = s["counts"] if s["counts"] is not None else torch.full_like(s["prefix"], n)
    live = torch.arange(n, device="cuda")[None] < counts[:, None]
    if s["mask"] is not None:
        tree = s["mask"].bool().gather(2, t.clamp(0, n - 1)[:, None].expand(batch, n, rows))
    else:
        tree = t[:, None] <= torch.arange(n, device="cuda")[None, :, None]
    inside = live.gather(1, t.clamp(0, n - 1)) & (t < n)
    see = live[:, :, None] & ((t < 0)[:, None] | (tree & inside[:, None]))
    v = torch.where(((t < 0) | inside)[:, None, :, None], v, 0)
    k = torch.where(((t < 0) | inside)[:, None, :, None], k, 0)
    x = q.to(dtype).reshape(batch, Hkv, H // Hkv * n, dh) @ k.transpose(2, 3)
    x = (x * dh ** -0.5).view(batch, H, n, rows).masked_fill_(~see[:, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    z = x.sum(-1, keepdim=True)
    y = (x.view(batch, Hkv, H // Hkv * n, rows) @ v).view(batch, H, n, dh)
    return torch.where(z > 0, y / z, 0)


# ------------------------------------------------------- the library's calls

def _rotary_plan(s, case):
    import conditional_draft_tree_gb300 as dt
    if "rotary" not in s:        # the tables that a model keeps
        s["rotary"] = dt.Rotary(case["rot"], interleaved=case["interleaved"], base=10000.0, scaling=case["scaling"],
                                factor=case["factor"], trained=case["trained"], beta_fast=32.0, beta_slow=1.0)
    return s["rotary"]


def _own(s):
    import conditional_draft_tree_gb300 as dt
    case = s["case"]
    op = case["op"]
    if op == "rotary":
        return dt.rotary(_rotary_plan(s, case), s["positions"], s["q"], s["k"], gradient=case["gradient"])
    if "paged" not in s:         # the cache that a server keeps
        s["paged"] = dt.PagedCache(**s["cache"])
    cache, kind = s["paged"], TYPES[case["type"]]
    if op == "write":
        plan = _rotary_plan(s, dict(WRITE_ROTARY, rot=case["dh"])) if case["rotary"] else None
        q = dt.cache_write(cache, s["k"], s["v"], s["first"], s["counts"], rotary=plan,
                           positions=s["positions"] if plan else None, q=s["q"] if plan else None)
        if case["cache"] == "e4m3":
            return dict(q=q, rows=dt.cache_read(cache, case["n"], s["first"], s["counts"], dtype=kind))
        return dict(q=q, k=s["cache"]["k"], v=s["cache"]["v"])
    if op == "read":
        return dt.cache_read(cache, case["n"], s["first"], s["counts"], dtype=kind)
    if op == "commit":
        dt.cache_commit(cache, s["first"], s["path"], s["lengths"], case["n"])
        if case["cache"] == "e4m3":
            return dt.cache_read(cache, s["path"].shape[1], s["first"], s["lengths"], dtype=kind)
        return s["cache"]["k"], s["cache"]["v"]
    if "workspace" not in s:
        s["workspace"] = dt.cache_attention_workspace(cache, case["H"], case["n"])
    return dt.cache_attention(cache, s["q"], s["prefix"], mask=s["mask"], counts=s["counts"],
                              workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    dt = TYPES[case["type"]]
    if case["op"] == "rotary":
        return tuple(_turned(case, state[name].float(), state["positions"], case["gradient"]).to(dt) for name in "qk")
    if case["op"] == "write":
        return _plain_write(state)
    if case["op"] == "read":
        return _plain_read(state["cache"], case["n"], state["first"], state["counts"], dt)
    if case["op"] == "commit":
        return _plain_commit(state)
    return _attend(state, torch.float32).to(dt)


# ------------------------------------------------------------ 64-bit answers

def _exact_turn(x, positions, f, magnitude, rot, interleaved, sign):
    """Pairs as complex numbers times magnitude exp(+- i position f)."""
    x = x.double()
    angle = positions.double()[:, None, :, None] * f
    turn = torch.polar(torch.full_like(angle, magnitude), sign * angle)
    y = x.clone()
    even = torch.arange(0, rot, 2, device="cuda") if interleaved else torch.arange(rot // 2, device="cuda")
    odd = even + (1 if interleaved else rot // 2)
    z = torch.complex(x[..., even], x[..., odd]) * turn
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _exact_frequencies(case):
    rot, factor = case["rot"], case["factor"]
    base = 10000.0 * (factor ** (rot / (rot - 2.0)) if case["scaling"] == "base" else 1.0)
    f, magnitude = [base ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    if case["scaling"] == "linear":
        f = [w / factor for w in f]
    elif case["scaling"] == "parts":
        keep = [min(1.0, max(0.0, (case["trained"] * w / math.tau - 1.0) / 31.0)) for w in f]
        f = [w * g + w / factor * (1.0 - g) for w, g in zip(f, keep)]
        magnitude = 1.0 + math.log(factor) / 10.0
    return torch.tensor(f, dtype=torch.float64, device="cuda"), magnitude


def _exact_store(x):
    """The value that an 8-bit row stands for, from the definition: three bits behind the leading one."""
    x = x.double()
    power = lambda e: ((e.long() + 1023) << 52).view(torch.float64)       # 2^e
    most = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -150)
    e = torch.ceil(torch.log2(most / 448.0))
    e = torch.where(most > 448.0 * power(e), e + 1, e)
    e = torch.where(most <= 448.0 * power(e - 1), e - 1, e).clamp(-117, 120)
    y = x * power(-e)
    step = power(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * power(e)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        f, magnitude = _exact_frequencies(case)
        sign = -1.0 if case["gradient"] else 1.0
        return tuple(_exact_turn(s[name], s["positions"], f, magnitude, case["rot"], case["interleaved"], sign)
                     for name in "qk")
    if op == "write":
        n = case["n"]
        k, v, q = s["k"].double(), s["v"].double(), None
        if case["rotary"]:
            f, magnitude = _exact_frequencies(dict(WRITE_ROTARY, rot=case["dh"]))
            k, q = (_exact_turn(s[name], s["positions"], f, magnitude, case["dh"], False, 1.0) for name in "kq")
        counts = s["counts"] if s["counts"] is not None else torch.full_like(s["first"], n)
        live = torch.arange(n, device="cuda")[None] < counts[:, None]
        if case["cache"] == "e4m3":
            return dict(q=q, rows=[torch.where(live[:, None, :, None], _exact_store(x), 0) for x in (k, v)])
        out = dict(q=q)
        for name, x in (("k", k), ("v", v)):
            pool = s["cache"][name].double()
            b, i = live.nonzero(as_tuple=True)
            index = s["first"].long()[b] + i
            page = s["cache"]["table"].long()[b, index // case["page"]]
            pool[page, :, index % case["page"]] = x.transpose(1, 2)[b, i]
            out[name] = pool
        return out
    if op == "read":
        n = case["n"]
        live = torch.arange(n, device="cuda")[None] < s["counts"][:, None]
        rows = [_dense(s["cache"], name, torch.float64)[:, :, :n] for name in "kv"]
        return [torch.where(live[:, None, :, None], x, 0) for x in rows]
    if op == "commit":
        m = s["path"].shape[1]
        live = torch.arange(m, device="cuda")[None] < s["lengths"][:, None]
        old = (s["first"][:, None] + s["path"]).long()
        rows = []
        for name in "kv":
            x = _dense(s["cache"], name, torch.float64)
            x = x.gather(2, old[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3]))
            rows.append(torch.where(live[:, None, :, None], x, 0))
        if case["cache"] == "e4m3":
            return rows
        pools = []
        for name, x in zip("kv", rows):
            pool = s["cache"][name].double()
            b, j = live.nonzero(as_tuple=True)
            index = s["first"].long()[b] + j
            page = s["cache"]["table"].long()[b, index // case["page"]]
            pool[page, :, index % case["page"]] = x.transpose(1, 2)[b, j]
            pools.append(pool)
        return tuple(pools)
    if 4.0 * case["batch"] * case["H"] * case["n"] * (case["prefix"] + case["n"]) * case["dh"] > 3e12:
        return None
    return _exact_attend(s)


def _exact_attend(s):
    """Row by row of the tree, from the definition: the keys that it sees, their weights, their values."""
    case, q = s["case"], s["q"].double()
    batch, H, n, dh = q.shape
    group, page = H // case["Hkv"], case["page"]
    out = torch.zeros(batch, H, n, dh, dtype=torch.float64, device="cuda")
    for b in range(batch):
        prefix = int(s["prefix"][b])
        count = int(s["counts"][b]) if s["counts"] is not None else n
        one = {name: (x[b:b + 1] if name == "table" else x) for name, x in s["cache"].items()}
        k, v = (_dense(one, name, torch.float64)[0, :, :prefix + count] for name in "kv")
        see = torch.ones(count, prefix + count, dtype=torch.bool, device="cuda")
        see[:, prefix:] = s["mask"][b, :count, :count].bool() if s["mask"] is not None else torch.ones(
            count, count, dtype=torch.bool, device="cuda").tril()
        x = torch.einsum("hgnd,hkd->hgnk", q[b, :, :count].view(-1, group, count, dh), k) / math.sqrt(dh)
        x = torch.where(see, x, -math.inf)
        w = torch.exp(x - x.logsumexp(-1, keepdim=True))
        out[b, :, :count] = torch.einsum("hgnk,hkd->hgnd", torch.where(see, w, 0.0), v).reshape(H, count, dh)
    return out


def work(case):
    """Inputs once, outputs once; the lengths at their means."""
    op, batch, dh, Hkv = case["op"], case["batch"], case["dh"], case["Hkv"]
    n = case["n"]
    row = 2 * dh if case.get("cache") != "e4m3" else dh + 1            # a cached head row
    if op == "rotary":
        values = batch * n * (case["H"] + Hkv) * dh
        return dict(bytes=2 * 2 * values + 4 * batch * n, flops=3 * values * case["rot"] / dh)
    if op == "write":
        rows = batch * n * (0.67 if case["cut"] else 1.0) * 2 * Hkv
        q = 2 * 2 * batch * n * case["H"] * dh if case["rotary"] else 0
        back = rows * row + 2 * batch * n * 2 * Hkv * dh if case["cache"] == "e4m3" else 0
        return dict(bytes=rows * (2 * dh + row) + q + back, flops=0)
    if op == "read":
        rows = batch * 2 * Hkv * (case["low"] + n) / 2
        return dict(bytes=rows * row + 2 * batch * n * 2 * Hkv * dh, flops=0)
    if op == "commit":
        most = min(case["depth"], n)
        rows = batch * 2 * Hkv * max(1.0, most / 3)
        back = rows * row + 2 * batch * most * 2 * Hkv * dh if case["cache"] == "e4m3" else 0
        return dict(bytes=2 * rows * row + back, flops=0)
    mean = (case["low"] + case["prefix"]) / 2
    tree = n * (0.67 if case["cut"] else 1.0)
    keys = mean + (tree if case["mask"] == "tree" else tree / 2)
    return dict(bytes=2 * batch * Hkv * (mean + tree) * row + 2 * 2 * batch * case["H"] * n * dh,
                flops=4 * batch * case["H"] * tree * keys * dh)
