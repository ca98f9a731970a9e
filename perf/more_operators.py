"""Workloads of the operators around the paged cache's attention: the norm with its residual, the
projection with low-rank adapters of many requests, block tables and slot maps from lengths.

A case names an operator (``op``), its sizes and its types. ``run`` computes one pass, either in
plain 32-bit torch operations or (``own``) through the library's entry points.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # the next token of a few requests between two layers: latency counts
        dict(name="norm-token", op="norm", type="bf16", rows=8, inner=1, d=4096, heads=1, pad=0, residual=True),
        # the query heads of two long prompts, each head normed, read where the projection wrote them
        dict(name="norm-heads", op="norm", type="fp16", rows=8198, inner=32, d=128, heads=48, pad=0, residual=False),
        # rows of an odd width at an odd distance, of a model that nobody padded
        dict(name="norm-odd", op="norm", type="bf16", rows=4099, inner=1, d=5001, heads=1, pad=2, residual=True),
        # the drafted trees of a serving batch: norm to 8 bits, then queries, keys and values of the
        # 8B shape in one 8-bit projection, some requests with adapters
        dict(name="norm-project-trees-e4m3", op="norm_project", type="bf16", weights="e4m3", batch=32, n=65, K=4096,
             O=6144, rank=16, adapters=8, bare=0.25),
        # one token of a few requests, each with an adapter or none: latency counts
        dict(name="project-token", op="project", type="bf16", weights="16", batch=8, n=1, K=4096, O=6144, rank=16,
             adapters=6, bare=0.25),
        # single tokens of the stress batch, many adapters, 8-bit weights
        dict(name="project-tokens-e4m3", op="project", type="bf16", weights="e4m3", batch=128, n=1, K=4096, O=4096,
             rank=32, adapters=64, bare=0.1),
        # the drafted trees of a serving batch, 16-bit weights
        dict(name="project-trees", op="project", type="bf16", weights="16", batch=32, n=65, K=4096, O=6144, rank=16,
             adapters=8, bare=0.25),
        # two long prompts through an output projection of an odd width, adapters of a high rank
        dict(name="project-prompt-odd", op="project", type="fp16", weights="16", batch=2, n=4099, K=4096, O=4001,
             rank=64, adapters=3, bare=0.0),
        # wide trees of many requests, 8-bit weights, nobody with an adapter
        dict(name="project-stress-e4m3", op="project", type="bf16", weights="e4m3", batch=32, n=257, K=4096, O=6144,
             rank=0, adapters=0, bare=1.0),
        # a verification round of a serving batch: pages for the trees, their rows' places, pages given back
        dict(name="reserve-round", op="reserve", batch=32, n=65, page=64, before=1024, after=1089, low=512, ended=0.0),
        # many requests in small pages: some end, some begin with long prompts, the others grow
        dict(name="reserve-stress", op="reserve", batch=512, n=33, page=16, before=16384, after=16417, low=0,
             ended=0.25),
        # the rows of long prompts in the pool, and their positions
        dict(name="slots-prompts", op="slots", batch=8, n=16385, page=64, low=9000),
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], its logarithm uniform."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_project", "project", "project", "project", "reserve", "slots"))
    kind = rng.choice(("bf16", "bf16", "fp16"))
    page = rng.choice((16, 32, 64, 128))
    if op == "norm":
        if rng.random() < 0.3:       # heads of a projection's output
            d, heads = rng.choice((64, 80, 96, 128, 256)), rng.choice((3, 6, 12, 24, 48))
            rows = _spread(rng, 1, max(1, 8198 * 48 * 128 // (heads * d)))
            return dict(op=op, type=kind, rows=rows, inner=max(1, heads * 2 // 3), d=d, heads=heads, pad=0,
                        residual=False)
        d = rng.choice((1, 8, 1, 8)) * _spread(rng, 16, 2048)
        rows = _spread(rng, 1, max(1, min(65536, 4099 * 5001 // d)))
        return dict(op=op, type=kind, rows=rows, inner=1, d=d, heads=1, pad=rng.choice((0, 0, 8, 3)),
                    residual=rng.random() < 0.6)
    if op in ("norm_project", "project"):
        weights = "e4m3" if op == "norm_project" else rng.choice(("16", "e4m3"))
        K = 16 * _spread(rng, 4, 512)
        O = rng.choice((1, 16, 128)) * _spread(rng, 8, 64)
        n = rng.choice((1, 1, _spread(rng, 2, 300), _spread(rng, 2, 300), _spread(rng, 300, 4099)))
        n = max(1, min(n, 32 * 257 * 4096 * 6144 // (K * O)))
        batch = _spread(rng, 1, max(1, min(128, 32 * 257 * 4096 * 6144 // (n * K * O), 32 * 257 // n)))
        rank = rng.choice((0, 16, 16, 32, 48, 64, 128))
        adapters = rng.choice((1, _spread(rng, 1, min(64, 2048 // rank)))) if rank else 0
        return dict(op=op, type=kind, weights=weights, batch=batch, n=n, K=K, O=O, rank=rank, adapters=adapters,
                    bare=rng.choice((0.0, 0.25, 0.8)) if adapters else 1.0)
    if op == "reserve":
        batch, after = _spread(rng, 1, 1024), _spread(rng, 1, 32768)
        after = min(after, 512 * 16417 // batch)
        before = rng.randrange(after + 1)
        return dict(op=op, batch=batch, n=_spread(rng, 1, 257), page=page, before=before, after=after,
                    low=rng.randrange(before + 1), ended=rng.choice((0.0, 0.0, 0.3)))
    batch = _spread(rng, 1, 128)
    n = _spread(rng, 1, max(1, 8 * 16385 // batch))
    return dict(op=op, batch=batch, n=n, page=page, low=rng.randrange(n + 1))


# ------------------------------------------------------------------ inputs

def _power(e):
    """2^e in 32 bits, exactly, for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _to_e4m3(x):
    """Rows of values as e4m3 codes and one exponent byte a row: the least e with max |x| <= 448 2^e."""
    x = x.float()
    most = x.abs().amax(-1)
    m, k = torch.frexp(most)
    e = (k.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)).clamp(-117, 120)
    q = x * _power(-e)[..., None]
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _from_e4m3(codes, exps, dtype):
    return codes.to(dtype) * _power(exps.to(torch.int32) - 127)[..., None].to(dtype)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _stream_rows(g, rows, d, dtype):
    """Rows of a residual stream: a few channels carry far larger values, as trained models' do."""
    x = _normal(g, rows, d)
    x *= 1.0 + 12.0 * (torch.arange(d, device="cuda") % 131 == 7)
    return x.to(dtype)


def _lengths(g, batch, low, high):
    return torch.randint(low, high + 1, (batch,), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "norm":
        dt = TYPES[case["type"]]
        rows, inner, d, heads, pad = (case[name] for name in ("rows", "inner", "d", "heads", "pad"))

        def view():
            x = _stream_rows(g, rows, heads * d + pad, dt)[:, :heads * d]
            return x.view(rows, heads, d)[:, :inner] if heads > 1 else x
        s["x"] = view()
        s["residual"] = view() if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * _normal(g, d)).to(dt)
    elif op in ("norm_project", "project"):
        dt = TYPES[case["type"]]
        batch, n, K, O, rank = (case[name] for name in ("batch", "n", "K", "O", "rank"))
        x = _stream_rows(g, batch * n, K, dt).view(batch, n, K)
        w = _normal(g, O, K) * K ** -0.5
        s["weight"] = tuple(_to_e4m3(w)) if case["weights"] == "e4m3" else w.to(dt)
        if op == "norm_project":
            s["x"], s["residual"] = x, _stream_rows(g, batch * n, K, dt).view(batch, n, K)
            s["norm"] = (1.0 + 0.2 * _normal(g, K)).to(dt)
        else:
            s["x"] = x
            if case["weights"] == "e4m3":      # the layer's input in both types, as the norm before it gave it
                s["x8"] = _to_e4m3(x)
        if rank:
            a = case["adapters"]
            s["down"] = (_normal(g, a, rank, K) * K ** -0.5).to(dt)
            s["up"] = (_normal(g, a, O, rank) * 0.3 * rank ** -0.5).to(dt)
            s["scale"] = 0.5 + torch.rand(a, generator=g, device="cuda")
            index = torch.randint(0, a, (batch,), generator=g, device="cuda", dtype=torch.int32)
            bare = torch.rand(batch, generator=g, device="cuda") < case["bare"]
            s["index"] = torch.where(bare, -1, index).to(torch.int32)
    elif op == "reserve":
        batch, page = case["batch"], case["page"]
        before = _lengths(g, batch, case["low"], case["before"])
        after = before + case["after"] - case["before"]
        ended = torch.rand(batch, generator=g, device="cuda") < case["ended"]
        begun = torch.rand(batch, generator=g, device="cuda") < case["ended"]
        s["before"] = torch.where(begun, 0, before).to(torch.int32)
        s["after"] = torch.where(ended, 0, after).to(torch.int32)
        s["first"] = (s["after"] - case["n"]).clamp(min=0)
        s["counts"] = torch.minimum(s["after"] - s["first"], torch.full_like(before, case["n"]))
        width = -(-max(case["after"], case["before"]) // page)
        held = -(-s["before"] // page)
        pages = batch * width + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        live = torch.arange(width, device="cuda")[None] < held[:, None]
        s["table"] = torch.where(live, order[:batch * width].view(batch, width), -1).to(torch.int32).contiguous()
        left = order[torch.cat([~live.view(-1), torch.ones(3, dtype=torch.bool, device="cuda")])]
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        s["free"][:left.numel()] = left
        s["held"] = held.to(torch.int32)
        s["state"] = torch.tensor([left.numel(), 0], dtype=torch.int32, device="cuda")
        s["pages"] = pages
    else:
        batch, page, n = case["batch"], case["page"], case["n"]
        s["counts"] = _lengths(g, batch, case["low"], n)
        s["first"] = _lengths(g, batch, 0, 2 * page)
        width = -(-(n + 2 * page) // page)
        s["pages"] = batch * width + 3
        s["table"] = torch.randperm(s["pages"], generator=g, device="cuda")[:batch * width].to(torch.int32)
        s["table"] = s["table"].view(batch, width).contiguous()
    if op in ("reserve", "slots"):       # the pool's rows play no part here: the smallest heads
        shape = (s["pages"], 1, case["page"], 16)
        s["k"], s["v"] = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return s


# ------------------------------------------------------------- plain forms

def _plain_norm(x, residual, weight):
    """The normed rows in 32 bits, and the sum of the two inputs."""
    r = x.float() if residual is None else x.float() + residual.float()
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS) * weight.float(), r


def _plain_project(s, x, x16):
    """x in 32 bits times the weights, and the adapters over the 16-bit rows."""
    w = s["weight"]
    w = _from_e4m3(*w, torch.float32) if isinstance(w, tuple) else w.float()
    y = x @ w.t()
    if "index" in s:
        at = s["index"].clamp(min=0).long()
        u = x16.float() @ s["down"][at].float().transpose(1, 2) * s["scale"][at][:, None, None]
        u = torch.where((s["index"] >= 0)[:, None, None], u, 0.0)
        y += u @ s["up"][at].float().transpose(1, 2)
    return y


def _plain_reserve(s, lengths):
    table, held, free, state = s["table"], s["held"], s["free"], s["state"]
    batch, width = table.shape
    need = (-(-lengths // s["case"]["page"])).clamp(min=0)
    grow, shrink = (need - held).clamp(min=0), (held - need).clamp(min=0)
    put = shrink.flip(0).cumsum(0).flip(0) - shrink          # pages that later requests give back
    take = grow.cumsum(0) - grow
    column = torch.arange(width, device="cuda")[None]
    count, back = state[0].long(), shrink.sum()
    # the free pages, and behind them those given back
    every = torch.cat([free.clone(), torch.full((batch * width + 1,), -1, dtype=torch.int32, device="cuda")])
    given = (column >= need[:, None]) & (column < held[:, None])
    place = torch.where(given, count + put[:, None] + held[:, None] - 1 - column, every.numel() - 1)
    every[place.view(-1)] = torch.where(given, table, -1).view(-1)
    wanted = (column >= held[:, None]) & (column < need[:, None]) & (take + grow <= count + back)[:, None]
    place = torch.where(wanted, count + back - 1 - take[:, None] - column + held[:, None], every.numel() - 1)
    table.copy_(torch.where(wanted, every[place], torch.where(given, -1, table)))
    held.copy_(torch.where(need < held, need, torch.where(take + grow <= count + back, need, held)))
    left = count + back - wanted.sum()
    at = torch.arange(free.numel(), device="cuda")
    free.copy_(torch.where((at >= count) & (at < left), every[:free.numel()], free))
    state[0] = left


def _plain_slots(s):
    case, page = s["case"], s["case"]["page"]
    at = torch.arange(case["n"], device="cuda")[None]
    live = at < s["counts"][:, None]
    row = torch.where(live, s["first"][:, None] + at, 0)
    slots = s["table"].long().gather(1, row // page) * page + row % page
    return torch.where(live, slots, -1), torch.where(live, row, -1).to(torch.int32)


# ------------------------------------------------------- the library's calls

def _projection(s):
    import conditional_draft_tree_gb300 as dt
    case = s["case"]
    if "projection" not in s:        # the weights, adapters and workspace that a server keeps
        w = s["weight"]
        s["projection"] = dt.Projection(dt.Rows8(*w) if isinstance(w, tuple) else w)
        s["set"] = dt.Adapters(s["down"], s["up"], s["scale"]) if "index" in s else None
        s["workspace"] = dt.project_workspace(s["projection"], case["batch"], case["n"], s["set"])
    return s["projection"], s["set"], s["workspace"]


def _own(s):
    import conditional_draft_tree_gb300 as dt
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        if "plan" not in s:
            s["plan"] = dt.Norm(s["weight"], eps=EPS)
        return dt.rms_norm(s["plan"], s["x"], s["residual"])
    if op == "project":
        projection, adapters, workspace = _projection(s)
        if "x8" not in s:
            return dt.project(projection, s["x"], adapters, s.get("index"), workspace=workspace)
        if "rows" not in s:
            s["rows"] = dt.Rows8(*s["x8"])
        return dt.project(projection, s["rows"], adapters, s.get("index"), x16=s["x"], workspace=workspace)
    if op == "norm_project":
        projection, adapters, workspace = _projection(s)
        if "plan" not in s:
            s["plan"] = dt.Norm(s["norm"], eps=EPS)
        (x16, rows), total = dt.rms_norm(s["plan"], s["x"], s["residual"], kind="both")
        return dt.project(projection, rows, adapters, s.get("index"), x16=x16, workspace=workspace), total
    if "cache" not in s:
        s["cache"] = dt.PagedCache(s["k"], s["v"], s["table"])
    if op == "slots":
        return dt.cache_slots(s["cache"], case["n"], s["first"], s["counts"])
    if "pool" not in s:
        s["pool"] = dt.PagePool(s["cache"], s["held"], s["free"], s["state"])
    dt.cache_reserve(s["pool"], s["after"])
    slots, positions = dt.cache_slots(s["cache"], case["n"], s["first"], s["counts"])
    dt.cache_reserve(s["pool"], s["before"])
    return slots, positions, s["table"], s["held"], s["free"], s["state"]


def run(state):
    if own:
        return _own(state)
    s, case = state, state["case"]
    op = case["op"]
    if op == "slots":
        return _plain_slots(s)
    if op == "reserve":
        _plain_reserve(s, s["after"])
        slots, positions = _plain_slots(s)
        _plain_reserve(s, s["before"])
        return slots, positions, s["table"], s["held"], s["free"], s["state"]
    dt = TYPES[case["type"]]
    if op == "norm":
        y, r = _plain_norm(s["x"], s["residual"], s["weight"])
        return y.to(dt) if s["residual"] is None else (y.to(dt), r.to(dt))
    if op == "norm_project":
        y, r = _plain_norm(s["x"], s["residual"], s["norm"])
        return _plain_project(s, _from_e4m3(*_to_e4m3(y), torch.float32), y.to(dt)).to(dt), r.to(dt)
    x = _from_e4m3(*s["x8"], torch.float32) if "x8" in s else s["x"].float()
    return _plain_project(s, x, s["x"]).to(dt)


# ------------------------------------------------------------ 64-bit answers

def _exact_norm(x, residual, weight):
    r = x.double() + (0 if residual is None else residual.double())
    size = r.pow(2).sum(-1, keepdim=True) / r.shape[-1] + EPS
    return weight.double() * r * size.rsqrt(), r


def _exact_e4m3(x):
    """The value that an 8-bit row stands for, from the definition: three bits behind the leading one."""
    power = lambda e: ((e.long() + 1023) << 52).view(torch.float64)       # 2^e
    most = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -150)
    e = torch.ceil(torch.log2(most / 448.0))
    e = torch.where(most > 448.0 * power(e), e + 1, e)
    e = torch.where(most <= 448.0 * power(e - 1), e - 1, e).clamp(-117, 120)
    y = x * power(-e)
    step = power(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * power(e)


def _exact_project(s, x, x16):
    """Request by request: the shared weights, and its own adapter's product added to them."""
    w = s["weight"]
    w = torch.ldexp(w[0].double(), w[1].long()[:, None] - 127) if isinstance(w, tuple) else w.double()
    out = []
    for b in range(x.shape[0]):
        y = torch.einsum("nk,ok->no", x[b], w)
        a = int(s["index"][b]) if "index" in s else -1
        if a >= 0:
            low = torch.einsum("nk,rk->nr", x16[b].double(), s["down"][a].double())
            y = y + float(s["scale"][a]) * torch.einsum("nr,or->no", low, s["up"][a].double())
        out.append(y)
    return torch.stack(out)


def _exact_round(s):
    """The pool as a list, request after request: what is given back first, then what is taken."""
    page, batch = s["case"]["page"], s["case"]["batch"]
    table, held = [row[:h] for row, h in zip(s["table"].tolist(), s["held"].tolist())], None
    array = s["free"].tolist()
    stack = array[:int(s["state"][0])]

    def reserve(lengths):
        need = [-(-x // page) for x in lengths.tolist()]
        for b in reversed(range(batch)):
            while len(table[b]) > need[b]:
                stack.append(table[b].pop())
        for b in range(batch):
            while len(table[b]) < need[b]:
                table[b].append(stack.pop())

    reserve(s["after"])
    places = [[-1] * s["case"]["n"] for _ in range(batch)]
    rows = [[-1] * s["case"]["n"] for _ in range(batch)]
    for b, (first, count) in enumerate(zip(s["first"].tolist(), s["counts"].tolist())):
        for i in range(count):
            rows[b][i] = first + i
            places[b][i] = table[b][(first + i) // page] * page + (first + i) % page
    reserve(s["before"])
    width = s["table"].shape[1]
    held = [len(row) for row in table]
    whole = [row + [-1] * (width - len(row)) for row in table]
    t = lambda x, kind=torch.int32: torch.tensor(x, dtype=kind, device="cuda")
    # behind the count the array keeps what it held: the round ends with as many pages as it began
    return (t(places, torch.int64), t(rows), t(whole), t(held), t(stack + array[len(stack):]), t([len(stack), 0]))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "reserve":
        return _exact_round(s)
    if op == "slots":
        page, n = case["page"], case["n"]
        slots = torch.full((case["batch"], n), -1, dtype=torch.int64, device="cuda")
        rows = torch.full((case["batch"], n), -1, dtype=torch.int32, device="cuda")
        for b, (first, count) in enumerate(zip(s["first"].tolist(), s["counts"].tolist())):
            at = torch.arange(first, first + count, device="cuda")
            rows[b, :count] = at.to(torch.int32)
            slots[b, :count] = (s["table"][b].long()[:, None] * page + torch.arange(page, device="cuda")).view(-1)[at]
        return slots, rows
    if op == "norm":
        y, r = _exact_norm(s["x"], s["residual"], s["weight"])
        return y if s["residual"] is None else (y, r)
    if 2.0 * case["batch"] * case["n"] * case["K"] * case["O"] > 3e12:
        return None
    if op == "norm_project":
        y, r = _exact_norm(s["x"], s["residual"], s["norm"])
        return _exact_project(s, _exact_e4m3(y), y.to(TYPES[case["type"]])), r
    x = torch.ldexp(s["x8"][0].double(), s["x8"][1].long()[..., None] - 127) if "x8" in s else s["x"].double()
    return _exact_project(s, x, s["x"])


def work(case):
    """Inputs once, outputs once; lengths and shares at their means."""
    op = case["op"]
    if op == "norm":
        values = case["rows"] * case["inner"] * case["d"]
        return dict(bytes=2 * values * (4 if case["residual"] else 2) + 2 * case["d"], flops=4 * values)
    if op in ("norm_project", "project"):
        rows, K, O, rank = case["batch"] * case["n"], case["K"], case["O"], case["rank"]
        size = 1 if case["weights"] == "e4m3" else 2
        with_one = case["batch"] * (1.0 - case["bare"])
        used = case["adapters"] * (1.0 - (1.0 - 1.0 / max(1, case["adapters"])) ** with_one)
        flops = 2 * rows * K * O + 2 * with_one * case["n"] * rank * (K + O)
        data = size * K * O + 2 * rows * O + 2 * used * rank * (K + O)
        if op == "norm_project":
            return dict(bytes=data + 6 * rows * K, flops=flops + 4 * rows * K)
        return dict(bytes=data + (2 if size == 2 else 1) * rows * K + (2 * with_one * case["n"] * K if size == 1 and rank else 0),
                    flops=flops)
    if op == "reserve":
        changed = case["batch"] * (case["ended"] * (case["low"] + case["before"]) + case["after"] - case["before"]) / case["page"]
        return dict(bytes=2 * (8 * case["batch"] * 3 + 8 * changed) + 12 * case["batch"] * case["n"], flops=0)
    rows = case["batch"] * (case["low"] + case["n"]) / 2
    return dict(bytes=4 * rows / case["page"] + 12 * case["batch"] * case["n"], flops=0)
