"""A served layer's round (profile_cases layer): page tables, norm, projections with adapters, the cache
and its attention, as they are used together, each step against a plain 64-bit form of what it was
given."""
import pytest
import torch

import _cache_ref
import _layer_ref as R

pytestmark = pytest.mark.gpu


def near(got, ref, slack, what):
    got = got.double().cpu().reshape(ref.shape)
    over = (got - ref).abs() - slack
    assert bool(torch.isfinite(got).all()) and float(over.max()) <= 0, f"{what}: over by {float(over.max()):.3g}"


@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
def test_layer_round(cache, capsys):
    from conditional_draft_tree_gb300 import build, profile_cases
    build.build()
    d, H, Hkv, dh, page, most, least = 256, 8, 2, 64, 16, 70, 33
    o = profile_cases.case_layer(0, 2, torch.device("cuda", 0), cache, d=d, H=H, Hkv=Hkv, dh=dh, page=page, most=most,
                                 least=least, adapters=3)
    assert "layer_us" in capsys.readouterr().out
    kind, eight = (torch.float16 if cache == "fp16" else torch.bfloat16), cache == "e4m3"
    batch, n = o["x"].shape[:2]
    prefix, kept = o["prefix"].tolist(), o["kept"].tolist()
    # pages: enough for the trees while they are there, then for what was accepted
    assert o["held"].tolist() == [-(-(p + n) // page) for p in prefix]
    assert o["pool"].held.tolist() == [-(-k // page) for k in kept]
    table = o["cache"].table.tolist()
    live = [x for row in table for x in row if x >= 0]
    free = o["pool"].free_pages[:int(o["pool"].state[0])].tolist()
    assert sorted(live + free) == list(range(o["cache"].k.shape[0]))
    assert o["rows"].tolist() == [list(range(p, p + n)) for p in prefix]
    for b in range(batch):
        for i in range(kept[b] - prefix[b]):        # rows on pages that are still held
            at = prefix[b] + i
            assert int(o["slots"][b, i]) == table[b][at // page] * page + at % page
    # norm and projections
    def projected(y, rows8, projection, adapters, got, what):
        w = projection.weight
        vw = R.from_rows8(w.codes.cpu(), w.exps.cpu()) if eight else w.cpu().double()
        vy = R.from_rows8(rows8.codes.cpu(), rows8.exps.cpu()) if eight else y.cpu().double()
        y, vy = y.cpu().reshape(-1, y.shape[-1]), vy.reshape(-1, vy.shape[-1])
        low = (o["index"].cpu(), y, adapters.down.cpu(), adapters.up.cpu(), adapters.scale.cpu())
        ref = R.project(vy, vw, n, *low)
        near(got, ref, R.project_slack(vy, vw, n, ref, kind, *low), what)

    for norm, x, res, y, total, what in ((o["norms"][0], o["x"], o["residual"], o["y"], o["total"], "first norm"),
                                         (o["norms"][1], o["z"], o["total"], o["w"], o["total2"], "second norm")):
        ref, t = R.norm(x.cpu(), res.cpu(), norm.weight.cpu(), norm.offset, norm.eps)
        near(y, ref, R.norm_slack(ref, kind), what)
        near(total, t, (R.HALF[kind] + 2.0 ** -24) * t.abs() + R.TINY[kind], what)
    projected(o["y"], o["y8"], o["qkv"], o["own_qkv"], o["p"].transpose(1, 2), "queries, keys and values")
    from conditional_draft_tree_gb300 import quantize_rows
    projected(o["seen"], quantize_rows(o["seen"]) if eight else None, o["output"], o["own_output"], o["z"], "output")
    # queries are turned to their positions
    f, mag = _cache_ref.frequencies(dh, 1e6)
    q = o["p"][:, :H].cpu()
    ref = _cache_ref.turn(q, o["positions"].cpu(), f, mag, False)
    near(o["q"], ref, R.HALF[kind] * ref.abs() + R.TINY[kind] + 2 * _cache_ref.turn_slack(q, dh, mag, False), "queries")
    o["cache"].check()
