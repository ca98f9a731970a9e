"""Fixed single-GPU workloads for kernel profiling and timing.

    python -m conditional_draft_tree_gb300.profile_cases topm  [--reps R] [--cfg C]
        top-M of a workload's base logits (Qwen3-8B batch 32 by default:
        480 rows x 151936 fp32, 292 MB) through dt_select_topm_noalloc. Its
        kernel is dt_build_trees' top-M kernel, and the launch shape is the same
        while the row segments' partial lists fit in the static scratch (true
        for this workload; a larger one, such as the batch-128 M = 256 stress
        configuration, falls back to one block per row segment). Only the
        logits and the outputs live on the device.
    python -m conditional_draft_tree_gb300.profile_cases round [--reps R] [--cfg C] [--flags F]
        R whole dt_build_trees rounds of the workload (weights, prepared table
        and workspace on the device: about 3.5 GB for the default workload);
        F = dt_options flags (default 0).
    python -m conditional_draft_tree_gb300.profile_cases marginal [--reps R] [--cfg C]
        R marginal-score rounds (DT_OPT_MARGINAL): top-M and the marginal tree
        kernel, no weights on the device.
    python -m conditional_draft_tree_gb300.profile_cases verify [--reps R] [--cfg C]
        R launches of one tree-attention layer over the workload's trees
        (32 query heads, 8 key/value heads, dh 128, prefix cache of 1024 keys
        with lengths in [512, 1024]; synthetic bf16 Q/K/V).
    python -m conditional_draft_tree_gb300.profile_cases serve [--reps R] [--cfg C] [--cache T]
        One verification round of the workload's trees against a paged cache, one
        layer of it as a server runs it: the trees' keys and values written behind
        each request's prefix (queries and keys turned to their positions on the
        way), attention of all rows over the cache, and the rows of one path of
        each tree (its deepest, in place of what a target model would accept)
        committed behind the prefix. T = bf16 (default), fp16 or e4m3; 32 query
        heads, 8 key/value heads, dh 128, pages of 64 rows, prefixes of 512 to
        1024 rows, synthetic Q/K/V.
    python -m conditional_draft_tree_gb300.profile_cases chain [--reps R] [--cfg C] [--greedy]
        R Domino chain-decoding rounds (dt_decode_chains) of the workload,
        sampled at its temperatures with seeded uniform draws, or greedy: one
        projection launch and one decoding launch per round.

Each case does one untimed launch first, then R timed ones (CUDA events on the
current stream, L2 flushed by a 256 MB write before each), and prints one line
with the mean time. Run it under ncu with -k / -s / -c to capture one launch.
"""
from __future__ import annotations

import argparse

import torch

import conditional_draft_tree_gb300 as dt
import dt_workloads as W

L2_FLUSH_BYTES = 256 << 20


def _timed(fn, reps, dev):
    flush = torch.empty(L2_FLUSH_BYTES, dtype=torch.uint8, device=dev)
    fn()
    torch.cuda.synchronize()
    ms = []
    for i in range(reps):
        flush.fill_(i & 0xff)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        fn()
        b.record()
        torch.cuda.synchronize()
        ms.append(a.elapsed_time(b))
    return sum(ms) / len(ms)


def case_topm(cfg, reps, dev):
    wl = W.make_workload(cfg)
    logits = torch.from_numpy(wl.base_logits).to(dev)
    topm = torch.empty(wl.batch, wl.D, wl.M, dtype=torch.int32, device=dev)
    status = torch.empty(wl.batch, dtype=torch.int32, device=dev)

    def run():
        rc = dt.select_topm_noalloc(logits, wl.M, topm, status)
        if rc != dt.OK:
            raise dt.DtError(dt.status_string(rc))

    ms = _timed(run, reps, dev)
    gbs = logits.numel() * 4 / (ms * 1e-3) / 1e9
    print(f"topm {wl.name}: rows={wl.batch * wl.D} V={wl.V} M={wl.M} "
          f"mean_us={1000 * ms:.1f} GB/s={gbs:.0f}")


def case_round(cfg, reps, dev, flags=0):
    wl = W.make_workload(cfg)
    tb = dt.TreeBuilder.from_numpy(wl, device=dev, flags=flags)
    inp = tb.inputs_to_device(wl)
    out = dt.alloc_outputs(tb.dims, dev)
    ms = _timed(lambda: tb.run(**inp, out=out), reps, dev)
    print(f"round {wl.name}: batch={wl.batch} mean_us={1000 * ms:.1f} "
          f"trees/s={wl.batch / (ms * 1e-3):.0f}")


def case_chain(cfg, reps, dev, greedy=False):
    wl = W.make_workload(cfg)
    dec = dt.ChainDecoder.from_numpy(wl, device=dev)
    inp = dec.inputs_to_device(wl, W.chain_uniforms(wl.batch, wl.D, seed=cfg))
    if greedy:
        inp["temperature"] = torch.zeros_like(inp["temperature"])
    out = dec.alloc_outputs()
    ms = _timed(lambda: dec.run(**inp, out=out), reps, dev)
    if not bool((out["status"] == 0).all()):
        raise dt.DtError("chain decoding reported a non-OK status")
    print(f"chain {wl.name}: batch={wl.batch} D={wl.D} mean_us={1000 * ms:.1f} "
          f"chains/s={wl.batch / (ms * 1e-3):.0f}")


def case_marginal(cfg, reps, dev):
    wl = W.make_workload(cfg)
    mb = dt.MarginalTreeBuilder.from_workload(wl, device=dev)
    inp = mb.inputs_to_device(wl)
    out = dt.alloc_outputs(mb.dims, dev)
    ms = _timed(lambda: mb.run(**inp, out=out), reps, dev)
    print(f"marginal {wl.name}: batch={wl.batch} mean_us={1000 * ms:.1f} "
          f"trees/s={wl.batch / (ms * 1e-3):.0f}")


def case_verify(cfg, reps, dev):
    import numpy as np
    wl = W.make_workload(cfg)
    tb = dt.TreeBuilder.from_numpy(wl, device=dev)
    trees = tb.run(**tb.inputs_to_device(wl))
    q, k, v, plen = W.verify_inputs(wl.batch, 32, 8, wl.N + 1, 1024, 128, seed=cfg,
                                    min_prefix=512)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(dev)
    qd, kd, vd, pd = t(q), t(k), t(v), torch.from_numpy(plen).to(dev)
    out = torch.empty((wl.batch, 32, wl.N + 1, 128), dtype=torch.float32, device=dev)
    ms = _timed(lambda: dt.tree_attention(qd, kd, vd, trees["mask"], pd, out=out), reps, dev)
    print(f"verify {wl.name}: batch={wl.batch} n1={wl.N + 1} mean_us={1000 * ms:.1f}")


def deepest_paths(parents, depths, width):
    """Rows from the root to each tree's deepest row: path [batch][width] int32 (-1 behind
    its end) and lengths [batch] int32. Rows that hold no node have depth -1."""
    parents, depths = parents.tolist(), depths.tolist()
    path = torch.full((len(parents), width), -1, dtype=torch.int32)
    lengths = torch.zeros(len(parents), dtype=torch.int32)
    for b, (up, depth) in enumerate(zip(parents, depths)):
        row, rows = max(range(len(depth)), key=depth.__getitem__), []
        while row > 0:
            rows.append(row)
            row = up[row]
        rows = [0] + rows[::-1]
        path[b, :len(rows)] = torch.tensor(rows, dtype=torch.int32)
        lengths[b] = len(rows)
    return path, lengths


def case_serve(cfg, reps, dev, cache_type="bf16", H=32, Hkv=8, dh=128, page=64, most=1024, least=512):
    wl = W.make_workload(cfg)
    tb = dt.TreeBuilder.from_numpy(wl, device=dev)
    trees = tb.run(**tb.inputs_to_device(wl))
    n, batch = wl.N + 1, wl.batch
    gen = torch.Generator(device=dev).manual_seed(cfg)
    normal = lambda heads, rows: torch.randn((batch, heads, rows, dh), device=dev, generator=gen).to(kind)
    kind = torch.float16 if cache_type == "fp16" else torch.bfloat16
    prefix = torch.randint(least, most + 1, (batch,), device=dev, generator=gen, dtype=torch.int32)
    pages = -(-(most + n) // page)        # of a request
    table = torch.randperm(batch * pages, device=dev, generator=gen).to(torch.int32).view(batch, pages)
    cache = dt.PagedCache.empty(batch * pages, Hkv, page, dh, table,
                                torch.float8_e4m3fn if cache_type == "e4m3" else kind)
    rot = dt.Rotary(dh, base=1e6, device=dev)
    # the prompts: positions 0 .. prefix - 1
    start = torch.zeros(batch, dtype=torch.int32, device=dev)
    positions = torch.arange(most, dtype=torch.int32, device=dev).repeat(batch, 1)
    dt.cache_write(cache, normal(Hkv, most), normal(Hkv, most), start, prefix, rotary=rot, positions=positions)
    # the round
    q, k, v = normal(H, n), normal(Hkv, n), normal(Hkv, n)
    positions = dt.tree_positions(trees["depths"], prefix)
    path, lengths = (t.to(dev) for t in deepest_paths(trees["parents"], trees["depths"], wl.D + 1))
    q_out, out = torch.empty_like(q), torch.empty_like(q)
    workspace = dt.cache_attention_workspace(cache, H, n)

    def write():
        dt.cache_write(cache, k, v, prefix, rotary=rot, positions=positions, q=q, q_out=q_out)

    def attend():
        dt.cache_attention(cache, q_out, prefix, mask=trees["mask"], out=out, workspace=workspace)

    def commit():
        dt.cache_commit(cache, prefix, path, lengths, n)

    def layer():
        write()
        attend()
        commit()

    ms = _timed(layer, reps, dev)
    parts = [_timed(f, reps, dev) for f in (write, attend, commit)]
    cache.check()
    if not bool(torch.isfinite(out).all()):
        raise dt.DtError("attention gave values that are not finite")
    print(f"serve {wl.name}: batch={batch} n={n} cache={cache_type} committed={int(lengths.sum())} rows "
          f"layer_us={1000 * ms:.1f} write_us={1000 * parts[0]:.1f} attend_us={1000 * parts[1]:.1f} "
          f"commit_us={1000 * parts[2]:.1f}")
    return out, cache, prefix + lengths


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=["topm", "round", "chain", "marginal", "verify", "serve"])
    ap.add_argument("--greedy", action="store_true")
    ap.add_argument("--reps", type=int, default=3)
    ap.add_argument("--cfg", type=int, default=3)
    ap.add_argument("--flags", type=int, default=0)
    ap.add_argument("--cache", choices=["bf16", "fp16", "e4m3"], default="bf16")
    args = ap.parse_args()
    dev = torch.device("cuda", 0)
    from conditional_draft_tree_gb300 import build
    build.build()
    if args.case == "round":
        case_round(args.cfg, args.reps, dev, args.flags)
    elif args.case == "chain":
        case_chain(args.cfg, args.reps, dev, args.greedy)
    elif args.case == "marginal":
        case_marginal(args.cfg, args.reps, dev)
    elif args.case == "verify":
        case_verify(args.cfg, args.reps, dev)
    elif args.case == "serve":
        case_serve(args.cfg, args.reps, dev, args.cache)
    else:
        case_topm(args.cfg, args.reps, dev)


if __name__ == "__main__":
    main()
