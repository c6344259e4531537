"""Run a few attention calls of one staged layer, for profiler captures.

    python -m sliding_window_gqa_ring_gb300.profile_case --case swa_mixed --calls 3

The layer is staged from the seeded workloads in ``synth`` (rings or caches
written with carat_ring_append), then the step's fused append+attention call
repeats ``--calls`` times (with ``--separate``: one carat_ring_append, then the
attention call alone repeats), so a profiler filtered on the attention kernel
sees exactly ``--calls`` launches.  The ``paged_*`` cases run the paged operators
over random contents instead.  Every case but global_mixed keeps a few
GB or less on the device; every case reads more than the 129 MB L2 per call.
"""
from __future__ import annotations

import argparse

import torch

from . import carat, engine, synth

CASES = {
    "swa_b1": lambda: synth.sliding_single(),
    "swa_b56": lambda: synth.sliding_batched(),
    "swa_mixed": lambda: synth.mixed_step()[0],
    "global_single": lambda: synth.global_single(),
    "global_sweep4": lambda: synth.global_sweep(4),
    "global_sweep15": lambda: synth.global_sweep(15),
    # the mixed step's global layer: about 9 GB of caches, for one-pass captures only
    "global_mixed": lambda: synth.mixed_step()[1],
    # the mixed step's sliding layer with FP8 e4m3 rings (append once, then the
    # attention call repeats)
    "swa_mixed_fp8": lambda: synth.mixed_step()[0],
}

# Paged operators over random contents: (requests, proposals, query heads, KV heads,
# head_dim, keys per request)
PAGED = {
    # attention over e4m3 pages with block scales, 268 MB of them
    "paged_fp8": (64, 4, 16, 2, 512, 2048),
    "paged_fp8_120_rows": (8, 15, 16, 2, 512, 8192),
    # its tiles of 8 rows, two CTAs an SM (235 MB of pages)
    "paged_fp8_decode": (56, 1, 16, 8, 256, 1024),
    # rotary appends of eight ragged prompts (the keys are the prompt's)
    "paged_rope": (8, 1024, 16, 8, 256, 0),
    "paged_rope_fp8": (8, 1024, 16, 8, 256, 0),
}


def run_paged(case: str, calls: int):
    batch, k, hq, hkv, d, keys = PAGED[case]
    page_rows, block_rows = 256, 64
    pages = -(-max(keys, k) // page_rows)
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randperm(batch * pages, generator=g, device="cuda").int().view(batch, pages)
    shape = (batch * pages, page_rows, hkv, d)
    q = torch.randn((batch, k, hq, d), generator=g, device="cuda").bfloat16()
    out = torch.empty_like(q)
    scales = torch.full((batch * pages, page_rows // block_rows, hkv), 2.0 ** -6, device="cuda")
    if case.startswith("paged_fp8"):
        kp, vp = (torch.randn(shape, generator=g, device="cuda").mul_(60).to(torch.float8_e4m3fn)
                  .view(torch.uint8) for _ in range(2))
        ctx = torch.full((batch,), keys - k, dtype=torch.int32, device="cuda")
        ws = carat.workspace_tensor(
            carat.paged_fp8_workspace_bytes(batch, k, hq, hkv, d, pages * page_rows))
        for _ in range(calls):
            carat.carat_paged_verify_attention_fp8(out, q, kp, vp, scales, scales, table, ctx,
                                                   scale=d ** -0.5, workspace=ws)
        return
    dtype = torch.uint8 if case.endswith("fp8") else torch.bfloat16
    kp, vp = (torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2))
    v_scales = scales.clone()
    kn, vn = (torch.randn((batch, k, hkv, d), generator=g, device="cuda").bfloat16()
              for _ in range(2))
    ctx = torch.zeros(batch, dtype=torch.int32, device="cuda")
    counts = torch.arange(batch, device="cuda", dtype=torch.int32) * (k // 2) // batch + k // 2
    rope = dict(cos_sin=engine.rotary_table(k, 64), interleaved=True, queries=q, queries_out=out,
                new_counts=counts)
    for _ in range(calls):
        if dtype == torch.uint8:
            carat.carat_paged_rope_append_fp8(kp, vp, scales, v_scales, table, kn, vn, ctx,
                                              **rope)
        else:
            carat.carat_paged_rope_append(kp, vp, table, kn, vn, ctx, **rope)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--case", choices=sorted([*CASES, *PAGED]), required=True)
    ap.add_argument("--calls", type=int, default=3)
    ap.add_argument("--separate", action="store_true",
                    help="time carat_ring_append + the attention call instead of the fused call")
    args = ap.parse_args()
    if args.case in PAGED:
        run_paged(args.case, args.calls)
        torch.cuda.synchronize()
        status = carat.carat_get_device_status(clear=True)
        print(f"{args.case}: {args.calls} calls, device status {status:#x}")
        if status:
            raise SystemExit(1)
        return
    w = CASES[args.case]()
    if args.case.endswith("_fp8"):
        # scales as a caller would calibrate them: max |x| / 448 over the layer
        probe = engine.SlidingLayer(w.batch, window=w.window, q_heads=w.q_heads,
                                    kv_heads=w.kv_heads, head_dim=w.head_dim,
                                    max_proposals=w.proposal_count, scale=w.scale)
        hist = engine.stage_sliding(w, 0, probe).host["hist"]
        kmax = max(float(abs(synth.bf16_to_float(h[1])).max()) for h in hist.values())
        vmax = max(float(abs(synth.bf16_to_float(h[2])).max()) for h in hist.values())
        del probe
        layer = engine.Fp8SlidingLayer(w.batch, k_scale=kmax / 448.0, v_scale=vmax / 448.0,
                                       window=w.window, q_heads=w.q_heads, kv_heads=w.kv_heads,
                                       head_dim=w.head_dim, max_proposals=w.proposal_count,
                                       scale=w.scale)
        inp = engine.stage_sliding(w, 0, layer)
        out = torch.empty(inp.queries.shape, dtype=torch.float32, device=layer.device)
        layer.append(inp.k_new, inp.v_new, inp.context_lengths)
        for _ in range(args.calls):
            layer.attend(inp.queries, inp.context_lengths, out=out)
        torch.cuda.synchronize()
        status = carat.carat_get_device_status(clear=True)
        print(f"{args.case}: {args.calls} calls, device status {status:#x}")
        if status:
            raise SystemExit(1)
        return
    if w.window:
        layer = engine.SlidingLayer(w.batch, window=w.window, q_heads=w.q_heads,
                                    kv_heads=w.kv_heads, head_dim=w.head_dim,
                                    max_proposals=w.proposal_count, scale=w.scale)
        inp = engine.stage_sliding(w, 0, layer)
    else:
        layer = engine.GlobalLayer(w.batch, capacity=w.capacity, q_heads=w.q_heads,
                                   kv_heads=w.kv_heads, head_dim=w.head_dim,
                                   max_proposals=w.proposal_count, scale=w.scale)
        inp = engine.stage_global(w, 0, layer, keep_history=False)
    out = torch.empty(inp.queries.shape, dtype=torch.float32, device=layer.device)
    if args.separate:
        layer.append(inp.k_new, inp.v_new, inp.context_lengths)
        for _ in range(args.calls):
            layer.attend(inp.queries, inp.context_lengths, out=out)
    else:
        for _ in range(args.calls):
            layer.step(inp.queries, inp.k_new, inp.v_new, inp.context_lengths, out=out)
    torch.cuda.synchronize()
    status = carat.carat_get_device_status(clear=True)
    print(f"{args.case}: {args.calls} calls, device status {status:#x}")
    if status:
        raise SystemExit(1)


if __name__ == "__main__":
    main()
