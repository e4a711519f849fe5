"""Run one API call on a named workload, a few times, for a profiler.

    python -m sliding_window_attention_band_gb300.run_workload \\
        --workload causal_fp16_n32768_w4096 --call band_attention --repeat 3

Builds the workload's seeded inputs on the current CUDA device, calls the
fused forward (``band_attention``), the fused forward then its backward
(``band_attention_bwd``, only the backward repeated) or, the workload's
sequences as prompts in the paged cache, steps of one token for each of them
(``decode``: cache_slots, rotary_append, band_decode) ``--repeat`` times,
synchronises, checks the device status word and exits 0.  It prints nothing
but one line with the call and the status, so a profiler's launch list holds
only the library's kernels and torch's input copies.
"""
from __future__ import annotations

import argparse

import torch

import sliding_window_attention_band_gb300 as swab
from sliding_window_attention_band_gb300.decode_loop import DecodeLoop
from sliding_window_attention_band_gb300.inputs import WORKLOADS, workload_inputs


def main() -> int:
    names = {wl.name: wl for wl in WORKLOADS.values()}
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", required=True, choices=sorted(names))
    ap.add_argument("--call", default="band_attention", choices=["band_attention", "band_attention_bwd", "decode"])
    ap.add_argument("--repeat", type=int, default=3)
    args = ap.parse_args()
    wl = names[args.workload]
    swab.load()
    if args.call == "decode":
        return decode(wl, args.repeat)
    d = swab.Desc.from_workload(wl)
    Q, K, V, dO = (x.cuda() for x in workload_inputs(wl))
    O = torch.empty_like(Q)
    lse = torch.empty(wl.BH, wl.n, dtype=torch.float32, device="cuda")
    fwd = lambda: swab.band_attention(d, wl.scale, Q, K, V, O, lse)
    if args.call == "band_attention":
        for _ in range(args.repeat):
            fwd()
    else:
        fwd()
        dQ, dK, dV = (torch.empty_like(Q) for _ in range(3))
        ws = torch.empty(swab.band_attention_bwd_workspace(d) // 4, dtype=torch.float32, device="cuda")
        for _ in range(args.repeat):
            swab.band_attention_bwd(d, wl.scale, Q, K, V, O, dO, lse, dQ, dK, dV, ws)
    torch.cuda.synchronize()
    status = swab.device_status(reset=True)
    print(f"{args.call} {wl.name} x{args.repeat}: status {status}")
    return 0 if status == 0 else 1


def decode(wl, repeat) -> int:
    """`repeat` steps behind the workload's sequences, replayed from a graph."""
    loop = DecodeLoop.from_workload(wl)
    heads = [x.view(wl.b, wl.h, wl.n, wl.head_dim).transpose(1, 2).reshape(wl.b * wl.n, wl.h, wl.head_dim).cuda()
             for x in workload_inputs(wl, count=3)]
    qkv = torch.cat(heads, dim=1)
    loop.fill(qkv, torch.full((wl.b,), wl.n, dtype=torch.int32, device="cuda"))
    loop.n_new.fill_(1)
    loop.qkv.copy_(qkv[:wl.b])
    loop.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step()
    for _ in range(repeat):
        graph.replay()
    torch.cuda.synchronize()
    status = swab.device_status(reset=True)
    ok = status == 0 and loop.lens.tolist() == [wl.n + 1 + repeat] * wl.b and bool(torch.isfinite(loop.out).all())
    print(f"decode {wl.name} x{repeat}: status {status}")
    return 0 if ok else 1


if __name__ == "__main__":
    raise SystemExit(main())
