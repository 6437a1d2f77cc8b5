"""Run chosen library calls of one rollout workload a few times, untimed.

For profilers (ncu with -k / -s / -c): the calls are the steps of
RacLinearPlan on synthetic inputs of the workload's shape, issued directly
(no CUDA graph), so each launch appears on its own.

    python -m precision_rl_rollout_nvfp4_b200.run_calls --M 32768 --K 4096 --N 4096 \
        --calls prepare_weight,quantize,select,weight_select,gemm --reps 2

The MXFP4 and gated feed-forward calls take the same sizes (N is the inner
size F of the block) and need none of the plan's steps:

    python -m precision_rl_rollout_nvfp4_b200.run_calls --M 8192 --K 4096 --N 11008 \
        --calls mxfp4_quantize,mxfp4_gemm,mxfp4_gated_gemm,gated_forward,gated_backward --reps 1
"""
from __future__ import annotations

import argparse


BLOCK_CALLS = ("mxfp4_quantize", "mxfp4_dequantize", "mxfp4_qdq", "mxfp4_gemm", "mxfp4_linear", "mxfp4_gated_gemm",
               "mxfp4_gated_mlp", "gated_forward", "gated_backward")


def block_calls(B, S, a, dev, names):
    """The MXFP4 and gated calls among `names`, on synthetic inputs; the operands
    that only other calls take are not made."""
    import torch
    names = [n for n in names if n in BLOCK_CALLS]
    if not names:
        return {}

    def needs(*calls):
        return any(n in calls for n in names)

    x = S.activations(a.M, a.K).to(dev)
    wg, wu = S.weights(a.N, a.K, seed=1).to(dev), S.weights(a.N, a.K, seed=2).to(dev)
    if needs("mxfp4_dequantize", "mxfp4_gemm", "mxfp4_gated_gemm"):
        qx = B.mxfp4_quantize(x)
    if needs("mxfp4_gemm", "mxfp4_linear", "mxfp4_gated_gemm", "mxfp4_gated_mlp"):
        qg, qu = B.mxfp4_quantize(wg), B.mxfp4_quantize(wu)
    if needs("mxfp4_gated_mlp"):
        qd = B.mxfp4_quantize(S.weights(a.K, a.N, seed=3).to(dev))
    if needs("gated_backward"):
        dh = S.activations(a.M, a.N, seed=4).to(dev)
    y_dtype = torch.bfloat16 if a.y_dtype == "bf16" else torch.float32
    saved = []
    fns = {"mxfp4_quantize": lambda: B.mxfp4_quantize(x), "mxfp4_dequantize": lambda: B.mxfp4_dequantize(qx),
           "mxfp4_qdq": lambda: B.mxfp4_qdq(wg), "mxfp4_gemm": lambda: B.mxfp4_gemm(qx, qg, y_dtype),
           "mxfp4_linear": lambda: B.mxfp4_linear(x, qg, y_dtype),
           "mxfp4_gated_gemm": lambda: B.mxfp4_gated_gemm(qx, qg, qu, out_dtype="mxfp4"),
           "mxfp4_gated_mlp": lambda: B.mxfp4_gated_mlp(x, qg, qu, qd, out_dtype=y_dtype),
           "gated_forward": lambda: saved.append(B.gated_linear_forward(x, wg, wu, save=True)[1]),
           "gated_backward": lambda: B.gated_linear_backward(x, wg, wu, dh, saved=saved[-1] if saved else None)}
    return {n: fns[n] for n in names}


def main(argv=None):
    import torch

    from . import binding as B
    from . import synthetic as S

    p = argparse.ArgumentParser()
    p.add_argument("--M", type=int, default=32768)
    p.add_argument("--K", type=int, default=4096)
    p.add_argument("--N", type=int, default=4096)
    p.add_argument("--k", type=float, default=50.0)
    p.add_argument("--calls", default="prepare_weight,quantize,select,weight_select,gemm")
    p.add_argument("--reps", type=int, default=2)
    p.add_argument("--y-dtype", choices=["bf16", "fp32"], default="bf16")
    a = p.parse_args(argv)
    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    calls = [c for c in a.calls.split(",") if c]
    block = block_calls(B, S, a, dev, calls)
    if block and len(block) == len(set(calls)):
        for _ in range(a.reps):
            for c in calls:
                block[c]()
        return finish(B, a, calls)
    if block:
        raise SystemExit("the MXFP4 and gated calls run apart from the plan's")
    x = S.activations(a.M, a.K).to(dev)
    w = S.weights(a.N, a.K).to(dev)
    plan = B.RacLinearPlan(a.M, a.K, a.N, a.k, out_dtype=torch.bfloat16 if a.y_dtype == "bf16" else torch.float32,
                           device=dev).bind(x, w)
    fns = {"prepare_weight": plan.prepare_weight, "quantize": plan.quantize, "select": plan.select,
           "weight_select": plan.weight_select, "gemm": plan.gemm, "gemm_plain": lambda: plan.gemm(plain=True),
           "quantize_plain": lambda: plan.quantize(scores=False), "quantize_select": plan.quantize_select,
           "second_pass": plan.second_pass, "select_channels": plan.select_channels}
    # the steps depend on each other: one full pass first
    plan.prepare_weight()
    plan.quantize()
    plan.select()
    plan.weight_select()
    plan.gemm()
    for _ in range(a.reps):
        for c in calls:
            fns[c]()
    finish(B, a, calls)


def finish(B, a, calls):
    import torch
    torch.cuda.synchronize()
    st = B.stream_status()
    if st != 0:
        raise SystemExit(f"device error word set: {st}")
    print(f"ok: {a.M}x{a.K}x{a.N} k={a.k} calls={calls} reps={a.reps}")


if __name__ == "__main__":
    main()
