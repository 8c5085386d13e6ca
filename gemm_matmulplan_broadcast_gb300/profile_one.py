"""Run one MatMul product, or one layer plan's forward and backward, a few
times, for a profiler or a quick timing.

    python -m gemm_matmulplan_broadcast_gb300.profile_one --a 2048,2048 --b 2048,2048 \\
        --dtype float64 [--reps 3] [--algorithm NAME] [--variant V] [--a-offset E]
    python -m gemm_matmulplan_broadcast_gb300.profile_one --layer norm --a 16384,4096
    python -m gemm_matmulplan_broadcast_gb300.profile_one --layer gate --a 2048,1024 --b 1024,2816
    python -m gemm_matmulplan_broadcast_gb300.profile_one --layer score --a 4096,50257

Inputs are the seeded synthetic operands (A ~ N(0,1), B ~ N(0,0.02), seed 0)
drawn on the host and copied to the device once; each repetition is one
execute of the same plan, timed with CUDA events on the launching stream.
`--a-offset E` places A E elements into its device buffer (a pointer off a
16-byte boundary).  Prints one line per repetition and the median.
"""

from __future__ import annotations

import argparse
import statistics


def _shape(text: str):
    return tuple(int(x) for x in text.split(",") if x)


def layer(args):
    """Forward and backward of one layer plan on N(0,1) inputs (weights N(0,0.02)),
    drawn on the device; a line per repetition: the two times."""
    import torch
    from . import GatedPlan, LayerNormPlan, TokenLogProbsPlan

    rows, cols = _shape(args.a)
    t = getattr(torch, args.dtype)
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s, scale=1.0: (torch.randn(s, generator=gen, device="cuda") * scale).to(t)  # noqa: E731
    stat = lambda: torch.empty(rows, device="cuda")  # noqa: E731
    x = rand(rows, cols)
    if args.layer == "norm":
        plan, w, b, y, dx, m, r = LayerNormPlan(rows, cols, args.dtype), rand(cols), rand(cols), x.clone(), x.clone(), stat(), stat()
        dw, db = w.clone(), b.clone()
        runs = (lambda: plan.forward(x, w, b, y, mean=m, rstd=r),
                lambda: plan.backward(y, x, w, m, r, dx, dw, db))
    elif args.layer == "gate":
        d_in, f = _shape(args.b)
        plan = GatedPlan(rows, d_in, f, args.dtype, trans_w=args.trans_w)
        wg, wu = (rand(*((f, d_in) if args.trans_w else (d_in, f)), scale=0.02) for _ in range(2))
        h, g, u = (rand(rows, f) for _ in range(3))
        dx, dwg, dwu = x.clone(), wg.clone(), wu.clone()
        runs = (lambda: plan.forward(x, wg, wu, h, G=g, U=u),
                lambda: plan.backward(h, x, wg, wu, g, u, dX=dx, dWg=dwg, dWu=dwu))
    else:
        plan, out = TokenLogProbsPlan(rows, cols, args.dtype, args.top), [stat() for _ in range(3)]
        tok = torch.randint(0, cols, (rows,), generator=gen, device="cuda")
        tl = torch.empty(rows, args.top, device="cuda") if args.top else None
        ti = torch.empty(rows, args.top, device="cuda", dtype=torch.int64) if args.top else None
        dz = x.clone()
        runs = (lambda: plan.forward(x, tok, out[0], entropy=out[1], lse=out[2], top_logprob=tl, top_index=ti),
                lambda: plan.backward(x, tok, out[2], out[1], out[0], dz, dentropy=out[1]))
    for i in range(args.reps):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        e[0].record()
        for j, run in enumerate(runs):
            run()
            e[j + 1].record()
        e[2].synchronize()
        print("rep %d: forward %.4f ms, backward %.4f ms" % (i, e[0].elapsed_time(e[1]), e[1].elapsed_time(e[2])))


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--a", required=True, help="A's shape (a layer's rows and columns), comma separated")
    ap.add_argument("--b", help="B's shape (the gated product's d_in and d_hidden), comma separated")
    ap.add_argument("--layer", choices=("norm", "gate", "score"))
    ap.add_argument("--trans-w", action="store_true", help="gate: weights stored [d_hidden, d_in]")
    ap.add_argument("--top", type=int, default=0, help="score: how many alternatives")
    ap.add_argument("--dtype", default="bfloat16")
    ap.add_argument("--reps", type=int, default=3)
    ap.add_argument("--algorithm", default=None)
    ap.add_argument("--variant", type=int, default=None)
    ap.add_argument("--a-offset", type=int, default=0)
    args = ap.parse_args(argv)
    if args.layer:
        return layer(args)
    if not args.b:
        ap.error("--b is required")

    import torch
    from . import Plan, synth

    a_shape, b_shape = _shape(args.a), _shape(args.b)
    a, b = synth.operands(a_shape, b_shape, args.dtype, synth.normal(1.0), synth.normal(0.02), 0)
    if args.a_offset:
        buf = torch.empty(a.numel() + args.a_offset, dtype=a.dtype, device="cuda")
        A = buf[args.a_offset:].view(a.shape)
        A.copy_(a.cuda())
    else:
        A = a.cuda()
    B = b.cuda()
    with Plan(a_shape, b_shape, args.dtype) as p:
        if args.algorithm:
            p.force(args.algorithm)
        if args.variant is not None:
            p.set_tc_variant(args.variant)
        Y = torch.empty(p.output_shape, device="cuda",
                        dtype=synth.TORCH_DTYPES[synth.output_dtype(args.dtype)])
        stream = torch.cuda.current_stream()
        times = []
        for i in range(args.reps):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record(stream)
            p.execute(A, B, Y, stream=stream)
            e1.record(stream)
            e1.synchronize()
            times.append(e0.elapsed_time(e1))
            print("rep %d: %.4f ms (%s)" % (i, times[-1], p.describe()))
        print("median %.4f ms" % statistics.median(times))


if __name__ == "__main__":
    main()
