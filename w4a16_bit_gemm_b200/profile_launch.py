"""A few launches of one libwq operation on one seeded workload, for profilers.

    python -m w4a16_bit_gemm_b200.profile_launch linear --N 4096 --K 4096 --M 1
    python -m w4a16_bit_gemm_b200.profile_launch quantize --N 4096 --K 4096
    python -m w4a16_bit_gemm_b200.profile_launch dequantize --N 4096 --K 4096
    python -m w4a16_bit_gemm_b200.profile_launch gemm --N 8192 --K 8192 --M 2048
    python -m w4a16_bit_gemm_b200.profile_launch linear_w8 --N 4096 --K 4096 --M 1
    python -m w4a16_bit_gemm_b200.profile_launch linear_w8a8 --N 4096 --K 4096 --M 1
    python -m w4a16_bit_gemm_b200.profile_launch grouped_w8a8 --experts 64 --N 2048 --K 4096 --M 128
    python -m w4a16_bit_gemm_b200.profile_launch tokens --M 8192 --K 8192

Each run quantizes one N(0, 0.02) weight matrix (group 128, asymmetric unless
--sym; linear_w8: symmetric INT8 per channel unless --g is given; the W8A8
operations: per channel, grouped_w8a8 with M rows dealt evenly to --experts
matrices, tokens with the M x K activations alone), keeps
--copies packed copies so that consecutive launches read different memory
(copies x artifact bytes > L2 at the default sizes), and issues --iters
launches of the operation eagerly on the current stream, then
checks the device status.  Under `ncu -k regex:<kernel> -s <skip> -c 1` one of
the later launches is captured; the launch sequence and the inputs are the
same as those of the benchmark's sweep of that shape.
"""
from __future__ import annotations

import argparse
import sys

import torch


def run_w8a8(args, b, syn) -> int:
    seed = 0x5EED0000 + 2
    X = [syn.activations(args.M, args.K, seed, 77 + i, "cuda") for i in range(args.copies)]
    smooth = (X[0].float().abs().mean(0) + 0.05).sqrt().to(torch.bfloat16) if args.smooth else None
    if args.op == "tokens":
        out = b.quantize_tokens(X[0])
        calls = [lambda i=i: b.quantize_tokens(X[i], smooth=smooth, out=out) for i in range(args.copies)]
    else:
        E = args.experts if args.op == "grouped_w8a8" else 1
        W = syn.weight(E * args.N, args.K, 0.02, seed, 0, "cuda").view(E, args.N, args.K)
        p0 = b.quantize_w8_experts(W)
        packs = [b.PackedExpertsW8(p0.qweight.clone(), p0.scales.clone()) for _ in range(args.copies)]
        x = [b.quantize_tokens(t) for t in X]
        Y = torch.empty(args.M, args.N, dtype=torch.bfloat16, device="cuda")
        if args.op == "grouped_w8a8":
            offsets = torch.linspace(0, args.M, E + 1).round().to(torch.int32).cuda()
            calls = [lambda i=i: b.linear_w8a8_grouped(x[i], packs[i], offsets, out=Y) for i in range(args.copies)]
        else:
            dense = [b.PackedLinearW8(p.qweight[0], p.scales[0], args.N, args.K, args.K) for p in packs]
            calls = [lambda i=i: b.linear_w8a8(x[i], dense[i], out=Y) for i in range(args.copies)]
    for i in range(args.iters):
        calls[i % args.copies]()
    torch.cuda.synchronize()
    st, flags = b.device_error()
    print(f"{args.op} N={args.N} K={args.K} M={args.M}: {args.iters} launches, status {st} flags {flags}")
    return 0 if st == b.WQ_OK else 1


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("op", choices=["linear", "quantize", "dequantize", "gemm", "linear_w8", "linear_w8a8", "grouped_w8a8", "tokens"])
    ap.add_argument("--N", type=int, default=4096)
    ap.add_argument("--K", type=int, default=4096)
    ap.add_argument("--M", type=int, default=1)
    ap.add_argument("--g", type=int, default=None, help="group size (default 128; per-channel for linear_w8)")
    ap.add_argument("--sym", action="store_true")
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--smooth", action="store_true", help="tokens: divide by smoothing scales on the way")
    ap.add_argument("--copies", type=int, default=8)
    ap.add_argument("--iters", type=int, default=16)
    args = ap.parse_args(argv)

    from w4a16_bit_gemm_b200 import binding as b
    from w4a16_bit_gemm_b200 import synthetic as syn

    if args.op in ("linear_w8a8", "grouped_w8a8", "tokens"):
        return run_w8a8(args, b, syn)
    W = syn.weight(args.N, args.K, 0.02, 0x5EED0000 + 2, 0, "cuda")
    if args.op == "linear_w8":
        p8 = b.quantize_w8(W, args.g)
        packs = [b.PackedLinearW8(p8.qweight.clone(), p8.scales.clone(), p8.d_out, p8.d_in, p8.group_size)
                 for _ in range(args.copies)]
    else:
        g = args.g or 128
        p0 = b.quantize_rtn(W, g, args.sym)
        packs = [b.PackedLinear(p0.qweight.clone(), p0.scales.clone(), None if p0.zeros is None else p0.zeros.clone(),
                                args.N, args.K, g, args.sym) for _ in range(args.copies)]
    X = syn.activations(args.M, args.K, 0x5EED0000 + 2, 77, "cuda")
    Y = torch.empty(args.M, args.N, dtype=torch.bfloat16, device="cuda")
    Wh = torch.empty(args.N, args.K, dtype=torch.bfloat16, device="cuda")
    for i in range(args.iters):
        p = packs[i % args.copies]
        if args.op in ("linear", "gemm"):
            b.linear_w4a16(X, p, out=Y)
        elif args.op == "linear_w8":
            b.linear_w8a16(X, p, out=Y)
        elif args.op == "quantize":
            b.quantize_rtn(W, args.g or 128, args.sym, out=p)
        else:
            b.dequantize(p, out=Wh)
    torch.cuda.synchronize()
    st, flags = b.device_error()
    print(f"{args.op} N={args.N} K={args.K} M={args.M}: {args.iters} launches, status {st} flags {flags}")
    return 0 if st == b.WQ_OK else 1


if __name__ == "__main__":
    sys.exit(main())
