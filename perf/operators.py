"""Measured cases of the 8-bit serving products: quantize_tokens with
linear_w8a8 (one weight matrix) and linear_w8a8_grouped (one weight matrix per
expert, tokens sorted by expert, ragged counts).

    scale   s_t = fl32(max_k |x_tk| / 127), 1 for a row of zeros
    code    q_tk = clamp(rint(fl32(x_tk / s_t)), -127, 127), ties to even
            (with smoothing, x_tk is bf16(x_tk / smooth_k) first)
    product y_tn = s_t w_n sum_k q_tk p_nk, p the weight's 8-bit codes and w_n
            its fp16 scale; the grouped form takes p and w from the expert
            whose range of rows holds t

A case is one projection of one layer.  `source` says what the caller holds:
"bf16" activations (the pass quantizes them, then multiplies; the codes stay
inside the pass) or "codes" (an earlier projection of the same layer quantized
these tokens, as gate and up, or q, k and v share theirs).

With own = False the module uses torch alone; with own = True the package's
entry points.
"""
import math

import torch

own = False

# Shapes are those of the repository's workloads (4096 x 4096 attention
# projections, 11008 x 4096 and 4096 x 11008 MLP projections, 8192 x 8192 and
# 28672 x 8192 prefill layers) and generic expert sizes.
_LISTED = (
    # one user decoding: the smallest call, bound by latency and the weight stream
    dict(name="decode-1-4096x4096", op="linear", source="bf16", tokens=1, d_out=4096, d_in=4096),
    # a full decode batch on the up projection, after gate quantized the tokens
    dict(name="decode-16-11008x4096", op="linear", source="codes", tokens=16, d_out=11008, d_in=4096),
    # a few users on the down projection, smoothed activations, fp32 result
    dict(name="decode-5-4096x11008-smooth", op="linear", source="bf16", tokens=5, d_out=4096, d_in=11008, smooth=True,
         out="fp32"),
    # odd sizes everywhere: ragged tokens, channels and a depth that ends inside a tile
    dict(name="ragged-77-1001x1056", op="linear", source="bf16", tokens=77, d_out=1001, d_in=1056, out="fp32"),
    # one chunk of a chunked prefill
    dict(name="chunk-512-8192x8192", op="linear", source="bf16", tokens=512, d_out=8192, d_in=8192),
    # a long prompt through a narrow projection (shared key/value heads): quantizing weighs as much as multiplying
    dict(name="narrow-8192-1024x8192-smooth", op="linear", source="bf16", tokens=8192, d_out=1024, d_in=8192,
         smooth=True),
    # a long prompt through the widest layer: dense tensor-core work
    dict(name="prefill-8192-28672x8192", op="linear", source="codes", tokens=8192, d_out=28672, d_in=8192),
    # one token sent to 2 of 8 experts: two weight matrices are read
    dict(name="experts8-2-11008x4096", op="grouped", source="bf16", rows=2, top=2, experts=8, d_out=11008, d_in=4096,
         skew=0.0),
    # 16 users, 8 of 64 experts each: most experts see a row or a few
    dict(name="experts64-128-2048x4096", op="grouped", source="codes", rows=128, top=8, experts=64, d_out=2048,
         d_in=4096, skew=0.6),
    # a prompt of 1024 tokens over 64 experts, unevenly loaded, gathered while it is quantized
    dict(name="experts64-8192-2048x4096", op="grouped", source="bf16", rows=8192, top=8, experts=64, d_out=2048,
         d_in=4096, skew=0.6),
    # the down product of a long batch over few experts
    dict(name="experts8-16384-4096x11008", op="grouped", source="codes", rows=16384, top=2, experts=8, d_out=4096,
         d_in=11008, skew=0.3),
    # odd sizes, experts without rows, and padding rows behind the last expert that keep what they held
    dict(name="experts40-61-1409x2080-pad", op="grouped", source="bf16", rows=61, top=3, experts=40, d_out=1409,
         d_in=2080, skew=1.0, pad=11, out="fp32"),
)


def _full(case):
    c = dict(source="bf16", out="bf16", smooth=False, pad=0, skew=0.0, top=1, experts=0)
    c.update(case)
    return c


def listed():
    return [_full(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    out = rng.choice(("bf16", "bf16", "fp32"))
    source = rng.choice(("bf16", "codes"))
    d_in = 32 * _log(rng, 8, 344)
    if rng.random() < 0.5:
        tokens = _log(rng, 1, 8192)
        d_out = _log(rng, 64, 28672)
        return _full(dict(op="linear", source=source, tokens=tokens, d_out=d_out, d_in=d_in, out=out,
                          smooth=source == "bf16" and rng.random() < 0.4))
    rows = _log(rng, 1, 16384)
    experts = _log(rng, 2, 128)
    d_out = _log(rng, 64, 11008)
    skew = rng.choice((0.0, 0.3, 0.6, 1.0))
    pad = rng.choice((0, 0, rng.randint(1, 40)))
    while experts * d_out * d_in > 1.2e9 or experts * max(_counts(rows, experts, skew)) * d_out * d_in > 1.5e12:
        experts, rows = max(2, experts // 2), max(1, rows // 2)
        d_out = max(64, d_out * 3 // 4)
    return _full(dict(op="grouped", source=source, rows=rows, top=rng.choice((1, 2, 4, 8)), experts=experts,
                      d_out=d_out, d_in=d_in, skew=skew, pad=pad, out=out,
                      smooth=source == "bf16" and rng.random() < 0.2))


def _counts(rows, experts, skew):
    """Rows of each expert, largest first: shares (1 + rank)^-skew, rounded so
    that they add up to `rows` (largest remainders first)."""
    share = [(1.0 + i) ** -skew for i in range(experts)]
    unit = rows / sum(share)
    n = [int(s * unit) for s in share]
    order = sorted(range(experts), key=lambda i: (n[i] - share[i] * unit, i))
    for i in order[:rows - sum(n)]:
        n[i] += 1
    return n


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _weight_codes(g, n, k):
    """Per-channel INT8 weights as the package's artifact holds them: N(0, 0.02)
    rows, symmetric codes, fp16 scales."""
    w = torch.randn(n, k, generator=g, device="cuda", dtype=torch.float32)
    w.mul_(0.02)
    s = (w.abs().amax(1) * (1.0 / 127)).half()
    w.div_(s.float()[:, None]).round_().clamp_(-127, 127)
    return w.to(torch.int8), s


def prepare(case, seed):
    c = _full(case)
    g = _generator(seed)
    k, n = c["d_in"], c["d_out"]
    s = {"out": c["out"], "op": c["op"]}
    if c["op"] == "linear":
        codes, scales = _weight_codes(g, n, k)
        tokens = rows = c["tokens"]
    else:
        e, live = c["experts"], c["rows"]
        rows = live + c["pad"]
        tokens = -(-live // c["top"])
        codes, scales = _weight_codes(g, e * n, k)
        codes, scales = codes.view(e, n, k), scales.view(e, n)
        counts = torch.tensor(_counts(live, e, c["skew"]), device="cuda")
        counts = counts[torch.randperm(e, generator=g, device="cuda")]
        s["cap"] = max(_counts(live, e, c["skew"]))  # the longest expert's rows: a plain padded product needs it
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        s["held"] = torch.randn(rows, n, generator=g, device="cuda").to(_dtype(c["out"]))
        if c["source"] == "bf16":
            spread = torch.randperm(rows, generator=g, device="cuda") % tokens
            s["rows"] = spread.to(torch.int32)
    # activations: N(0, 1) with a few channels fifty times as large
    x = torch.randn(tokens if c["source"] == "bf16" else rows, k, generator=g, device="cuda", dtype=torch.float32)
    loud = torch.randperm(k, generator=g, device="cuda")[:max(1, k // 1000)]
    x[:, loud] *= 50.0
    x = x.to(torch.bfloat16)
    s["smooth"] = None
    if c["smooth"]:
        # what a smoothing calibration gives: about the root of each channel's magnitude
        s["smooth"] = (x.float().abs().mean(0) + 0.05).sqrt().to(torch.bfloat16)
    if c["source"] == "codes":
        s["x_codes"], s["x_scales"] = _quantize(x.float())
    else:
        s["x"] = x
    s["codes"], s["scales"] = codes, scales
    return s


def _dtype(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _quantize(x):
    amax = x.abs().amax(1)
    s = amax / torch.full_like(amax, 127.0)
    s = torch.where(s == 0, torch.ones_like(s), s)
    return torch.round(x / s[:, None]).clamp(-127, 127).to(torch.int8), s


def run(s):
    if own:
        return _run_own(s)
    if "x" in s:
        x = s["x"].float()
        if "rows" in s:
            x = x[s["rows"].long()]
        if s["smooth"] is not None:
            x = (x / s["smooth"].float()).to(torch.bfloat16).float()
        q, xs = _quantize(x)
    else:
        q, xs = s["x_codes"], s["x_scales"]
    if s["op"] == "linear":
        y = q.float() @ s["codes"].float().t()
        return (y * s["scales"].float() * xs[:, None]).to(_dtype(s["out"]))
    # each expert's rows padded to the longest one's, one batched product, then back to the rows' places
    off = s["offsets"].long()
    row = torch.arange(q.shape[0], device=q.device)
    at = (off[:-1, None] + torch.arange(s["cap"], device=q.device)).clamp(max=q.shape[0] - 1)
    y = torch.bmm(q.float()[at], s["codes"].float().transpose(1, 2)) * s["scales"].float()[:, None, :]
    e = (torch.searchsorted(off, row, right=True) - 1).clamp(max=off.numel() - 2)
    y = y[e, (row - off[e]).clamp(max=s["cap"] - 1)] * xs[:, None]
    return torch.where((row < off[-1])[:, None], y.to(_dtype(s["out"])), s["held"])


def _run_own(s):
    from w4a16_bit_gemm_b200 import binding as wq
    x = s["x"] if "x" in s else wq.QuantizedTokens(s["x_codes"], s["x_scales"])
    codes = s["codes"]
    if s["op"] == "linear":
        p = wq.PackedLinearW8(codes.view(torch.int32), s["scales"], codes.shape[0], codes.shape[1], codes.shape[1])
        return wq.linear_w8a8(x, p, out_dtype=_dtype(s["out"]), smooth=s["smooth"])
    p = wq.PackedExpertsW8(codes.view(torch.int32), s["scales"])
    # the caller's output: its rows behind the last expert stay as they were
    return wq.linear_w8a8_grouped(x, p, s["offsets"], rows=s.get("rows"), smooth=s["smooth"], out=s["held"])


def work(case):
    c = _full(case)
    k, n = c["d_in"], c["d_out"]
    size = 4 if c["out"] == "fp32" else 2
    if c["op"] == "linear":
        tokens = rows = c["tokens"]
        weights = 1
    else:
        rows, tokens = c["rows"], -(-c["rows"] // c["top"])
        weights = sum(x > 0 for x in _counts(rows, c["experts"], c["skew"]))
    if c["source"] == "bf16":
        read = tokens * k * 2 + (k * 2 if c["smooth"] else 0) + (rows * 4 if c["op"] == "grouped" else 0)
    else:
        read = rows * (k + 4)
    if c["op"] == "grouped":
        read += 4 * (c["experts"] + 1)
    return {"bytes": read + weights * n * (k + 2) + rows * n * size, "flops": 2 * rows * n * k}


def exact(case, seed):
    c = _full(case)
    s = prepare(case, seed)
    if c["source"] == "bf16":
        x = s["x"].double()
        if c["smooth"]:
            # the smoothed activation is a bf16 value by definition (one fp32 division, one rounding)
            x = (x / s["smooth"].double()).float().bfloat16().double()
        if c["op"] == "grouped":
            x = x.index_select(0, s["rows"].long())
        # scale and quotient are fp32 values by definition: the fp64 quotient rounded to fp32 is the fp32 quotient
        xs = (x.abs().max(dim=1).values / 127.0).float().double()
        xs[xs == 0] = 1.0
        q = (x / xs.unsqueeze(1)).float().double().round().clamp(-127.0, 127.0)
    else:
        q, xs = s["x_codes"].double(), s["x_scales"].double()
    if c["op"] == "linear":
        return torch.einsum("tk,nk->tn", q, s["codes"].double()) * xs.unsqueeze(1) * s["scales"].double().unsqueeze(0)
    y = s["held"].double()
    edges = s["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(edges, edges[1:])):
        if hi > lo:
            y[lo:hi] = (q[lo:hi] * xs[lo:hi, None]) @ (s["codes"][e].double() * s["scales"][e].double()[:, None]).t()
    return y
