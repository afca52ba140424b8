"""Plain definitions of the 8-bit serving products for tests: numpy, IEEE fp32
where the definition names fp32, 64 bits elsewhere."""
import numpy as np
import torch

U32, UBF16 = 2.0 ** -24, 2.0 ** -8  # half a step, relative


def smoothed(X: torch.Tensor, smooth: torch.Tensor) -> torch.Tensor:
    """bf16_rn(fl32(X / smooth)) (CPU tensors)."""
    with np.errstate(all="ignore"):
        q = X.float().numpy() / smooth.float().numpy()
    return torch.from_numpy(q).to(torch.bfloat16)


def quantize_tokens(X: torch.Tensor):
    """(codes int8 [R, K], scales fp32 [R], any non-finite) of bf16 X (CPU)."""
    x = X.float().numpy()
    finite = np.isfinite(x)
    amax = np.where(finite, np.abs(x), np.float32(0)).max(axis=1, initial=np.float32(0))
    s = (amax / np.float32(127)).astype(np.float32)
    s[s == 0] = 1
    with np.errstate(all="ignore"):
        q = np.clip(np.rint(x / s[:, None]), -127, 127)
    q[np.isnan(x)] = 0
    return q.astype(np.int8), s, bool((~finite).any())


def sums(xq: np.ndarray, wq: np.ndarray) -> np.ndarray:
    """Exact integer sums: every partial sum of the fp64 product is an integer below 2^53."""
    return (xq.astype(np.float64) @ wq.astype(np.float64).T).astype(np.int64)


def product(xq, xs, wq, ws):
    """(value as the definition rounds it, fp32; the value in 64 bits)."""
    acc = sums(xq, wq)
    w, s = ws.astype(np.float32), xs.astype(np.float32)
    with np.errstate(all="ignore"):
        y = (acc.astype(np.float32) * w[None, :]).astype(np.float32) * s[:, None]
        y64 = acc.astype(np.float64) * w.astype(np.float64)[None, :] * s.astype(np.float64)[:, None]
    return y.astype(np.float32), y64


def check(Y: torch.Tensor, y: np.ndarray, y64: np.ndarray):
    """Bit for bit the definition's value; and within its roundings of the
    64-bit one: three fp32 ones, (1 + u)^3 - 1 <= 3.001 u, and one to bf16.
    Below 2^-126 a type's values are evenly spaced (2^-149 in fp32, 2^-133 in
    bf16) and a rounding is off by at most half of that; of the fp32 ones only
    the last can get there (|sum| w is 0 or at least 2^-24)."""
    got = Y.detach().cpu()
    want = torch.from_numpy(y).to(got.dtype)
    assert torch.equal(got, want), float((got.double() - want.double()).abs().max())
    bound = 3.001 * U32 * np.abs(y64) + 2.0 ** -150
    if got.dtype == torch.bfloat16:
        bound = bound + UBF16 * (np.abs(y64) + bound) + 2.0 ** -134
    assert np.all(np.abs(got.double().numpy() - y64) <= bound)


def grouped(xq, xs, wq, ws, offsets, held: torch.Tensor):
    """Per-expert product into a copy of `held`; rows of no expert keep theirs."""
    y = held.float().numpy().copy()
    y64 = held.double().numpy().copy()
    for e in range(len(offsets) - 1):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            y[lo:hi], y64[lo:hi] = product(xq[lo:hi], xs[lo:hi], wq[e], ws[e])
    return y, y64


def words(codes: np.ndarray) -> torch.Tensor:
    """INT8 codes [..., K] as the packed artifact's words [..., K / 4]."""
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.int32)
