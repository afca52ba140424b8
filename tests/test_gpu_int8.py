"""8-bit serving products on the GPU against their plain definition: codes and
scales bit for bit, products bit for bit (integer sums, three fp32 roundings,
one to bf16) and within those roundings of the 64-bit value."""
import numpy as np
import pytest
import torch

from tests import _int8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_status():
    from w4a16_bit_gemm_b200 import binding
    binding.device_error()
    yield
    st, flags = binding.device_error()
    assert st == binding.WQ_OK, (st, flags)


def _b():
    from w4a16_bit_gemm_b200 import binding
    return binding


def activations(R, K, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g)
    if spread:
        x *= torch.exp(torch.randn(R, 1, generator=g) * 3)
        x[:, torch.randperm(K, generator=g)[:1]] *= 50
    return x.to(torch.bfloat16)


UBF16_FP32 = (1 + ref.UBF16) * (1 + ref.U32) - 1  # an fp32 rounding, then one to bf16


def operands(R, N, K, seed, E=None):
    """Random codes over the whole int8 range, fp16 weight scales, fp32 row scales."""
    rng = np.random.default_rng(seed)
    lead = () if E is None else (E,)
    xq = rng.integers(-128, 128, (R, K), dtype=np.int8)
    wq = rng.integers(-128, 128, lead + (N, K), dtype=np.int8)
    xs = np.exp(rng.normal(-4, 2, R)).astype(np.float32)
    ws = np.exp(rng.normal(-6, 1, lead + (N,))).astype(np.float16)
    return xq, xs, wq, ws


def tokens(xq, xs):
    return _b().QuantizedTokens(torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda())


def dense(wq, ws):
    N, K = wq.shape
    return _b().PackedLinearW8(ref.words(wq).cuda(), torch.from_numpy(ws).cuda(), N, K, K)


def experts(wq, ws):
    return _b().PackedExpertsW8(ref.words(wq).cuda(), torch.from_numpy(ws).cuda())


# ---------------------------------------------------------------------------
# quantize_tokens
# ---------------------------------------------------------------------------

def check_tokens(X, rows=None, smooth=None):
    b = _b()
    x = X if rows is None else X[rows.long()]
    if smooth is not None:
        x = ref.smoothed(x, smooth)
    q, s, bad = ref.quantize_tokens(x)
    got = b.quantize_tokens(X.cuda(), None if rows is None else rows.cuda(), None if smooth is None else smooth.cuda())
    assert np.array_equal(got.scales.cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(got.codes.cpu().numpy(), q)
    st, flags = b.device_error()
    assert flags == (b.WQ_DEVFLAG_NONFINITE if bad else 0)


# every kernel variant: row lengths on both sides of each thread count, register-held and re-read
@pytest.mark.parametrize("K", [32, 96, 256, 1024, 1056, 2048, 2080, 4096, 4128, 8192, 8224, 11008, 16384, 16416, 20000,
                               32768, 32800, 65536, 65568, 131040])
@pytest.mark.parametrize("R", [1, 2, 9])
def test_tokens_match_definition(K, R):
    check_tokens(activations(R, K, K + R))


def test_tokens_many_rows():
    check_tokens(activations(3000, 512, 5))
    check_tokens(activations(700, 4096, 6))


def test_tokens_values_on_and_next_to_ties():
    # amax = 127 * 2^j: x / s is exact, so half-integers are exact ties; the row
    # holds every bf16 value of [2^j / 4, 127 * 2^j]
    bits = np.arange(0x3e80, 0x42ff, dtype=np.uint16)  # 0.25 ... 127.5
    v = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).float()
    v = v[v <= 127]
    rows = []
    for j in (-130, -100, -3, 0, 5, 100):
        x = torch.cat([v, -v, torch.full((32 - (2 * len(v)) % 32,), 127.0)])
        rows.append(x * 2.0 ** j)
    check_tokens(torch.stack(rows).to(torch.bfloat16))
    # other maxima: 127 of them, so that ties and near-ties fall everywhere
    top = torch.from_numpy(np.arange(0x42c0, 0x42ff, dtype=np.uint16).view(np.int16)).view(torch.bfloat16).float()
    n = 32 * (len(v) // 32)
    check_tokens(torch.cat([top[:, None], v[None, :n - 1].clamp(max=90).expand(len(top), -1)], 1).to(torch.bfloat16))


def test_tokens_tiny_huge_and_zero_rows():
    x = torch.randn(8, 288, generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1] *= 2.0 ** -133      # subnormal bf16, subnormal scale
    x[2] *= 2.0 ** -126
    x[3] *= 2.0 ** -118      # on both sides of the scale where the reciprocal is used
    x[4] *= 2.0 ** -112
    x[5] *= 2.0 ** 124
    x[6] = -0.0
    x[7, 1:] = 0
    check_tokens(x.to(torch.bfloat16))


@pytest.mark.parametrize("K", [64, 1056, 4096, 16416, 70016])
def test_tokens_nonfinite(K):
    x = activations(9, K, 8).float()
    x[1, 3] = float("nan")
    x[2, K - 1] = float("inf")
    x[3, 7] = -float("inf")
    x[4] = float("nan")
    x[5] = float("inf")
    x[5, 4] = 3.0
    x[7, ::2] = float("nan")
    check_tokens(x.to(torch.bfloat16))


@pytest.mark.parametrize("K", [32, 1056, 4096, 16416, 40000, 70016])
def test_tokens_smoothed_and_gathered(K):
    X = activations(13, K, 9)
    g = torch.Generator().manual_seed(4)
    smooth = (torch.rand(K, generator=g) * 8 + 0.01).to(torch.bfloat16)
    rows = torch.randint(0, 13, (57,), generator=g).to(torch.int32)
    check_tokens(X, smooth=smooth)
    check_tokens(X, rows=rows)
    check_tokens(X, rows=rows, smooth=smooth)
    # the smoothed values are awq_scale_activations' own
    b = _b()
    a = b.quantize_tokens(b.awq_scale_activations(X.cuda(), smooth.cuda()))
    c = b.quantize_tokens(X.cuda(), smooth=smooth.cuda())
    assert torch.equal(a.codes, c.codes) and torch.equal(a.scales, c.scales)


@pytest.mark.parametrize("R,K", [(2371, 2080), (2400, 4096), (1190, 4128), (1200, 8192), (601, 11008), (700, 16384)])
def test_tokens_smoothed_many_rows(R, K):
    """Many rows at once: ordinary ones, zeros, non-finite and tiny ones,
    gathered ones, smoothing scales of 0 and near the largest bf16."""
    g = torch.Generator().manual_seed(R)
    X = activations(R, K, 17)
    X[5] = 0
    X[R - 1, 3] = float("nan")
    X[R // 2, K - 1] = float("inf")
    X[R // 3] = X[R // 3] * 2.0 ** -110
    smooth = (torch.rand(K, generator=g) * 4 + 0.1).to(torch.bfloat16)
    check_tokens(X, smooth=smooth)
    X[R - 1, 3], X[R // 2, K - 1] = 1.0, 1.0
    rows = torch.randint(0, R, (R,), generator=g).to(torch.int32)
    check_tokens(X, rows=rows, smooth=smooth)
    smooth[7] = 3e38
    check_tokens(X, smooth=smooth)
    smooth[9] = 0.0
    check_tokens(X, smooth=smooth)


# 148 SMs: both sides of the row counts where one more block per SM is needed
@pytest.mark.parametrize("R,K", [(592, 8192), (593, 8192), (740, 8192), (741, 8192), (1185, 4096), (1481, 2080),
                                 (148, 20000), (149, 20000), (296, 11008), (297, 11008)])
def test_tokens_row_counts(R, K):
    X = activations(R, K, R)
    X[R - 1, K - 1] = float("inf")
    X[R // 2] = 0
    smooth = (torch.rand(K, generator=torch.Generator().manual_seed(K)) * 4 + 0.1).to(torch.bfloat16)
    check_tokens(X)
    check_tokens(X, smooth=smooth)
    smooth[K - 1], smooth[K // 2] = 0.0, 3e38
    check_tokens(X, smooth=smooth)


@pytest.mark.parametrize("R,K", [(1, 4096), (3, 11008), (3, 20000), (700, 8192), (2000, 1056)])
def test_tokens_smoothing_scales_off_16_bytes(R, K):
    b = _b()
    X = activations(R, K, 31)
    held = (torch.rand(K + 8, generator=torch.Generator().manual_seed(5)) * 4 + 0.1).to(torch.bfloat16)
    for shift in (1, 4):
        smooth = held[shift:shift + K]
        q, s, _ = ref.quantize_tokens(ref.smoothed(X, smooth))
        got = b.quantize_tokens(X.cuda(), smooth=held.cuda()[shift:shift + K])
        assert np.array_equal(got.codes.cpu().numpy(), q) and np.array_equal(got.scales.cpu().numpy(), s)


def test_tokens_smoothed_many_rows_with_bad_indices():
    b = _b()
    R, K = 3000, 4096
    X = activations(50, K, 18)
    rows = torch.randint(0, 50, (R,), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    rows[::11] = 50
    rows[5::17] = -1
    smooth = torch.full((K,), 2.0)
    smooth[3] = 2.0 ** 127
    smooth = smooth.to(torch.bfloat16)
    got = b.quantize_tokens(X.cuda(), rows.cuda(), smooth.cuda())
    _, flags = b.device_error()
    assert flags == b.WQ_DEVFLAG_INDEX
    q, s, _ = ref.quantize_tokens(ref.smoothed(X[rows.clamp(0, 49).long()], smooth))
    dead = ((rows < 0) | (rows >= 50)).numpy()
    q[dead], s[dead] = 0, 1
    assert np.array_equal(got.codes.cpu().numpy(), q) and np.array_equal(got.scales.cpu().numpy(), s)


def test_tokens_smoothing_at_the_ends_of_the_range():
    K = 256
    X = activations(6, K, 10).float()
    X[1] *= 2.0 ** -120
    X[2] *= 2.0 ** 100
    smooth = torch.ones(K)
    smooth[::7] = 2.0 ** -60
    smooth[1::7] = 2.0 ** 60
    smooth[2::7] = -3.0
    smooth[3::7] = 2.0 ** -133
    smooth[4::7] = 3e38
    check_tokens(X.to(torch.bfloat16), smooth=smooth.to(torch.bfloat16))


@pytest.mark.parametrize("exponent", [-133, -126, -110, -97, -90, -60, 60, 90, 119, 125])
@pytest.mark.parametrize("K", [64, 70016])
def test_tokens_smoothing_scales_of_every_size(K, exponent):
    """Rows and smoothing scales at the borders of what the reciprocal covers."""
    X = activations(5, K, 14).float()
    X[1] *= 2.0 ** -90
    X[2] *= 2.0 ** 90
    X[3] = 0
    smooth = torch.rand(K, generator=torch.Generator().manual_seed(2)) + 1
    check_tokens(X.to(torch.bfloat16), smooth=(smooth * 2.0 ** exponent).to(torch.bfloat16))
    smooth[5] = smooth[5] * 2.0 ** exponent  # one such channel among ordinary ones
    check_tokens(X.to(torch.bfloat16), smooth=smooth.to(torch.bfloat16))
    smooth[6], smooth[7], smooth[8] = 0, float("inf"), float("nan")
    check_tokens(X.to(torch.bfloat16), smooth=smooth.to(torch.bfloat16))


@pytest.mark.parametrize("exponent", [-90, -7, 0, 5, 60])
def test_tokens_smoothing_of_every_pair_of_mantissas(exponent):
    """One value per row: the row's scale tells which bf16 the quotient rounded to."""
    m = 1 + torch.arange(128) / 128
    X = torch.zeros(128, 128, 128)  # value, channel it stands in, channel
    X[:, torch.arange(128), torch.arange(128)] = m[:, None]
    check_tokens(X.view(-1, 128).to(torch.bfloat16), smooth=(m * 2.0 ** exponent).to(torch.bfloat16))


def test_tokens_bad_row_index_is_flagged_and_coded_zero():
    b = _b()
    X = activations(5, 128, 11)
    rows = torch.tensor([0, 5, 4, -1, 2, 1 << 30], dtype=torch.int32)
    got = b.quantize_tokens(X.cuda(), rows.cuda(), torch.ones(128, dtype=torch.bfloat16).cuda())
    st, flags = b.device_error()
    assert st == b.WQ_ERR_INVALID_ARG and flags == b.WQ_DEVFLAG_INDEX
    q, s, _ = ref.quantize_tokens(X[rows.clamp(0, 4).long()])
    dead = ((rows < 0) | (rows >= 5)).numpy()
    q[dead], s[dead] = 0, 1
    assert np.array_equal(got.codes.cpu().numpy(), q) and np.array_equal(got.scales.cpu().numpy(), s)


@pytest.mark.parametrize("T,R,K", [(128, 256, 64), (130, 1001, 1056), (200, 4097, 4096), (300, 601, 4128),
                                   (128, 1500, 8192), (150, 900, 11008), (140, 280, 16384), (130, 300, 16416),
                                   (1024, 8192, 512)])
def test_tokens_gathered_into_several_rows(T, R, K):
    g = torch.Generator().manual_seed(T + R)
    X = activations(T, K, R)
    X[3] = 0
    X[5, 7] = float("nan")
    X[6, K - 1] = -float("inf")
    X[7] = X[7] * 2.0 ** -115
    rows = torch.randint(0, T, (R,), generator=g).to(torch.int32)
    rows[:9] = torch.tensor([3, 5, 6, 7, 0, T - 1, T - 1, 0, 5])
    smooth = (torch.rand(K, generator=g) * 4 + 0.1).to(torch.bfloat16)
    check_tokens(X, rows=rows)
    check_tokens(X, rows=rows, smooth=smooth)
    check_tokens(X, rows=torch.full((R,), 5, dtype=torch.int32))   # all rows one token
    # an index that starts off a 16-byte border
    b = _b()
    q, s, _ = ref.quantize_tokens(X[rows[1:].long()])
    if R - 1 >= 2 * T:
        got = b.quantize_tokens(X.cuda(), rows.cuda()[1:])
        assert np.array_equal(got.codes.cpu().numpy(), q) and np.array_equal(got.scales.cpu().numpy(), s)
        b.device_error()


def test_tokens_gathered_into_several_rows_with_bad_indices():
    b = _b()
    T, R, K = 160, 2000, 544
    X = activations(T, K, 21)
    rows = torch.randint(0, T, (R,), generator=torch.Generator().manual_seed(9)).to(torch.int32)
    rows[::13] = T
    rows[1::29] = -(1 << 31)
    rows[2::31] = (1 << 31) - 1
    got = b.quantize_tokens(X.cuda(), rows.cuda())
    st, flags = b.device_error()
    assert st == b.WQ_ERR_INVALID_ARG and flags == b.WQ_DEVFLAG_INDEX
    q, s, _ = ref.quantize_tokens(X[rows.clamp(0, T - 1).long()])
    dead = ((rows < 0) | (rows >= T)).numpy()
    q[dead], s[dead] = 0, 1
    assert np.array_equal(got.codes.cpu().numpy(), q) and np.array_equal(got.scales.cpu().numpy(), s)


def test_tokens_none_to_gather_from():
    b = _b()
    rows = torch.zeros(3, dtype=torch.int32, device="cuda")
    got = b.quantize_tokens(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), rows)
    _, flags = b.device_error()
    assert flags == b.WQ_DEVFLAG_INDEX and not got.codes.any() and torch.equal(got.scales, torch.ones_like(got.scales))
    none = b.quantize_tokens(torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), rows[:0])
    assert none.codes.shape == (0, 64) and none.scales.shape == (0,)


# ---------------------------------------------------------------------------
# linear_w8a8
# ---------------------------------------------------------------------------

def check_linear(M, N, K, seed=0, dtype=torch.bfloat16):
    xq, xs, wq, ws = operands(M, N, K, seed)
    y, y64 = ref.product(xq, xs, wq, ws)
    ref.check(_b().linear_w8a8(tokens(xq, xs), dense(wq, ws), out_dtype=dtype), y, y64)


@pytest.mark.parametrize("M", [1, 2, 3, 8, 15, 16, 17, 31, 33, 64, 65])
@pytest.mark.parametrize("N,K", [(1, 32), (37, 96), (128, 128), (129, 416), (1000, 1056), (301, 4096)])
def test_linear_few_tokens(M, N, K):
    check_linear(M, N, K, M + N + K, torch.float32 if (M + N) % 2 else torch.bfloat16)


@pytest.mark.parametrize("M,N,K", [(127, 300, 160), (128, 640, 512), (129, 257, 1056), (255, 128, 96), (256, 1000, 288),
                                   (257, 255, 2080), (300, 1001, 1056), (513, 600, 128), (777, 1409, 544),
                                   (1030, 2049, 1024), (2500, 513, 256),
                                   # deep: tiles of 512 channels, whole and ragged ones
                                   (1100, 1000, 8192), (2100, 513, 8224), (700, 2050, 11008),
                                   # deep and narrow: the stream kernel with several token tiles and K split
                                   (65, 200, 4096), (129, 300, 4100 // 32 * 32), (250, 520, 8192), (511, 130, 2080)])
def test_linear_many_tokens(M, N, K):
    check_linear(M, N, K, M, torch.float32 if N % 2 else torch.bfloat16)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (5, 4096, 11008), (16, 11008, 4096), (3, 28672, 256),
                                   (40, 4096, 4096)])
def test_linear_decode_shapes(M, N, K):
    check_linear(M, N, K, 3)


@pytest.mark.parametrize("M", [2, 300])
def test_linear_deepest_sum_does_not_wrap(M):
    K, N = 131040, 130
    xq, wq = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
    wq[1] = 127
    y, y64 = ref.product(xq, np.ones(M, np.float32), wq, np.ones(N, np.float16))
    ref.check(_b().linear_w8a8(tokens(xq, np.ones(M, np.float32)), dense(wq, np.ones(N, np.float16)),
                               out_dtype=torch.float32), y, y64)
    assert y64[0, 0] == 128 * 128 * K


def test_linear_scales_at_the_ends_of_the_range():
    xq, xs, wq, ws = operands(6, 200, 256, 1)
    xs[:] = [3e36, 1e-45, 1e-38, 0.0, float("inf"), float("nan")]
    ws[:4] = [65504, 6e-8, 0.0, 1.0]
    wq[5] = 0
    y, _ = ref.product(xq, xs, wq, ws)
    got = _b().linear_w8a8(tokens(xq, xs), dense(wq, ws), out_dtype=torch.float32).cpu().numpy()
    assert np.array_equal(got, y, equal_nan=True)


def test_linear_whole_path_from_bf16():
    """quantize_w8 weights, bf16 activations with smoothing: the two calls and
    the one call agree with the definition."""
    b = _b()
    W = (torch.randn(333, 1056, generator=torch.Generator().manual_seed(2)) * 0.02).to(torch.bfloat16)
    X = activations(21, 1056, 12, spread=False)
    smooth = (X.float().abs().mean(0) + 0.1).sqrt().to(torch.bfloat16)
    p = b.quantize_w8(W.cuda())
    xq, xs, _ = ref.quantize_tokens(ref.smoothed(X, smooth))
    wq = p.qweight.cpu().view(torch.int8).numpy()
    y, y64 = ref.product(xq, xs, wq, p.scales.cpu().numpy()[:, 0])
    one = b.linear_w8a8(X.cuda(), p, smooth=smooth.cuda(), out_dtype=torch.float32)
    ref.check(one, y, y64)
    two = b.linear_w8a8(b.quantize_tokens(X.cuda(), smooth=smooth.cuda()), p, out_dtype=torch.float32)
    assert torch.equal(one, two)


def test_linear_smoothed_path_approximates_the_product():
    """SmoothQuant from end to end: X / smooth against W diag(smooth), both in 8
    bits, bounded against X W^T; the same without smoothing is worse where a few
    channels are loud."""
    b = _b()
    M, N, K = 40, 300, 1056
    g = torch.Generator().manual_seed(21)
    X = torch.randn(M, K, generator=g)
    X[:, torch.randperm(K, generator=g)[:5]] *= 60
    X = X.to(torch.bfloat16)
    W = (torch.randn(N, K, generator=g) * 0.02).to(torch.bfloat16)
    x64, w64 = X.double().numpy(), W.double().numpy()
    want = x64 @ w64.T
    smooth = (X.float().abs().amax(0) / W.float().abs().amax(0)).sqrt().to(torch.bfloat16)  # alpha = 1/2
    rms = {}
    for name, s in (("smoothed", smooth), ("plain", None)):
        fold = W if s is None else (W.float() * s.float()).to(torch.bfloat16)
        p = b.quantize_w8(fold.cuda())
        y = b.linear_w8a8(X.cuda(), p, smooth=None if s is None else s.cuda(), out_dtype=torch.float32)
        # A code is off by half a step (and the quotient's rounding, 2^-24 of at
        # most 127 steps); smoothing and folding round each value to bf16 once
        # (2^-8 of it; the quotient and the product in fp32 before that, 2^-24).
        d = 1.0 if s is None else s.double().numpy()[None, :]
        rounded = 0.0 if s is None else UBF16_FP32
        xs = b.quantize_tokens(X.cuda(), smooth=None if s is None else s.cuda()).scales.cpu().double().numpy()
        ws = p.scales.cpu().double().numpy()[:, 0]
        half = 0.5 + 127 * 2.0 ** -23
        a, c = np.abs(x64) / d, np.abs(w64) * d
        da, dc = xs[:, None] * half + rounded * a, ws[:, None] * half + rounded * c
        bound = da @ c.T + a @ dc.T + da @ dc.T
        err = np.abs(y.cpu().double().numpy() - want)
        # the sum's own three fp32 roundings, of a value within `bound` of the product's
        assert np.all(err <= bound + 3.001 * ref.U32 * (np.abs(want) + bound))
        rms[name] = float(np.sqrt((err ** 2).mean()))
    assert rms["smoothed"] < rms["plain"], rms


def check_linear_bf16(M, N, K, seed=0, dtype=torch.bfloat16, smooth=False, X=None):
    """bf16 activations in one call: quantized, then multiplied."""
    b = _b()
    X = activations(M, K, seed) if X is None else X
    sm = (torch.rand(K, generator=torch.Generator().manual_seed(seed)) + 0.2).to(torch.bfloat16) if smooth else None
    _, _, wq, ws = operands(1, N, K, seed)
    xq, xs, bad = ref.quantize_tokens(ref.smoothed(X, sm) if smooth else X)
    y, y64 = ref.product(xq, xs, wq, ws)
    got = b.linear_w8a8(X.cuda(), dense(wq, ws), out_dtype=dtype, smooth=sm.cuda() if smooth else None)
    ref.check(got, y, y64)
    _, flags = b.device_error()
    assert flags == (b.WQ_DEVFLAG_NONFINITE if bad else 0)


@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 13, 16, 17, 80])
@pytest.mark.parametrize("N,K", [(1, 32), (130, 96), (128, 128), (300, 288), (1000, 1056), (520, 4096), (2050, 2080)])
def test_linear_from_bf16(M, N, K, smooth):
    check_linear_bf16(M, N, K, M + N + K, torch.float32 if (M + N) % 2 else torch.bfloat16, smooth)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 4096, 11008), (5, 4096, 11008), (16, 11008, 4096),
                                   (2, 28672, 1024), (16, 128, 20480), (9, 300, 40000), (1, 130, 131040)])
def test_linear_from_bf16_decode_shapes(M, N, K):
    check_linear_bf16(M, N, K, 5)
    check_linear_bf16(M, N, K, 6, torch.float32, True)


@pytest.mark.parametrize("M,N,K", [(6, 300, 1056), (16, 4096, 512), (40, 200, 512)])
def test_linear_from_bf16_odd_values(M, N, K):
    x = activations(M, K, 3).float()
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, K - 1] = float("inf")
    x[2, 3] = -float("inf")
    x[3] *= 2.0 ** -126
    x[4] = float("nan")
    x[5, : K // 2] = 0
    check_linear_bf16(M, N, K, X=x.to(torch.bfloat16))


def test_linear_no_tokens():
    b = _b()
    _, _, wq, ws = operands(1, 40, 64, 0)
    x = b.quantize_tokens(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert b.linear_w8a8(x, dense(wq, ws)).shape == (0, 40)
    assert b.linear_w8a8(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), dense(wq, ws)).shape == (0, 40)
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert b.linear_w8a8_grouped(x, experts(wq[None], ws[None]), off).shape == (0, 40)


# ---------------------------------------------------------------------------
# linear_w8a8_grouped
# ---------------------------------------------------------------------------

def check_grouped(counts, N, K, seed=0, dtype=torch.bfloat16, before=0, behind=0):
    E = len(counts)
    R = before + sum(counts) + behind
    offsets = np.concatenate([[0], np.cumsum(counts)]) + before
    xq, xs, wq, ws = operands(R, N, K, seed, E)
    held = torch.randn(R, N, generator=torch.Generator().manual_seed(seed)).to(dtype)
    y, y64 = ref.grouped(xq, xs, wq, ws, offsets, held)
    out = held.cuda()
    got = _b().linear_w8a8_grouped(tokens(xq, xs), experts(wq, ws),
                                   torch.from_numpy(offsets.astype(np.int32)).cuda(), out=out)
    assert got is out
    ref.check(out, y, y64)


@pytest.mark.parametrize("counts", [
    [1], [0, 1], [1, 0, 0], [0, 0, 0], [1] * 40, [16, 17, 15], [0, 33, 0, 64, 1], [100, 0, 3], [5, 250, 1],
    [257, 0, 513, 31], [2000, 1], [0] * 30 + [70] + [0] * 30,
], ids=lambda c: "-".join(map(str, c))[:24])
@pytest.mark.parametrize("N,K", [(70, 96), (257, 1056)])
def test_grouped_counts(counts, N, K):
    check_grouped(counts, N, K, len(counts) + N, torch.float32 if N % 2 else torch.bfloat16)


@pytest.mark.parametrize("E", [2, 191, 192, 193, 400, 1024])
def test_grouped_many_experts(E):
    rng = np.random.default_rng(E)
    check_grouped(rng.integers(0, 4, E).tolist(), 36, 64, E)


def test_grouped_skewed_prompt():
    rng = np.random.default_rng(7)
    check_grouped(rng.multinomial(1500, rng.dirichlet(np.full(24, 0.4))).tolist(), 640, 512, 7)


# more than one wave of tiles: experts with a part of a tile's 256 rows, with
# several tiles and with none, depths on both sides of the ring's length
@pytest.mark.parametrize("K", [32, 1024, 1056, 2304])
@pytest.mark.parametrize("counts", [[70] * 40, [0, 161, 159, 160, 1, 321, 96, 0, 0, 200] * 5, [5000] + [0] * 39,
                                    [3] * 39 + [2900]])
def test_grouped_medium_loads(counts, K):
    check_grouped(counts, 648, K, len(counts) + K, torch.float32 if K % 128 else torch.bfloat16, before=3, behind=5)


@pytest.mark.parametrize("counts", [[255, 256, 257, 511, 512, 513, 0, 1] * 4, [256] * 26, [513, 767, 769, 0] * 5])
def test_grouped_tile_borders(counts):
    """Experts at the borders of a tile's 256 rows, in more than one wave."""
    check_grouped(counts, 648, 160, len(counts), before=1, behind=2)


def test_grouped_from_bf16_chain_at_full_size():
    """Quantizer and loaded experts in a row, many times without a wait between."""
    b = _b()
    E, N, K, R, T = 64, 2048, 4096, 8192, 1024
    g = torch.Generator(device="cuda").manual_seed(11)
    counts = (torch.rand(E, generator=g, device="cuda") ** 2 * 255).long()
    counts[-1] += R - counts.sum()
    assert counts.min() >= 0
    off = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
    rows = (torch.randperm(R, generator=g, device="cuda") % T).to(torch.int32)
    X = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    codes = torch.randint(-127, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    p = b.PackedExpertsW8(codes.view(torch.int32), torch.rand(E, N, generator=g, device="cuda").half())
    y = b.linear_w8a8_grouped(X, p, off, rows=rows)
    torch.cuda.synchronize()
    outs = [torch.empty_like(y) for _ in range(3)]
    for i in range(400):
        b.linear_w8a8_grouped(X, p, off, rows=rows, out=outs[i % 3])
    torch.cuda.synchronize()
    assert b.device_error() == (b.WQ_OK, 0)
    assert all(torch.equal(o, y) for o in outs)
    e = int(counts.argmax())
    lo = int(off[e])
    want = b.linear_w8a8(X[rows[lo:lo + 70].long()], b.PackedLinearW8(p.qweight[e], p.scales[e], N, K, K))
    assert torch.equal(y[lo:lo + 70], want)


def test_grouped_leaves_other_rows_as_they_were():
    check_grouped([3, 0, 20], 130, 160, 1, before=7, behind=9)
    check_grouped([300, 280], 130, 160, 2, torch.float32, before=1, behind=300)
    check_grouped([0, 0], 130, 160, 3, before=4, behind=4)


@pytest.mark.parametrize("offsets", [[0, 5, 3, 8], [-4, 2, 9, 10], [0, 4, 40, 50], [9, 2, 1, 0], [50, 60, 70, 80],
                                     [-9, -8, -7, -6], [0, 0, 10, 2]])
def test_grouped_bad_offsets_are_flagged_and_stay_in_bounds(offsets):
    b = _b()
    R, N, K = 10, 140, 64
    xq, xs, wq, ws = operands(R, N, K, 3, 3)
    held = torch.randn(R, N, generator=torch.Generator().manual_seed(1))
    taken = np.maximum.accumulate(np.clip(offsets, 0, R))
    y, y64 = ref.grouped(xq, xs, wq, ws, taken, held)
    got = b.linear_w8a8_grouped(tokens(xq, xs), experts(wq, ws), torch.tensor(offsets, dtype=torch.int32).cuda(),
                                out=held.cuda())
    st, flags = b.device_error()
    assert st == b.WQ_ERR_INVALID_ARG and flags == b.WQ_DEVFLAG_INDEX
    ref.check(got, y, y64)


def check_grouped_bf16(counts, N, K, T, seed=0, dtype=torch.bfloat16, smooth=False, behind=0, bad_rows=False):
    b = _b()
    E, R = len(counts), sum(counts) + behind
    g = torch.Generator().manual_seed(seed)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    X = activations(T, K, seed)
    rows = torch.randint(0, T, (R,), generator=g).to(torch.int32)
    dead = torch.zeros(R, dtype=torch.bool)
    if bad_rows:
        rows[1::5], dead[1::5] = T, True
        rows[2::7], dead[2::7] = -3, True
    sm = (torch.rand(K, generator=g) + 0.2).to(torch.bfloat16) if smooth else None
    _, _, wq, ws = operands(1, N, K, seed, E)
    x = X[rows.clamp(0, T - 1).long()]
    xq, xs, _ = ref.quantize_tokens(ref.smoothed(x, sm) if smooth else x)
    xq[dead.numpy()], xs[dead.numpy()] = 0, 1
    held = torch.randn(R, N, generator=g).to(dtype)
    y, y64 = ref.grouped(xq, xs, wq, ws, offsets, held)
    out = b.linear_w8a8_grouped(X.cuda(), experts(wq, ws), torch.from_numpy(offsets.astype(np.int32)).cuda(),
                                out=held.cuda(), rows=rows.cuda(), smooth=sm.cuda() if smooth else None)
    ref.check(out, y, y64)
    _, flags = b.device_error()
    assert flags == (b.WQ_DEVFLAG_INDEX if bad_rows else 0)


@pytest.mark.parametrize("counts", [[1, 1], [0, 2, 0], [8], [9, 0, 1], [16, 0, 3], [17, 2], [40], [0, 0, 5, 1, 1],
                                    [1] * 20, [3] * 60, [200, 30]], ids=lambda c: "-".join(map(str, c))[:24])
@pytest.mark.parametrize("N,K", [(70, 96), (257, 1056), (520, 2048)])
def test_grouped_from_bf16(counts, N, K):
    check_grouped_bf16(counts, N, K, 7, len(counts) + N)
    check_grouped_bf16(counts, N, K, 50, len(counts) + K, torch.float32, True, behind=3)


def test_grouped_from_bf16_one_user():
    check_grouped_bf16([0, 1, 0, 0, 0, 1, 0, 0], 11008, 512, 1, 1)
    check_grouped_bf16([0, 1, 0, 0, 0, 1, 0, 0], 2048, 4096, 1, 2, smooth=True)


@pytest.mark.parametrize("counts", [[5, 0, 6], [100, 120]])
def test_grouped_from_bf16_bad_rows(counts):
    check_grouped_bf16(counts, 200, 288, 6, 3, torch.float32, bad_rows=True)


def test_grouped_equals_dense_per_expert():
    b = _b()
    W = (torch.randn(3, 200, 288, generator=torch.Generator().manual_seed(5)) * 0.02).to(torch.bfloat16).cuda()
    X = activations(50, 288, 13).cuda()
    p = b.quantize_w8_experts(W)
    off = torch.tensor([0, 12, 12, 50], dtype=torch.int32, device="cuda")
    y = b.linear_w8a8_grouped(X, p, off, out_dtype=torch.float32)
    for e in (0, 2):
        lo, hi = int(off[e]), int(off[e + 1])
        assert torch.equal(y[lo:hi], b.linear_w8a8(X[lo:hi].contiguous(), b.quantize_w8(W[e]), out_dtype=torch.float32))


# ---------------------------------------------------------------------------
# Offsets beyond 32 bits: activations, codes, weights and outputs of more than
# 2^31 elements, checked on rows at both ends and around the border
# ---------------------------------------------------------------------------

def _codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def test_more_than_2_31_activations():
    b = _b()
    R, K, N = 266_000, 8192, 130
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(R, K, generator=g, device="cuda", dtype=torch.bfloat16)
    x = b.quantize_tokens(X)
    at = torch.tensor([0, 1, 131071, 131072, 262143, 262144, R - 2, R - 1], device="cuda")
    q, s, _ = ref.quantize_tokens(X[at].cpu())
    assert np.array_equal(x.codes[at].cpu().numpy(), q) and np.array_equal(x.scales[at].cpu().numpy(), s)
    del X
    wq, ws = _codes(g, N, K), torch.rand(N, generator=g, device="cuda").half()
    Y = b.linear_w8a8(x, b.PackedLinearW8(wq.view(torch.int32), ws, N, K, K), out_dtype=torch.float32)
    y, y64 = ref.product(q, s, wq.cpu().numpy(), ws.cpu().numpy())
    ref.check(Y[at], y, y64)


def test_more_than_2_31_outputs():
    b = _b()
    M, N, K = 76_000, 28672, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    xq, xs = _codes(g, M, K), torch.rand(M, generator=g, device="cuda")
    wq, ws = _codes(g, N, K), torch.rand(N, generator=g, device="cuda").half()
    p = b.PackedLinearW8(wq.view(torch.int32), ws, N, K, K)
    at = torch.tensor([0, 37449, 74898, 74899, M - 1], device="cuda")
    y, y64 = ref.product(xq[at].cpu().numpy(), xs[at].cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy())
    ref.check(b.linear_w8a8(b.QuantizedTokens(xq, xs), p)[at], y, y64)
    # a few rows per expert: the stream kernel's stores
    pe = b.PackedExpertsW8(wq.view(torch.int32).expand(2, N, K // 4).contiguous(), ws.expand(2, N).contiguous())
    off = torch.tensor([M - 40, M - 20, M], dtype=torch.int32, device="cuda")
    held = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    got = b.linear_w8a8_grouped(b.QuantizedTokens(xq, xs), pe, off, out=held)
    ref.check(got[at[-1:]], y[-1:], y64[-1:])
    assert not got[:M - 40].any()


@pytest.mark.parametrize("rows", [3, 200])
def test_more_than_2_31_weights(rows):
    b = _b()
    E, N, K = 50, 11008, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    wq, ws = _codes(g, E, N, K), torch.rand(E, N, generator=g, device="cuda").half()
    xq, xs = _codes(g, 2 * rows, K), torch.rand(2 * rows, generator=g, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[48:] = rows        # expert 47 (its weights straddle 2^31 bytes) and the last one
    off[E:] = 2 * rows
    got = b.linear_w8a8_grouped(b.QuantizedTokens(xq, xs), b.PackedExpertsW8(wq.view(torch.int32), ws), off)
    for e, lo in ((47, 0), (E - 1, rows)):
        y, y64 = ref.product(xq[lo:lo + rows].cpu().numpy(), xs[lo:lo + rows].cpu().numpy(), wq[e].cpu().numpy(),
                             ws[e].cpu().numpy())
        ref.check(got[lo:lo + rows], y, y64)


# ---------------------------------------------------------------------------
# Used together, streams, graphs
# ---------------------------------------------------------------------------

def expert_layer(b, X, up, down, rows, offsets, smooth):
    """Tokens to their experts: up product, relu squared, down product."""
    h = b.linear_w8a8_grouped(X, up, offsets, rows=rows, smooth=smooth)
    h = torch.relu(h).square()
    return b.linear_w8a8_grouped(h, down, offsets, out_dtype=torch.float32)


def expert_layer_case(seed=0, T=37, top=2, E=6, d=256, f=416):
    b = _b()
    g = torch.Generator().manual_seed(seed)
    up = b.quantize_w8_experts((torch.randn(E, f, d, generator=g) * 0.05).to(torch.bfloat16).cuda())
    down = b.quantize_w8_experts((torch.randn(E, d, f, generator=g) * 0.05).to(torch.bfloat16).cuda())
    X = torch.randn(T, d, generator=g).to(torch.bfloat16)
    choice = torch.stack([torch.randperm(E, generator=g)[:top] for _ in range(T)])
    order = torch.argsort(choice.flatten(), stable=True)
    rows = (order // top).to(torch.int32)
    offsets = torch.nn.functional.pad(torch.bincount(choice.flatten(), minlength=E).cumsum(0), (1, 0)).to(torch.int32)
    smooth = (torch.rand(d, generator=g) + 0.5).to(torch.bfloat16)
    return X, up, down, rows, offsets, smooth


def expert_layer_ref(X, up, down, rows, offsets, smooth):
    wq = [p.qweight.cpu().view(torch.int8).numpy() for p in (up, down)]
    ws = [p.scales.cpu().numpy() for p in (up, down)]
    xq, xs, _ = ref.quantize_tokens(ref.smoothed(X[rows.long()], smooth))
    held = torch.zeros(len(rows), wq[0].shape[1])
    h, _ = ref.grouped(xq, xs, wq[0], ws[0], offsets.tolist(), held)
    h = torch.relu(torch.from_numpy(h).to(torch.bfloat16)).square()
    xq, xs, _ = ref.quantize_tokens(h)
    return ref.grouped(xq, xs, wq[1], ws[1], offsets.tolist(), torch.zeros(len(rows), wq[1].shape[1]))


def test_expert_layer_end_to_end():
    b = _b()
    for seed, T, top, E in ((0, 37, 2, 6), (1, 1, 2, 8), (2, 300, 4, 5)):
        X, up, down, rows, offsets, smooth = expert_layer_case(seed, T, top, E)
        y, y64 = expert_layer_ref(X, up, down, rows, offsets, smooth)
        ref.check(expert_layer(b, X.cuda(), up, down, rows.cuda(), offsets.cuda(), smooth.cuda()), y, y64)


def test_expert_layer_captured_and_replayed_on_new_inputs():
    b = _b()
    X, up, down, rows, offsets, smooth = expert_layer_case(3)
    buf = [t.cuda() for t in (X, rows, offsets, smooth)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(2):
            expert_layer(b, buf[0], up, down, buf[1], buf[2], buf[3])
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = expert_layer(b, buf[0], up, down, buf[1], buf[2], buf[3])
    for seed in (4, 5):
        X2, _, _, rows2, offsets2, smooth2 = expert_layer_case(seed)
        for dst, src in zip(buf, (X2, rows2, offsets2, smooth2)):
            dst.copy_(src)
        graph.replay()
        y, y64 = expert_layer_ref(X2, up, down, rows2, offsets2, smooth2)
        ref.check(out, y, y64)


def test_back_to_back_launches_keep_their_order():
    """A chain of dependent layers, many times over: each kernel may start
    before the one ahead of it ends, and must not read or write too early."""
    b = _b()
    g = torch.Generator().manual_seed(6)
    p = b.quantize_w8((torch.randn(512, 512, generator=g) * 0.05).to(torch.bfloat16).cuda())
    for M in (1, 20, 300):
        x = torch.randn(M, 512, generator=g).to(torch.bfloat16).cuda()
        buf = [torch.empty_like(x) for _ in range(2)]
        first = None
        for _ in range(20):
            cur = x
            for i in range(12):
                cur = b.linear_w8a8(cur, p, out=buf[i % 2])
            first = cur.clone() if first is None else first
            assert torch.equal(cur, first)
        cur = x
        for i in range(12):
            torch.cuda.synchronize()
            cur = b.linear_w8a8(cur, p).clone()
        assert torch.equal(cur, first)


@pytest.mark.parametrize("M,N,K", [(70, 512, 512), (300, 2000, 1056), (2100, 1000, 1024), (1100, 600, 8192)])
def test_many_rows_from_bf16_back_to_back(M, N, K):
    """Quantizer and SM-pair product in turn, the buffers of one call freed for
    the next: dense and by expert."""
    b = _b()
    _, _, wq, ws = operands(1, N, K, 3, 4)
    X = activations(M, K, 4)
    p, pe = dense(wq[1], ws[1]), experts(wq, ws)
    off = [0, M // 2, M // 2, M - 5, M]
    xq, xs, _ = ref.quantize_tokens(X)
    X, offsets = X.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda")
    held = torch.zeros(M, N)
    for call, want in ((lambda: b.linear_w8a8(X, p, out_dtype=torch.float32), ref.product(xq, xs, wq[1], ws[1])),
                       (lambda: b.linear_w8a8_grouped(X, pe, offsets, out_dtype=torch.float32),
                        ref.grouped(xq, xs, wq, ws, off, held))):
        outs = [call() for _ in range(12)]
        ref.check(outs[0], *want)
        assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_mixed_with_the_other_linear_layers():
    """Kernels that start early beside each other and share tensor memory: 4-bit
    and 8-bit layers of every path in one stream, many times over."""
    b = _b()
    g = torch.Generator().manual_seed(8)
    W = (torch.randn(2048, 2048, generator=g) * 0.03).to(torch.bfloat16).cuda()
    p4, p8 = b.quantize_rtn(W, 128, True), b.quantize_w8(W)
    for M in (1, 2, 8, 16, 40, 200):
        x = torch.randn(M, 2048, generator=g).to(torch.bfloat16).cuda()
        first = None
        for _ in range(15):
            cur = x
            for _ in range(3):
                cur = b.linear_w8a8(cur, p8)
                cur = b.linear_w4a16(cur, p4)
                cur = b.linear_w8a8(b.quantize_tokens(cur), p8)
                cur = b.linear_w8a16(cur, p8)
            first = cur.clone() if first is None else first
            assert torch.equal(cur, first)


def test_two_streams_at_once():
    b = _b()
    cases = []
    for i in range(2):
        xq, xs, wq, ws = operands(9 + 200 * i, 700, 1056, i)
        cases.append((tokens(xq, xs), dense(wq, ws), ref.product(xq, xs, wq, ws)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            outs[i].append(b.linear_w8a8(cases[i][0], cases[i][1], out_dtype=torch.float32, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            ref.check(o, *cases[i][2])


def test_binding_refuses():
    b = _b()
    xq, xs, wq, ws = operands(4, 64, 128, 0)
    x, p, pe = tokens(xq, xs), dense(wq, ws), experts(wq[None], ws[None])
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    X = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    ok = torch.empty(4, 64, dtype=torch.bfloat16, device="cuda")
    per_group = b.quantize_w8(torch.randn(64, 128, device="cuda").to(torch.bfloat16), 32)
    bad = [
        lambda: b.linear_w8a8(x, per_group),
        lambda: b.linear_w8a8(x, b.PackedLinearW8(p.qweight[:63], p.scales, 64, 128, 128)),
        lambda: b.linear_w8a8(x, b.PackedLinearW8(p.qweight, p.scales.float(), 64, 128, 128)),
        lambda: b.linear_w8a8(x, b.PackedLinearW8(p.qweight, p.scales[:60], 64, 128, 128)),
        lambda: b.linear_w8a8(x, b.PackedLinearW8(p.qweight, p.scales.cpu(), 64, 128, 128)),
        lambda: b.linear_w8a8_grouped(x, b.PackedExpertsW8(pe.qweight, pe.scales.float()), off),
        lambda: b.linear_w8a8(X.float(), p),
        lambda: b.linear_w8a8(X[:, :96].contiguous(), p),
        lambda: b.linear_w8a8(X.t().contiguous().t(), p),
        lambda: b.linear_w8a8(x, p, smooth=torch.ones(128, dtype=torch.bfloat16, device="cuda")),
        lambda: b.linear_w8a8(X, p, smooth=torch.ones(64, dtype=torch.bfloat16, device="cuda")),
        lambda: b.linear_w8a8(x, p, out_dtype=torch.float16),
        lambda: b.linear_w8a8(x, p, out=ok, out_dtype=torch.float32),
        lambda: b.linear_w8a8(x, p, out=ok[:3]),
        lambda: b.linear_w8a8(x, p, out=ok.half()),
        lambda: b.linear_w8a8(b.QuantizedTokens(x.codes, x.scales[:3]), p),
        lambda: b.linear_w8a8(b.QuantizedTokens(x.codes.int(), x.scales), p),
        lambda: b.linear_w8a8_grouped(x, pe, off.long()),
        lambda: b.linear_w8a8_grouped(x, pe, off[:1]),
        lambda: b.linear_w8a8_grouped(x, pe, off.cpu()),
        lambda: b.linear_w8a8_grouped(x, pe, off, rows=off),
        lambda: b.linear_w8a8_grouped(X, pe, off, rows=off.long()),
        lambda: b.quantize_tokens(X, out=b.QuantizedTokens(x.codes[:2], x.scales)),
        lambda: b.quantize_tokens(X, rows=off.view(2, 1)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------------------
# Weights written on the stream shortly before
# ---------------------------------------------------------------------------

_WRITE_LATE = r'''
extern "C" __global__ void write_late(int* words, int value, int n) {
    // lets the next kernel start at once, then writes after about 100 us
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long t0 = clock64();
    while (clock64() - t0 < 200000) {}
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) words[i] = value;
}
'''


@pytest.mark.parametrize("between", ["quantizer", "product", "w4a16"])
@pytest.mark.parametrize("M", [1, 20, 200])
def test_weights_written_two_kernels_ahead(M, between):
    """A kernel that starts its successors early writes the weights; behind it
    come the quantizer, a product with other weights or a 4-bit layer, all of
    which do the same, then the product."""
    b = _b()
    N, K = 600, 2048
    write = torch.cuda._compile_kernel(_WRITE_LATE, "write_late")
    _, _, other, ws = operands(1, N, K, 5)
    held = torch.zeros(N, K // 4, dtype=torch.int32, device="cuda")
    p, q = b.PackedLinearW8(held, torch.from_numpy(ws).cuda(), N, K, K), dense(other, ws)
    X = activations(M, K, 6)
    xq, xs, _ = ref.quantize_tokens(X)
    X, x = X.cuda(), tokens(xq, xs)
    out = torch.empty(M, N, dtype=torch.float32, device="cuda")
    p4 = b.quantize_rtn(torch.randn(N, K, device="cuda").to(torch.bfloat16))
    b.linear_w8a8(X, q, out=out)  # the kernels are loaded
    b.linear_w4a16(X, p4)
    torch.cuda.synchronize()
    for code in (1, 2, 3):
        write(grid=(64, 1, 1), block=(256, 1, 1), args=[held, code * 0x01010101, held.numel()])
        if between == "product":
            b.linear_w8a8(x, q, out=out)
        elif between == "w4a16":
            b.linear_w4a16(X, p4)
        y = b.linear_w8a8(X if between == "quantizer" else x, p, out_dtype=torch.float32)
        torch.cuda.synchronize()
        ref.check(y, *ref.product(xq, xs, np.full((N, K), code, np.int8), ws))


def test_weights_quantized_just_ahead():
    """New weights into the same buffer, quantizer and product, no wait of the host between."""
    b = _b()
    N, K = 520, 2080
    g = torch.Generator().manual_seed(12)
    X = activations(9, K, 2)
    xq, xs, _ = ref.quantize_tokens(X)
    Ws = [(torch.randn(N, K, generator=g) * 0.02).to(torch.bfloat16) for _ in range(4)]
    X, dev = X.cuda(), [W.cuda() for W in Ws]
    p = b.quantize_w8(dev[0])
    torch.cuda.synchronize()
    got = []
    for W in dev:
        b.quantize_w8(W, out=p)
        got.append(b.linear_w8a8(X, p, out_dtype=torch.float32))
    torch.cuda.synchronize()
    for W, y in zip(dev, got):
        q = b.quantize_w8(W)
        ref.check(y, *ref.product(xq, xs, q.qweight.cpu().view(torch.int8).numpy(), q.scales.cpu().numpy()[:, 0]))
