// tokens.cu -- per-token INT8 codes of bf16 activations (sm_100a).
//
// s = fl32(max |x| / 127) over a row's finite values (1 if 0), q = clamp(
// rint(fl32(x / s)), -127, 127); optionally x is bf16_rn(fl32(x / smooth)) and
// the row is gathered through an index.  Bound by HBM: 2 bytes in, 1 out per
// value, so a row is read once and kept in registers between its maximum and
// its codes.  The arithmetic is in tokens_device.cuh.  Measured: 8192 x 8192
// 34.4 us (5.9 TB/s, 89 % of the copy rate), smoothed 44 us; 16384 x 11008 89 us
// (93 %); one row of 4096 1.6 us.  Issue takes 58 % of the cycles (10
// instructions per value), smoothed 71 % (17): there the issue slots bound it,
// with too few warps to fill the gaps (5 blocks of 256 threads per SM at 47
// registers), not the reciprocals' pipe (38 % busy).
#include <stdint.h>

#include "tokens_device.cuh"
#include "w8a8.h"
#include "wq_device.cuh"

namespace wq {
namespace {

constexpr int block_threads(int lanes) { return lanes > 256 ? lanes : 256; }  // a row's threads, or several rows'

// smooth8_exact through approximate reciprocals; `largest` takes the largest |smooth|.
//
// x and smooth have 8 significant bits, so in the normal range their quotient
// a / b is never halfway between two bf16 values (that would need a = b m with
// m odd and of 9 bits, more than 8 bits) and at least 2^-18 of itself away
// from such a point.  x times the reciprocal is within 2^-22, fl32(x / smooth)
// within 2^-24: both round to the same bf16.  The row's maximum m tells where
// this does not hold: beyond 2^120 or NaN a reciprocal or a product may have
// overflowed (smooth 0, subnormal or NaN among the causes); below 2^-96 values
// outside the normal range could matter, while under a larger maximum they are
// coded 0 anyway; a smooth of 2^126 or more has a reciprocal that is flushed
// to 0.  Such rows are done again with the division.
__device__ __forceinline__ uint4 smooth8(const uint4& v, const uint4& sm, __nv_bfloat162& largest) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w}, d[4] = {sm.x, sm.y, sm.z, sm.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float r0, r1;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(__uint_as_float(d[i] << 16)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(__uint_as_float(d[i] & 0xffff0000u)));
        const float2 t = __fmul2_rn(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)),
                                    make_float2(r0, r1));
        o[i] = bf2_bits(__floats2bfloat162_rn(t.x, t.y));
        largest = __hmax2_nan(largest, __habs2(bits_bf2(d[i])));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Largest |x| of 8 values; NaN if one is NaN.
__device__ __forceinline__ __nv_bfloat162 max8(__nv_bfloat162 m, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2_nan(m, __habs2(bits_bf2(w[i])));
    return m;
}

// Maximum over the threads of a row (kWarps whole warps; `sub` numbers the
// block's rows).  All threads of the block call it.
template <int kWarps>
__device__ __forceinline__ float row_max(float m, float* part, int sub) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (kWarps > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, part[sub * kWarps + w]);
    }
    return m;
}

struct TokenArgs {
    const uint16_t* X;
    const int32_t* rows;
    const uint16_t* smooth;
    int8_t* Xq;
    float* x_scales;
    uint32_t* status;
    int T, R, K;
};

// LANES threads per row (32 ... 1024), NV 16-byte pieces of the row per thread
// in registers; NV = 0: rows too long for that are read twice.
template <int LANES, int NV>
__global__ void __launch_bounds__(block_threads(LANES)) quantize_tokens_kernel(const TokenArgs a) {
    constexpr int kThreads = block_threads(LANES), kRows = kThreads / LANES, kWarps = LANES / 32;
    __shared__ float part[kThreads / 32], part2[kThreads / 32], part3[kThreads / 32];
    const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const int r = (int)blockIdx.x * kRows + sub;
    const int pieces = a.K / 8;
    pdl_launch_dependents();
    pdl_wait_prior();
    bool live = r < a.R;
    int src = live ? r : 0;
    if (live && a.rows) {
        src = a.rows[r];
        if (src < 0 || src >= a.T) {
            live = false;
            if (l == 0) raise_flag(a.status, WQ_DEVFLAG_INDEX);
        }
    }
    const uint16_t* x = a.X + (live ? (int64_t)src * a.K : 0);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool smoothed = a.smooth && live;
    __nv_bfloat162 m2 = bits_bf2(0u), largest = bits_bf2(0u);
    const auto load = [&](int c, bool exact) {
        if (!live || c >= pieces) return zero;
        const uint4 v = load_row16(x + 8 * c);
        if (!smoothed) return v;
        const uint4 sm = load_smooth(a.smooth, 8 * c);
        return exact ? smooth8_exact(v, sm) : smooth8(v, sm, largest);
    };

    constexpr int kHold = NV > 0 ? NV : 1;
    uint4 held[kHold];
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = l + i * LANES;
            held[i] = live && c < pieces ? load_row16(x + 8 * c) : zero;
        }
        if (smoothed) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = l + i * LANES;
                if (c < pieces) held[i] = smooth8(held[i], load_smooth(a.smooth, 8 * c), largest);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) m2 = max8(m2, held[i]);
    } else {
        for (int c = l; c < pieces; c += LANES) m2 = max8(m2, load(c, false));
    }
    float amax = __bfloat162float(__hmax_nan(m2.x, m2.y));
    // NaN, infinities and reciprocals that were flushed to 0 as +inf, so that the maximum carries them
    if (!(amax <= 3.4e38f) || !(__bfloat162float(__hmax_nan(largest.x, largest.y)) < 8.507059e37f))
        amax = __uint_as_float(0x7f800000u);
    amax = row_max<kWarps>(amax, part, sub);
    const bool sure = amax <= 3.4e38f && (!smoothed || (amax >= 1.26217745e-29f && amax <= 1.32922800e36f));
    bool finite = true;
    if (__syncthreads_or(!sure)) {  // rare: some row of the block needs a closer look
        float f = 0.0f, bad = 0.0f;
        if (!sure) {
            if constexpr (NV > 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (smoothed) held[i] = load(l + i * LANES, true);
                    finite_max8(held[i], f, bad);
                }
            } else {
                for (int c = l; c < pieces; c += LANES) finite_max8(load(c, true), f, bad);
            }
        }
        f = row_max<kWarps>(f, part2, sub);
        bad = row_max<kWarps>(bad, part3, sub);
        if (!sure) {
            amax = f;
            finite = bad == 0.0f;
            if (!finite && l == 0) raise_flag(a.status, WQ_DEVFLAG_NONFINITE);
        }
    }
    const float s = token_scale(amax);
    const float rcp = __frcp_rn(s);
    const bool fast = finite && s >= kFastScale;
    if (r >= a.R) return;
    if (l == 0) a.x_scales[r] = s;
    uint2* out = reinterpret_cast<uint2*>(a.Xq + (int64_t)r * a.K);
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = l + i * LANES;
            if (c < pieces) out[c] = codes8(held[i], s, rcp, fast);
        }
    } else {
        for (int c = l; c < pieces; c += LANES) out[c] = codes8(load(c, !sure), s, rcp, fast);
    }
}

template <int LANES, int NV>
cudaError_t launch_tokens(const TokenArgs& a, bool pdl, cudaStream_t stream) {
    constexpr int kRows = block_threads(LANES) / LANES;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)a.R + kRows - 1) / kRows));
    cfg.blockDim = dim3(block_threads(LANES));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, quantize_tokens_kernel<LANES, NV>, a);
}

}  // namespace

cudaError_t launch_quantize_tokens(const void* X, int64_t T, int64_t K, const int32_t* rows, int64_t R,
                                   const void* smooth, int8_t* Xq, float* x_scales, uint32_t* status, bool pdl,
                                   cudaStream_t stream) {
    TokenArgs a = {};
    a.X = static_cast<const uint16_t*>(X);
    a.rows = rows;
    a.smooth = static_cast<const uint16_t*>(smooth);
    a.Xq = Xq;
    a.x_scales = x_scales;
    a.status = status;
    a.T = (int)T;
    a.R = (int)R;
    a.K = (int)K;
    // 4 pieces (64 bytes) per thread hide the load latency; longer rows take
    // more registers before they take a second pass
    const int64_t pieces = K / 8;
    if (pieces <= 32 * 4) return launch_tokens<32, 4>(a, pdl, stream);
    if (pieces <= 64 * 4) return launch_tokens<64, 4>(a, pdl, stream);
    if (pieces <= 128 * 4) return launch_tokens<128, 4>(a, pdl, stream);
    if (pieces <= 256 * 4) return launch_tokens<256, 4>(a, pdl, stream);
    if (pieces <= 256 * 8) return launch_tokens<256, 8>(a, pdl, stream);
    if (pieces <= 512 * 8) return launch_tokens<512, 8>(a, pdl, stream);
    if (pieces <= 1024 * 8) return launch_tokens<1024, 8>(a, pdl, stream);
    return launch_tokens<1024, 0>(a, pdl, stream);
}

}  // namespace wq
