// tokens.cu -- per-token INT8 codes of bf16 activations (sm_100a).
//
// s = fl32(max |x| / 127) over a row's finite values (1 if 0), q = clamp(
// rint(fl32(x / s)), -127, 127); optionally x is bf16_rn(fl32(x / smooth)) and
// the row is gathered through an index.  Bound by HBM: 2 bytes in, 1 out per
// value, so a row is read once and kept in registers between its maximum and
// its codes.
//
// An IEEE division per value would make the kernel issue-bound (about 10 of
// the ~16 instructions per value that the copy rate leaves).  t = x * fl(1/s)
// is within 1.6e-5 of x / s (|t| <= 127.0001, three roundings of 2^-24), and
// fl32(x / s) within 8e-6, so rint(t) is rint(fl32(x / s)) unless t lies
// within 1e-4 of a half-integer; only there is the division done.  rint is the
// addition of 1.5 * 2^23, whose low byte is the code in two's complement.
#include <stdint.h>

#include "w8a8.h"
#include "wq_device.cuh"

namespace wq {
namespace {

constexpr int kTokThreads = 256;
constexpr float kRint = 12582912.0f;  // 1.5 * 2^23

__device__ __forceinline__ void unpack8(const uint4& v, float f[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// bf16_rn(fl32(x / smooth)) for 8 values
__device__ __forceinline__ uint4 smooth8(const uint4& v, const uint16_t* smooth, int k) {
    float f[8];
    unpack8(v, f);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float s0 = __uint_as_float((uint32_t)__ldg(smooth + k + 2 * i) << 16);
        const float s1 = __uint_as_float((uint32_t)__ldg(smooth + k + 2 * i + 1) << 16);
        o[i] = bf2_bits(__floats2bfloat162_rn(__fdiv_rn(f[2 * i], s0), __fdiv_rn(f[2 * i + 1], s1)));
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

// Largest finite |x| of 8 values.
__device__ __forceinline__ float finite_max8(float m, const uint4& v) {
    float f[8];
    unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (isfinite(f[i])) m = fmaxf(m, fabsf(f[i]));
    return m;
}

__device__ __forceinline__ uint32_t code_exact(float x, float s) {
    if (isnan(x)) return 0u;
    return (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.0f), 127.0f) & 0xffu;
}

__device__ __forceinline__ uint2 codes8_exact(const float f[8], float s) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= code_exact(f[i], s) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

// fast: every value of the row is finite and 1/s is a normal number.
__device__ __forceinline__ uint2 codes8(const uint4& v, float s, float rcp, bool fast) {
    float f[8];
    unpack8(v, f);
    if (fast) {
        uint32_t m[8];
        float far = 0.0f;  // largest distance to the nearest integer
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = f[i] * rcp;
            const float r = __fadd_rn(t, kRint);
            m[i] = __float_as_uint(r);
            far = fmaxf(far, fabsf(t - __fadd_rn(r, -kRint)));
        }
        if (far < 0.4999f) {
            const uint32_t lo = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
            const uint32_t hi = __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410);
            return make_uint2(lo, hi);
        }
    }
    return codes8_exact(f, s);
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

// LANES threads per row (32 ... 256), NV 16-byte pieces of the row per thread
// in registers; NV = 0: rows too long for that are read twice.
template <int LANES, int NV>
__global__ void __launch_bounds__(kTokThreads) quantize_tokens_kernel(const TokenArgs a) {
    constexpr int kRows = kTokThreads / LANES, kWarps = LANES / 32;
    __shared__ float part[kTokThreads / 32];
    __shared__ float part_finite[kTokThreads / 32];
    const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES, warp = threadIdx.x >> 5;
    const int r = (int)blockIdx.x * kRows + sub;
    const int pieces = a.K / 8;
    pdl_launch_dependents();
    pdl_wait_prior();
    bool live = r < a.R;
    int src = live ? r : 0;
    if (live && a.rows) {
        src = __ldg(a.rows + r);
        if (src < 0 || src >= a.T) {
            live = false;
            if (l == 0) raise_flag(a.status, WQ_DEVFLAG_INDEX);
        }
    }
    const uint16_t* x = a.X + (live ? (int64_t)src * a.K : 0);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const auto load = [&](int c) {
        uint4 v = live && c < pieces ? ld_nc_v4(x + 8 * c) : zero;
        if (a.smooth && live && c < pieces) v = smooth8(v, a.smooth, 8 * c);
        return v;
    };

    constexpr int kHold = NV > 0 ? NV : 1;
    uint4 held[kHold];
    __nv_bfloat162 m2 = bits_bf2(0u);
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = l + i * LANES;
            held[i] = live && c < pieces ? ld_nc_v4(x + 8 * c) : zero;
        }
        if (a.smooth && live) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (l + i * LANES < pieces) held[i] = smooth8(held[i], a.smooth, 8 * (l + i * LANES));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) m2 = max8(m2, held[i]);
    } else {
        for (int c = l; c < pieces; c += LANES) m2 = max8(m2, load(c));
    }
    float amax = __bfloat162float(__hmax_nan(m2.x, m2.y));
    // a NaN or infinity as +inf, so that the maximum carries it
    if (!(amax <= 3.4e38f)) amax = __uint_as_float(0x7f800000u);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if constexpr (kWarps > 1) {
        if ((threadIdx.x & 31) == 0) part[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, part[sub * kWarps + w]);
    }
    const bool finite = amax <= 3.4e38f;
    if (__syncthreads_or(!finite)) {  // some row of the block holds NaN or infinities: maximum of the others
        float f = 0.0f;
        if (!finite) {
            if constexpr (NV > 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i) f = finite_max8(f, held[i]);
            } else {
                for (int c = l; c < pieces; c += LANES) f = finite_max8(f, load(c));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, o));
        if ((threadIdx.x & 31) == 0) part_finite[warp] = f;
        __syncthreads();
        if (!finite) {
            amax = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, part_finite[sub * kWarps + w]);
            if (l == 0) raise_flag(a.status, WQ_DEVFLAG_NONFINITE);
        }
    }
    float s = __fdiv_rn(amax, 127.0f);
    if (s == 0.0f) s = 1.0f;
    const float rcp = __frcp_rn(s);
    const bool fast = finite && s >= 7.52316385e-37f;  // 2^-120: 1/s and the products stay normal
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
        for (int c = l; c < pieces; c += LANES) out[c] = codes8(load(c), s, rcp, fast);
    }
}

template <int LANES, int NV>
cudaError_t launch_tokens(const TokenArgs& a, bool pdl, cudaStream_t stream) {
    constexpr int kRows = kTokThreads / LANES;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)a.R + kRows - 1) / kRows));
    cfg.blockDim = dim3(kTokThreads);
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
    return launch_tokens<256, 0>(a, pdl, stream);
}

}  // namespace wq
