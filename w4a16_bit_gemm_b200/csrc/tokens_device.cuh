// tokens_device.cuh -- the arithmetic of per-token INT8 codes (sm_100a only).
//
//   s = fl32(max |x| / 127) over a row's finite values (1 if 0),
//   q = clamp(rint(fl32(x / s)), -127, 127); NaN -> 0, +-Inf -> +-127.
//
// An IEEE division per value would make a kernel issue-bound.  With y =
// fl32(1/s), q0 = fl32(x y), r = fma(-q0, s, x) and q1 = fma(r, y, q0)
// (Markstein's correction) rint(q1) = rint(fl32(x / s)): x and the row maximum
// behind s are bf16, so there are few cases up to a power of two, and
// tests/token_quotient.c goes through all of them.  (A test for values close
// to a half-integer with the division done there was tried first: with 8-bit
// significands exact ties are common, 18.8 instructions per value.)  rint is
// the addition of 1.5 * 2^23, whose low byte is the code in two's complement.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "wq_device.cuh"

namespace wq {

constexpr float kRint = 12582912.0f;  // 1.5 * 2^23

__device__ __forceinline__ void unpack8(const uint4& v, float f[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// 16 bytes of a row, read once.  Not a read-only (.nc) load: with programmatic
// dependent launch the kernel ahead may write them while this one is resident.
__device__ __forceinline__ uint4 load_row16(const uint16_t* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// 8 smoothing scales
__device__ __forceinline__ uint4 load_smooth(const uint16_t* smooth, int k) {
    if ((reinterpret_cast<uintptr_t>(smooth) & 15) == 0) return *reinterpret_cast<const uint4*>(smooth + k);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)smooth[k + 2 * i] | ((uint32_t)smooth[k + 2 * i + 1] << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// bf16_rn(fl32(x / smooth)) for 8 values, with the division.
__device__ __forceinline__ uint4 smooth8_exact(const uint4& v, const uint4& sm) {
    float f[8], s[8];
    unpack8(v, f);
    unpack8(sm, s);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = bf2_bits(__floats2bfloat162_rn(__fdiv_rn(f[2 * i], s[2 * i]), __fdiv_rn(f[2 * i + 1], s[2 * i + 1])));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Largest finite |x| of 8 values; bad becomes 1 if one is not finite.
__device__ __forceinline__ void finite_max8(const uint4& v, float& m, float& bad) {
    float f[8];
    unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (isfinite(f[i]))
            m = fmaxf(m, fabsf(f[i]));
        else
            bad = 1.0f;
    }
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

// The scale of a row whose largest finite |x| is amax.
__device__ __forceinline__ float token_scale(float amax) {
    const float s = __fdiv_rn(amax, 127.0f);
    return s == 0.0f ? 1.0f : s;
}

constexpr float kFastScale = 1.26217745e-29f;  // 2^-96: from here on the products of codes8 stay normal

// fast: these values are finite and s >= kFastScale.
__device__ __forceinline__ uint2 codes8(const uint4& v, float s, float rcp, bool fast) {
    if (!fast) {
        float f[8];
        unpack8(v, f);
        return codes8_exact(f, s);
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const float2 y = make_float2(rcp, rcp), ns = make_float2(-s, -s), one = make_float2(kRint, kRint);
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        const float2 q0 = __fmul2_rn(x, y);
        const float2 q1 = __ffma2_rn(__ffma2_rn(q0, ns, x), y, q0);
        const float2 n = __fadd2_rn(q1, one);
        m[i] = __byte_perm(__float_as_uint(n.x), __float_as_uint(n.y), 0x0040);
    }
    return make_uint2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[2], m[3], 0x5410));
}

}  // namespace wq
