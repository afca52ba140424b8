// w8a8.cu -- the extern "C" boundary of the 8-bit serving products (declared
// in include/wq_int8.h): argument checks and the choice of kernel.
#include <cuda_runtime.h>
#include <stdint.h>

#include "w8a8.h"

using namespace wq;

namespace {

constexpr int64_t kMaxInt32 = (1ll << 31) - 1;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool depth_ok(int64_t d_in) { return d_in >= 32 && d_in % 32 == 0 && d_in <= WQ_INT8_MAX_D_IN; }

// `rows` of activations and outputs; their arrays may be NULL when there are none.
wq_status check_product(const int8_t* Xq, const float* x_scales, int64_t rows, const uint32_t* qweight,
                        const void* scales, int64_t d_out, int64_t d_in, const void* Y, int32_t y_dtype) {
    if (rows < 0 || rows > kMaxInt32 || d_out < 1 || d_out > kMaxInt32 || !depth_ok(d_in)) return WQ_ERR_INVALID_ARG;
    if (y_dtype != WQ_OUT_BF16 && y_dtype != WQ_OUT_FP32) return WQ_ERR_INVALID_ARG;
    if (!qweight || !scales || !aligned(qweight, 16) || !aligned(scales, 2)) return WQ_ERR_INVALID_ARG;
    if (rows > 0 && (!Xq || !x_scales || !Y)) return WQ_ERR_INVALID_ARG;
    if (!aligned(Xq, 16) || !aligned(x_scales, 4) || !aligned(Y, 16)) return WQ_ERR_INVALID_ARG;
    return WQ_OK;
}

wq_status run_product(W8A8Args a, void* stream) {
    int num_sms = 0;
    const wq_status v = device_info(&a.status, &num_sms);
    if (v != WQ_OK) return v;
    if (a.R == 0) return WQ_OK;
    // average rows of an expert that has any
    const int64_t mean = a.R / (a.E < a.R ? a.E : a.R);
    const auto launch = mean <= 64 ? launch_w8a8_stream : launch_w8a8_pair;
    const cudaError_t e = launch(a, num_sms, pdl_enabled(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? WQ_OK : e == cudaErrorNotSupported ? WQ_ERR_UNSUPPORTED : WQ_ERR_CUDA;
}

}  // namespace

extern "C" {

wq_status wq_quantize_tokens(const void* X_bf16, int64_t T, int64_t d_in, const int32_t* rows, int64_t R,
                             const void* smooth_bf16, int8_t* Xq, float* x_scales, void* stream) {
    if (T < 0 || T > kMaxInt32 || R < 0 || R > kMaxInt32 || !depth_ok(d_in)) return WQ_ERR_INVALID_ARG;
    if (!rows && R != T) return WQ_ERR_INVALID_ARG;
    if (R > 0 && (!Xq || !x_scales || (T > 0 && !X_bf16))) return WQ_ERR_INVALID_ARG;
    if (!aligned(X_bf16, 16) || !aligned(Xq, 16) || !aligned(x_scales, 4) || !aligned(rows, 4) ||
        !aligned(smooth_bf16, 2))
        return WQ_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    int num_sms = 0;
    const wq_status v = device_info(&status, &num_sms);
    if (v != WQ_OK) return v;
    if (R == 0) return WQ_OK;
    const cudaError_t e = launch_quantize_tokens(X_bf16, T, d_in, rows, R, smooth_bf16, Xq, x_scales, status,
                                                 pdl_enabled(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

wq_status wq_linear_w8a8(const int8_t* Xq, const float* x_scales, int64_t M, const uint32_t* qweight,
                         const void* scales_fp16, int64_t d_out, int64_t d_in, void* Y, int32_t y_dtype,
                         void* stream) {
    const wq_status v = check_product(Xq, x_scales, M, qweight, scales_fp16, d_out, d_in, Y, y_dtype);
    if (v != WQ_OK) return v;
    W8A8Args a = {};
    a.Xq = Xq;
    a.xs = x_scales;
    a.qweight = qweight;
    a.ws = static_cast<const uint16_t*>(scales_fp16);
    a.Y = Y;
    a.R = (int)M;
    a.N = (int)d_out;
    a.K = (int)d_in;
    a.E = 1;
    a.y_fp32 = y_dtype == WQ_OUT_FP32;
    return run_product(a, stream);
}

wq_status wq_linear_w8a8_grouped(const int8_t* Xq, const float* x_scales, int64_t R, const int32_t* offsets, int64_t E,
                                 const uint32_t* qweight, const void* scales_fp16, int64_t d_out, int64_t d_in,
                                 void* Y, int32_t y_dtype, void* stream) {
    const wq_status v = check_product(Xq, x_scales, R, qweight, scales_fp16, d_out, d_in, Y, y_dtype);
    if (v != WQ_OK) return v;
    if (!offsets || !aligned(offsets, 4) || E < 1) return WQ_ERR_INVALID_ARG;
    if (E > WQ_INT8_MAX_EXPERTS) return WQ_ERR_UNSUPPORTED;
    if (E * d_out > kMaxInt32) return WQ_ERR_INVALID_ARG;
    W8A8Args a = {};
    a.Xq = Xq;
    a.xs = x_scales;
    a.offsets = offsets;
    a.qweight = qweight;
    a.ws = static_cast<const uint16_t*>(scales_fp16);
    a.Y = Y;
    a.R = (int)R;
    a.N = (int)d_out;
    a.K = (int)d_in;
    a.E = (int)E;
    a.y_fp32 = y_dtype == WQ_OUT_FP32;
    return run_product(a, stream);
}

}  // extern "C"
