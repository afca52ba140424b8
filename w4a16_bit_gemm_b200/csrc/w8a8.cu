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

// `rows` of outputs; arrays that belong to them may be NULL when there are none.
wq_status check_product(int64_t rows, const uint32_t* qweight, const void* scales, int64_t d_out, int64_t d_in,
                        const void* Y, int32_t y_dtype) {
    if (rows < 0 || rows > kMaxInt32 || d_out < 1 || d_out > kMaxInt32 || !depth_ok(d_in)) return WQ_ERR_INVALID_ARG;
    if (y_dtype != WQ_OUT_BF16 && y_dtype != WQ_OUT_FP32) return WQ_ERR_INVALID_ARG;
    if (!qweight || !scales || !aligned(qweight, 16) || !aligned(scales, 2)) return WQ_ERR_INVALID_ARG;
    if ((rows > 0 && !Y) || !aligned(Y, 16)) return WQ_ERR_INVALID_ARG;
    return WQ_OK;
}

wq_status check_codes(const int8_t* Xq, const float* x_scales, int64_t rows) {
    if (rows > 0 && (!Xq || !x_scales)) return WQ_ERR_INVALID_ARG;
    return aligned(Xq, 16) && aligned(x_scales, 4) ? WQ_OK : WQ_ERR_INVALID_ARG;
}

wq_status check_tokens(const void* X, int64_t T, int64_t d_in, const int32_t* rows, int64_t R, const void* smooth) {
    if (T < 0 || T > kMaxInt32 || R < 0 || R > kMaxInt32 || !depth_ok(d_in)) return WQ_ERR_INVALID_ARG;
    if (!rows && R != T && R != 0) return WQ_ERR_INVALID_ARG;
    if (R > 0 && T > 0 && !X) return WQ_ERR_INVALID_ARG;
    return aligned(X, 16) && aligned(rows, 4) && aligned(smooth, 2) ? WQ_OK : WQ_ERR_INVALID_ARG;
}

wq_status check_experts(const int32_t* offsets, int64_t E, int64_t d_out) {
    if (!offsets || !aligned(offsets, 4) || E < 1) return WQ_ERR_INVALID_ARG;
    if (E > WQ_INT8_MAX_EXPERTS) return WQ_ERR_UNSUPPORTED;
    return E * d_out <= kMaxInt32 ? WQ_OK : WQ_ERR_INVALID_ARG;
}

W8A8Args product_args(int64_t R, const int32_t* offsets, int64_t E, const uint32_t* qweight, const void* scales,
                      int64_t d_out, int64_t d_in, void* Y, int32_t y_dtype) {
    W8A8Args a = {};
    a.offsets = offsets;
    a.qweight = qweight;
    a.ws = static_cast<const uint16_t*>(scales);
    a.Y = Y;
    a.R = (int)R;
    a.N = (int)d_out;
    a.K = (int)d_in;
    a.E = (int)E;
    a.y_fp32 = y_dtype == WQ_OUT_FP32;
    return a;
}

wq_status status_of(cudaError_t e) {
    return e == cudaSuccess ? WQ_OK : e == cudaErrorNotSupported ? WQ_ERR_UNSUPPORTED : WQ_ERR_CUDA;
}

// The product of quantized rows.  Up to 64 rows per matrix (on average over the
// experts that can have any) stream the weights; more share tiles between two
// SMs.  Where the pairs' tiles do not give every pair one, a product of some
// depth streams all the same: only that kernel splits K, and it starts beside
// the kernel ahead.  Measured, us stream / pair, and behind a quantizer:
//   65 x 4096 x 11008   15.8 / 24.5   18.4 / 27.7     256 x 2048 x 8192   13.1 / 18.6   15.6 / 22.3
//   128 x 4096 x 4096   10.3 / 12.5   12.1 / 15.7     192 x 4096 x 4096   13.4 / 12.7   15.5 / 16.2
//   65 x 8192 x 8192    21.2 / 22.4   23.6 / 25.4     160 x 8192 x 8192   27.3 / 23.4   29.4 / 26.9
//   77 x 1001 x 1056     5.1 /  6.5    7.0 /  8.9     320 x 512 x 512      6.4 /  5.3    8.2 /  7.7
//   64 experts of 2048 x 4096, 65 rows each 93.7 / 94.2, 94 rows 114 / 98
//   2 experts of 512 x 4096, 75 rows 8.3 / 12.3; of 4096 x 4096 15.8 / 15.4; of 512 x 1024, 65 rows 7.2 / 8.1
cudaError_t run_product(const W8A8Args& a, int num_sms, cudaStream_t stream) {
    const int64_t experts = a.E < a.R ? a.E : a.R;
    const int pairs = num_sms / 2;
    const int64_t n_ct = ((int64_t)a.N + 255) / 256;
    const bool few_tiles = a.offsets ? (experts + a.R / 256) * n_ct < pairs / 4 : ((int64_t)a.R + 31) / 32 * n_ct < pairs;
    const bool streams = a.R <= 64 * experts || (few_tiles && a.K >= 1024);
    return streams ? launch_w8a8_stream(a, num_sms, pdl_enabled(), stream) : launch_w8a8_pair(a, num_sms, stream);
}

wq_status product_of_codes(W8A8Args a, const int8_t* Xq, const float* x_scales, void* stream) {
    int num_sms = 0;
    const wq_status v = device_info(&a.status, &num_sms);
    if (v != WQ_OK) return v;
    if (a.R == 0) return WQ_OK;
    a.Xq = Xq;
    a.xs = x_scales;
    return status_of(run_product(a, num_sms, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

wq_status wq_quantize_tokens(const void* X_bf16, int64_t T, int64_t d_in, const int32_t* rows, int64_t R,
                             const void* smooth_bf16, int8_t* Xq, float* x_scales, void* stream) {
    wq_status v = check_tokens(X_bf16, T, d_in, rows, R, smooth_bf16);
    if (v == WQ_OK) v = check_codes(Xq, x_scales, R);
    if (v != WQ_OK) return v;
    uint32_t* status = nullptr;
    int num_sms = 0;
    v = device_info(&status, &num_sms);
    if (v != WQ_OK) return v;
    if (R == 0) return WQ_OK;
    const cudaError_t e = launch_quantize_tokens(X_bf16, T, d_in, rows, R, smooth_bf16, Xq, x_scales, status,
                                                 pdl_enabled(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

wq_status wq_linear_w8a8(const int8_t* Xq, const float* x_scales, int64_t M, const uint32_t* qweight,
                         const void* scales_fp16, int64_t d_out, int64_t d_in, void* Y, int32_t y_dtype,
                         void* stream) {
    wq_status v = check_product(M, qweight, scales_fp16, d_out, d_in, Y, y_dtype);
    if (v == WQ_OK) v = check_codes(Xq, x_scales, M);
    if (v != WQ_OK) return v;
    return product_of_codes(product_args(M, nullptr, 1, qweight, scales_fp16, d_out, d_in, Y, y_dtype), Xq, x_scales,
                            stream);
}

wq_status wq_linear_w8a8_grouped(const int8_t* Xq, const float* x_scales, int64_t R, const int32_t* offsets, int64_t E,
                                 const uint32_t* qweight, const void* scales_fp16, int64_t d_out, int64_t d_in,
                                 void* Y, int32_t y_dtype, void* stream) {
    wq_status v = check_product(R, qweight, scales_fp16, d_out, d_in, Y, y_dtype);
    if (v == WQ_OK) v = check_codes(Xq, x_scales, R);
    if (v == WQ_OK) v = check_experts(offsets, E, d_out);
    if (v != WQ_OK) return v;
    return product_of_codes(product_args(R, offsets, E, qweight, scales_fp16, d_out, d_in, Y, y_dtype), Xq, x_scales,
                            stream);
}

}  // extern "C"
