// w8a8.h -- host-side launch functions of the W8A8 kernels (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/wq_int8.h"

namespace wq {

// The current device's status word and SM count (wq_api.cu); the injected host
// faults land here.  Must not run first inside a stream capture.
wq_status device_info(uint32_t** status, int* num_sms);
// WQ_DISABLE_PDL=1 turns programmatic dependent launch off.
bool pdl_enabled();

// Tensor map of an int8 matrix [rows][k] for tiles of `box_rows` rows and 128
// bytes of k ("atoms", SWIZZLE_128B).  k a multiple of 128: coordinates (0,
// row, atom), a load brings `atoms` atoms, one behind the other.  Else:
// coordinates (byte, row, 0), a load brings one.  Outside the matrix: zeros.
CUresult encode_tensor_map_k_atoms(CUtensorMap* map, const void* base, uint64_t k, uint64_t rows, int box_rows,
                                   int atoms);

cudaError_t launch_quantize_tokens(const void* X, int64_t T, int64_t K, const int32_t* rows, int64_t R,
                                   const void* smooth, int8_t* Xq, float* x_scales, uint32_t* status, bool pdl,
                                   cudaStream_t stream);

// One product: R rows against one weight matrix (offsets == nullptr, E == 1)
// or against the matrix of the expert that holds each row.
struct W8A8Args {
    const int8_t* Xq;         // [R][K]
    const float* xs;          // [R]
    const int32_t* offsets;   // [E + 1] or nullptr
    const uint32_t* qweight;  // [E][N][K/4]
    const uint16_t* ws;       // fp16 [E][N]
    void* Y;                  // [R][N] bf16 or fp32
    uint32_t* status;
    int R, N, K, E;
    int y_fp32;
};

// Sets a kernel's shared-memory limit once per device (the call costs 1.4 us).
cudaError_t allow_shared_memory(const void* kernel, int bytes, std::atomic<uint64_t>& done);

// Few rows per weight matrix: one CTA per tile of 128 channels, K split over a
// cluster when there are few tiles (w8a8_stream.cu).
cudaError_t launch_w8a8_stream(const W8A8Args& a, int num_sms, bool pdl, cudaStream_t stream);

// Many rows per weight matrix: pairs of CTAs share tiles of 256 channels x up
// to 256 rows (w8a8_pair.cu).  Never beside the other kernels of its stream.
cudaError_t launch_w8a8_pair(const W8A8Args& a, int num_sms, cudaStream_t stream);

}  // namespace wq
