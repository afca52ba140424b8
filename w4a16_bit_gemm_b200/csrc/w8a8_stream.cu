// w8a8_stream.cu -- INT8 x INT8 linear layer, few rows per weight matrix
// (sm_100a): decode, short chunks, sparsely loaded experts.
//
// Y[m, n] = s_m w_n sum_k Xq[m, k] q[n, k].  With few rows the product is bound
// by the weight stream (one byte per weight), so the weights are the A operand:
// a tile is 128 output channels x up to NT rows, D[channel][row] int32 in
// tensor memory, and INT8 needs no dequantization between the two.  TMA brings
// 128-byte-wide boxes (SWIZZLE_128B, K-major) of weights and rows into a ring,
// one thread issues tcgen05.mma kind::i8 (M = 128, N = rows rounded up to 16,
// K = 32), four warps scale and store.  The CUDA cores touch no weight.
//
// Few tiles (one token against 4096 channels has 32) would leave most SMs
// idle: then a cluster of up to 8 CTAs splits K.  Each CTA owns some of the
// tile's rows (columns of D); the others send it their int32 partials with
// st.async, counted on its mbarrier, and it adds them up.  Integer sums do not
// depend on their order, so the result is the same for every split.
//
// For one weight matrix, the first weights are requested before the wait for
// the previous kernel (programmatic dependent launch): they do not depend on
// it, the activations do.  Every wait is bounded (WQ_DEVFLAG_TIMEOUT).
#include <stdint.h>

#include "w8a8.h"
#include "w8a8_device.cuh"
#include "wq_kernels.h"

namespace wq {
namespace {

constexpr int kCh = 128;                  // output channels per tile (MMA M)
constexpr int kKB = 128;                  // k per stage (one swizzle atom of bytes)
constexpr int kATile = kCh * kKB;         // bytes
constexpr int kThreads = 192;             // copy warp, MMA warp, 4 epilogue warps
constexpr int kMaxStages = 16;
constexpr int kMaxSplit = 8;

struct StreamPlan {
    int nt;       // most rows of a tile (16, 32 or 64)
    int box;      // rows of one TMA box of Xq
    int stages;
    int split;    // CTAs that share a tile's K
    int n_ct;     // channel tiles
    int grid;
    int smem;
};

struct StreamBars {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t recv;
    uint64_t drain;
    uint32_t tmem_slot;
    int abort_flag;
};

__host__ __device__ constexpr int align16(int x) { return (x + 15) & ~15; }

// Shared memory behind the stages: partials from the cluster, row scales,
// tile table, barriers.
__host__ __device__ constexpr int recv_bytes(int nt, int split) { return split > 1 ? (nt + kMaxSplit) * kCh * 4 : 0; }
__host__ __device__ constexpr int tail_bytes(int nt, int split, int E) {
    return recv_bytes(nt, split) + 2 * nt * 4 + align16((E + 1) * 4) * 2 + 64 * 4 + (int)sizeof(StreamBars);
}

__global__ void __launch_bounds__(kThreads) w8a8_stream_kernel(const __grid_constant__ CUtensorMap tmap_x,
                                                               const __grid_constant__ CUtensorMap tmap_w,
                                                               const W8A8Args a, const StreamPlan p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int b_tile = p.nt * kKB;
    uint8_t* smem_a = smem;
    uint8_t* smem_b = smem + p.stages * kATile;
    uint8_t* tail = smem_b + p.stages * b_tile;
    uint32_t* recv = reinterpret_cast<uint32_t*>(tail);
    float* row_scale = reinterpret_cast<float*>(tail + recv_bytes(p.nt, p.split));  // [2][nt]
    int* off = reinterpret_cast<int*>(row_scale + 2 * p.nt);
    int* cum = off + align16((a.E + 1) * 4) / 4;
    int* warp_part = cum + align16((a.E + 1) * 4) / 4;
    StreamBars& bar = *reinterpret_cast<StreamBars*>(warp_part + 64);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % (unsigned)p.split);
    const int worker = (int)(blockIdx.x / (unsigned)p.split), workers = (int)(gridDim.x / (unsigned)p.split);
    const int nkb = (a.K + kKB - 1) / kKB;
    const int kb0 = nkb * rank / p.split, kb1 = nkb * (rank + 1) / p.split;
    const int tmem_cols = p.nt * 2 < 32 ? 32 : p.nt * 2;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar.acc_full[s], 1);
            mbar_init(&bar.acc_empty[s], 4);
        }
        mbar_init(&bar.recv, 1);
        mbar_init(&bar.drain, 1);
        bar.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bar.tmem_slot, (uint32_t)tmem_cols);
        tmem_relinquish();
        tc_fence_before();
    }
    // one weight matrix: the weights of this CTA's first stages are requested
    // before anything that depends on the previous kernel
    int ahead = 0;
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmap_w);
        prefetch_tmap(&tmap_x);
    }
    if (a.offsets) pdl_wait_prior();
    build_tiles(a.offsets, a.E, a.R, p.nt, off, cum, warp_part, kThreads, a.status);  // ends with __syncthreads
    if (p.split > 1) cluster_arrive();
    tc_fence_after();
    const uint32_t tmem_base = bar.tmem_slot;
    const int total = cum[a.E] * p.n_ct;
    volatile int* abort_flag = &bar.abort_flag;

    if (warp == 0) {
        // ---------------- copy warp ----------------
        if (lane == 0) {
            int it = 0;
            bool waited = a.offsets != nullptr;
            for (int t = worker; t < total && !*abort_flag; t += workers) {
                const TokenTile w = find_tile(t, p.n_ct, a.E, off, cum, 16);
                const int boxes = ceil_div(w.n, p.box);
                const uint32_t bytes = (uint32_t)(kATile + boxes * p.box * kKB);
                const int wrow = w.e * a.N + w.ct * kCh;
                if (!waited) {
                    ahead = min(p.stages, kb1 - kb0);
                    for (int i = 0; i < ahead; ++i) {
                        mbar_arrive_expect_tx(&bar.full[i], bytes);
                        tma_load_2d(smem_a + i * kATile, &tmap_w, &bar.full[i], (kb0 + i) * kKB, wrow);
                    }
                    pdl_wait_prior();
                    waited = true;
                }
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % p.stages;
                    if (it >= ahead) {
                        if (it >= p.stages && !mbar_wait(&bar.empty[s], (uint32_t)(it / p.stages - 1) & 1u, a.status)) {
                            atomicExch(&bar.abort_flag, 1);
                            break;
                        }
                        mbar_arrive_expect_tx(&bar.full[s], bytes);
                        tma_load_2d(smem_a + s * kATile, &tmap_w, &bar.full[s], kb * kKB, wrow);
                    }
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(smem_b + s * b_tile + b * p.box * kKB, &tmap_x, &bar.full[s], kb * kKB,
                                    w.row0 + b * p.box);
                }
            }
            // the loads in flight land before the CTA ends
            for (int j = max(0, it - p.stages); j < it; ++j)
                mbar_wait(&bar.full[j % p.stages], (uint32_t)(j / p.stages) & 1u, a.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA warp ----------------
        if (lane == 0) {
            int it = 0, ti = 0;
            for (int t = worker; t < total && !*abort_flag; t += workers, ++ti) {
                const TokenTile w = find_tile(t, p.n_ct, a.E, off, cum, 16);
                const uint32_t idesc = mma_idesc_s8(kCh, (w.n + 15) & ~15);
                const int acc = ti & 1;
                bool ok = ti < 2 || mbar_wait(&bar.acc_empty[acc], (uint32_t)((ti >> 1) - 1) & 1u, a.status);
                tc_fence_after();
                for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                    const int s = it % p.stages;
                    ok = mbar_wait(&bar.full[s], (uint32_t)(it / p.stages) & 1u, a.status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(smem_a + s * kATile), b_addr = smem_u32(smem_b + s * b_tile);
#pragma unroll
                    for (int kk = 0; kk < kKB / 32; ++kk)
                        tc_mma_i8(tmem_base + (uint32_t)(acc * p.nt), sw128_kmajor_desc(a_addr + kk * 32),
                                  sw128_kmajor_desc(b_addr + kk * 32), idesc, (kb != kb0 || kk != 0) ? 1u : 0u);
                    tc_commit(&bar.empty[s]);
                }
                if (!ok) {
                    atomicExch(&bar.abort_flag, 1);
                    break;
                }
                tc_commit(&bar.acc_full[acc]);
            }
            tc_commit(&bar.drain);  // completes once every MMA issued above has
            mbar_wait(&bar.drain, 0u, a.status);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue warps ----------------
        if (!a.offsets) pdl_wait_prior();
        const int q = warp & 3;            // tensor memory lanes this warp may read
        const int ch = q * 32 + lane;      // channel within the tile
        const int et = threadIdx.x - 64;   // 0 .. 127
        bool joined = p.split == 1;
        int ti = 0;
        for (int t = worker; t < total; t += workers, ++ti) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            const TokenTile w = find_tile(t, p.n_ct, a.E, off, cum, 16);
            const int acc = ti & 1;
            float* rs = row_scale + acc * p.nt;
            for (int i = et; i < w.n; i += 128) rs[i] = a.xs[w.row0 + i];
            const int c = w.ct * kCh + ch;
            const bool cv = c < a.N;
            const float sw = cv ? __half2float(__ushort_as_half(a.ws[(int64_t)w.e * a.N + c])) : 0.0f;
            named_sync(1, 128);
            const bool ok = __all_sync(0xffffffffu, mbar_wait(&bar.acc_full[acc], (uint32_t)(ti >> 1) & 1u, a.status));
            tc_fence_after();
            if (!ok) {
                atomicExch(&bar.abort_flag, 1);
                break;
            }
            const uint32_t dcol = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * p.nt);
            if (p.split == 1) {
                for (int c0 = 0; c0 < w.n; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(dcol + (uint32_t)c0, v);
                    tc_wait_ld();
                    if (!cv) continue;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c0 + j < w.n)
                            w8a8_store(a.Y, a.y_fp32, (int64_t)(w.row0 + c0 + j) * a.N + c,
                                       w8a8_value((int)v[j], sw, rs[c0 + j]));
                }
            } else {
                // CTA r of the cluster owns columns [lo(r), lo(r + 1)), lo(r) = ceil(n r / split)
                const int own0 = (w.n * rank + p.split - 1) / p.split, own1 = (w.n * (rank + 1) + p.split - 1) / p.split;
                const int pitch = (w.n + p.split - 1) / p.split;  // columns kept per sender
                if (et == 0) mbar_arrive_expect_tx(&bar.recv, (uint32_t)((p.split - 1) * (own1 - own0) * kCh * 4));
                if (!joined) {
                    cluster_wait();  // the others' barriers are initialised
                    joined = true;
                }
                const uint32_t slot = smem_u32(recv) + (uint32_t)((rank * pitch * kCh + ch) * 4);
                const uint32_t recv_bar = smem_u32(&bar.recv);
                int r = 0, lo = 0, hi = (w.n + p.split - 1) / p.split;
                for (int c0 = 0; c0 < w.n; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(dcol + (uint32_t)c0, v);
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (c0 + j < w.n) {
                            while (c0 + j >= hi) {
                                ++r;
                                lo = hi;
                                hi = (w.n * (r + 1) + p.split - 1) / p.split;
                            }
                            const uint32_t at = slot + (uint32_t)((c0 + j - lo) * kCh * 4);
                            if (r == rank)
                                recv[(rank * pitch + c0 + j - lo) * kCh + ch] = v[j];
                            else
                                st_async_b32(map_rank(at, (uint32_t)r), v[j], map_rank(recv_bar, (uint32_t)r));
                        }
                    }
                }
                if (!__all_sync(0xffffffffu, mbar_wait(&bar.recv, 0u, a.status))) {
                    atomicExch(&bar.abort_flag, 1);
                    break;
                }
                for (int j = own0; j < own1 && cv; ++j) {
                    int sum = 0;
                    for (int s = 0; s < p.split; ++s) sum += (int)recv[(s * pitch + j - own0) * kCh + ch];
                    w8a8_store(a.Y, a.y_fp32, (int64_t)(w.row0 + j) * a.N + c, w8a8_value(sum, sw, rs[j]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.acc_empty[acc]);
        }
        __syncwarp();
        if (!joined) cluster_wait();
    }

    // ---------------- teardown ----------------
    if (p.split > 1) {
        // no CTA ends while another may still write into its shared memory
        if (warp < 2) cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, (uint32_t)tmem_cols);
    }
}

}  // namespace

cudaError_t launch_w8a8_stream(const W8A8Args& a, int num_sms, bool pdl, cudaStream_t stream) {
    StreamPlan p = {};
    p.n_ct = ceil_div(a.N, kCh);
    const int per_expert = ceil_div(a.R, a.E < a.R ? a.E : a.R);
    // rows per tile: what an expert holds, with room for an uneven share
    p.nt = 16;
    while (p.nt < 64 && p.nt < (a.offsets ? 2 * per_expert : per_expert)) p.nt *= 2;
    // one matrix: all rows in one box; experts: only boxes that hold rows of theirs
    p.box = a.offsets ? 16 : p.nt;
    const int64_t token_tiles = a.offsets ? (int64_t)(a.E < a.R ? a.E : a.R) + a.R / p.nt : ceil_div(a.R, p.nt);
    const int64_t tiles = token_tiles * p.n_ct;
    if (tiles > 0x7fffffff) return cudaErrorNotSupported;
    const int nkb = ceil_div(a.K, kKB);
    constexpr int per_sm = 2;
    p.split = 1;
    while (p.split < kMaxSplit && tiles * (p.split + 1) <= (int64_t)num_sms * per_sm && nkb >= 2 * (p.split + 1)) ++p.split;
    const int budget = 112 * 1024 - 1024 - tail_bytes(p.nt, p.split, a.E);
    p.stages = budget / (kATile + p.nt * kKB);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    if (p.stages < 2) return cudaErrorInvalidConfiguration;
    p.smem = 1024 + p.stages * (kATile + p.nt * kKB) + tail_bytes(p.nt, p.split, a.E);
    p.grid = (int)(p.split > 1 || tiles < (int64_t)num_sms * per_sm ? tiles : (int64_t)num_sms * per_sm) * p.split;

    CUtensorMap tx, tw;
    CUresult cr = encode_tensor_map_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.Xq, (uint64_t)a.K, (uint64_t)a.R,
                                       (uint64_t)a.K, kKB, (uint32_t)p.box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (cr == CUDA_SUCCESS)
        cr = encode_tensor_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.qweight, (uint64_t)a.K,
                                  (uint64_t)a.E * (uint64_t)a.N, (uint64_t)a.K, kKB, kCh, CU_TENSOR_MAP_SWIZZLE_128B);
    if (cr != CUDA_SUCCESS) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(w8a8_stream_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, w8a8_stream_kernel, tx, tw, a, p);
}

}  // namespace wq
