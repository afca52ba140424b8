// w8a8_stream.cu -- INT8 x INT8 linear layer, few rows per weight matrix
// (sm_100a): decode, short chunks, sparsely loaded experts.
//
// Y[m, n] = s_m w_n sum_k Xq[m, k] q[n, k].  With few rows the product is bound
// by the weight stream (one byte per weight), so the weights are the A operand:
// a tile is 128 output channels x up to 64 rows, D[channel][row] int32 in
// tensor memory, and INT8 needs no dequantization between the two.  TMA brings
// 128-byte-wide atoms (SWIZZLE_128B, K-major) of weights and rows into a ring,
// two atoms per stage and instruction, one thread issues tcgen05.mma kind::i8
// (M = 128, N = rows rounded up to 16, K = 32), four warps scale and store.
// The CUDA cores touch no weight.
//
// Few tiles (one token against 4096 channels has 32) would leave most SMs
// idle: then a cluster of up to 8 CTAs splits K.  The columns of D are dealt
// out to the CTAs in groups of 4; each sends the others their groups of its
// int32 partials with 16-byte st.async, counted on the receiver's mbarrier,
// and adds up its own.  Integer sums do not depend on their order, so the
// result is the same for every split.
//
// For one weight matrix, a ring's worth of the first weights is brought into L2
// before the wait for the previous kernel (programmatic dependent launch).  All
// loads follow the wait: the kernels between this one and the writer of its
// weights may have started early too, so that "the kernel ahead does not write
// weights" does not mean that they are written.  Weights loaded into shared
// memory before the wait saved 0.6 us more (4096 x 4096, 1 row 5.75 against 6.4)
// and were stale behind such a chain; a quantizer that lets this kernel start
// only after its own wait took 9.0 us with it, this 7.6.  What follows the wait
// is kept short: one load, the MMAs, one exchange.  Every wait on an mbarrier is
// bounded (WQ_DEVFLAG_TIMEOUT).
//
// Measured (weights from HBM, launches back to back): 4096 x 4096 6.4 us for
// 1 row, 6.6 for 16, 8.8 for 64; 11008 x 4096, 16 rows 11.8 us (3.9 TB/s);
// 28672 x 8192, 1 row 39.6 us (5.9 TB/s, 90 % of the measured copy rate); 64
// experts of 2048 x 4096, 2 rows each 84 us (97 %).  Beyond the stream itself a
// call costs about 4 us (one matrix) to 6 us (experts: the offsets come first).
#include <stdint.h>

#include "w8a8.h"
#include "w8a8_device.cuh"
#include "wq_kernels.h"

namespace wq {
namespace {

constexpr int kCh = 128;                  // output channels per tile (MMA M)
constexpr int kAtom = 128;                // k per swizzle atom
constexpr int kMaxAtoms = 2;              // atoms per stage and copy
constexpr int kATile = kCh * kAtom;       // bytes of weights per atom
constexpr int kMaxRows = 64;              // rows per tile
constexpr int kThreads = 192;             // copy warp, MMA warp, 4 epilogue warps
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;

struct StreamPlan {
    int nt;       // most rows of a tile (16, 32 or 64)
    int stages;
    int atoms;    // per stage: 2, or 1 where two stages of 2 would not fit
    int split;    // CTAs that share a tile's K
    int n_ct;     // channel tiles
    int grid;
    int smem;
};

// Boxes of 16, 32, 48 and 64 rows: a tile's rows rounded up to 16, in one copy.
struct RowMaps {
    CUtensorMap m[kMaxRows / 16];
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

__host__ __device__ constexpr int table_ints(int E) { return (E + 1 + 3) & ~3; }
// Shared memory behind the stages: partials from the cluster, row scales, tile
// table, barriers.
__host__ __device__ constexpr int recv_bytes(int nt, int split) {
    return split > 1 ? split * ((nt / 4 + split - 1) / split) * kCh * 16 : 0;
}
__host__ __device__ constexpr int tail_bytes(int nt, int split, int E) {
    return recv_bytes(nt, split) + 2 * nt * 4 + 2 * table_ints(E) * 4 + 64 * 4 + (int)sizeof(StreamBars);
}

__global__ void __launch_bounds__(kThreads) w8a8_stream_kernel(const __grid_constant__ RowMaps tmap_x,
                                                               const __grid_constant__ CUtensorMap tmap_w,
                                                               const W8A8Args a, const StreamPlan p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int b_tile = p.nt * kAtom;
    uint8_t* smem_a = smem;
    uint8_t* smem_b = smem + p.stages * p.atoms * kATile;
    uint8_t* tail = smem_b + p.stages * p.atoms * b_tile;
    uint4* recv = reinterpret_cast<uint4*>(tail);  // [sender][own group][channel]
    float* row_scale = reinterpret_cast<float*>(tail + recv_bytes(p.nt, p.split));  // [2][nt]
    int* off = reinterpret_cast<int*>(row_scale + 2 * p.nt);
    int* cum = off + table_ints(a.E);
    int* warp_part = cum + table_ints(a.E);
    StreamBars& bar = *reinterpret_cast<StreamBars*>(warp_part + 64);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % (unsigned)p.split);
    const int worker = (int)(blockIdx.x / (unsigned)p.split), workers = (int)(gridDim.x / (unsigned)p.split);
    const int atoms = (a.K + kAtom - 1) / kAtom, nkb = (atoms + p.atoms - 1) / p.atoms;
    const int kb0 = nkb * rank / p.split, kb1 = nkb * (rank + 1) / p.split;
    const bool whole = a.K % kAtom == 0;  // a stage's atoms in one copy
    const int tmem_cols = p.nt * 2;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmap_w);
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
    // With experts the tiles come from the work ahead: nothing is held before it has ended.
    if (a.offsets) pdl_wait_prior();
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(&bar.tmem_slot, (uint32_t)tmem_cols);
        tmem_relinquish();
        tc_fence_before();
    }
    build_tiles(a.offsets, a.E, a.R, p.nt, off, cum, warp_part, kThreads, a.status);  // ends with __syncthreads
    // Only now may the next kernel start: it could take the tensor memory that
    // this one still has to allocate, and wait for it.
    pdl_launch_dependents();
    if (p.split > 1) cluster_arrive();
    tc_fence_after();
    const uint32_t tmem_base = bar.tmem_slot;
    const int total = cum[a.E] * p.n_ct;
    volatile int* abort_flag = &bar.abort_flag;

    if (warp == 0) {
        // ---------------- copy warp ----------------
        const bool one = elect_one();
        const uint32_t a0 = smem_u32(smem_a), b0 = smem_u32(smem_b), full0 = smem_u32(bar.full);
        int it = 0;
        bool waited = a.offsets != nullptr;
        for (int t = worker; t < total && !__any_sync(0xffffffffu, *abort_flag); t += workers) {
            const TokenTile w = find_tile(t, p.n_ct, a.E, off, cum, 16);
            const int rows = (w.n + 15) & ~15;
            const CUtensorMap* tx = &tmap_x.m[rows / 16 - 1];
            const int wrow = w.e * a.N + w.ct * kCh;
            const auto expect = [&](int s, int kb) {
                const int here = whole ? p.atoms : min(p.atoms, atoms - kb * p.atoms);
                if (one) mbar_arrive_expect_tx(&bar.full[s], (uint32_t)(here * (kATile + rows * kAtom)));
            };
            const auto load = [&](uint32_t dst, int atom_bytes, const CUtensorMap* map, int s, int kb, int row) {
                if (whole) {
                    tma_load_3d(one, dst, map, full0 + 8 * s, 0, row, kb * p.atoms);
                } else {
                    for (int at = 0; at < p.atoms && kb * p.atoms + at < atoms; ++at)
                        tma_load_3d(one, dst + at * atom_bytes, map, full0 + 8 * s, (kb * p.atoms + at) * kAtom, row, 0);
                }
            };
            if (!waited) {
                // one weight matrix: the first weights come into L2 meanwhile
                for (int i = kb0; i < min(kb0 + p.stages, kb1); ++i) {
                    if (whole) {
                        tma_prefetch_3d(one, &tmap_w, 0, wrow, i * p.atoms);
                    } else {
                        for (int at = 0; at < p.atoms && i * p.atoms + at < atoms; ++at)
                            tma_prefetch_3d(one, &tmap_w, (i * p.atoms + at) * kAtom, wrow, 0);
                    }
                }
                prefetch_tmap(tx);
                pdl_wait_prior();
                waited = true;
            }
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % p.stages;
                if (it >= p.stages &&
                    !__all_sync(0xffffffffu, mbar_wait(&bar.empty[s], (uint32_t)(it / p.stages - 1) & 1u, a.status))) {
                    atomicExch(&bar.abort_flag, 1);
                    break;
                }
                expect(s, kb);
                load(a0 + s * p.atoms * kATile, kATile, &tmap_w, s, kb, wrow);
                load(b0 + s * p.atoms * b_tile, rows * kAtom, tx, s, kb, w.row0);
            }
        }
        // the loads in flight land before the CTA ends
        for (int j = max(0, it - p.stages); j < it; ++j)
            mbar_wait(&bar.full[j % p.stages], (uint32_t)(j / p.stages) & 1u, a.status);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA warp ----------------
        if (!a.offsets) pdl_wait_prior();  // the bounded waits below do not cover the previous kernel
        const bool one = elect_one();
        int it = 0, ti = 0;
        for (int t = worker; t < total && !__any_sync(0xffffffffu, *abort_flag); t += workers, ++ti) {
            const TokenTile w = find_tile(t, p.n_ct, a.E, off, cum, 16);
            const int rows = (w.n + 15) & ~15;
            const uint32_t idesc = mma_idesc_s8(kCh, rows);
            const int acc = ti & 1;
            bool ok = ti < 2 || __all_sync(0xffffffffu, mbar_wait(&bar.acc_empty[acc], (uint32_t)((ti >> 1) - 1) & 1u, a.status));
            tc_fence_after();
            for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                const int s = it % p.stages;
                const uint64_t ad = sw128_kmajor_desc(smem_u32(smem_a + s * p.atoms * kATile));
                const uint64_t bd = sw128_kmajor_desc(smem_u32(smem_b + s * p.atoms * b_tile));
                const int here = min(p.atoms, atoms - kb * p.atoms);
                ok = __all_sync(0xffffffffu, mbar_wait(&bar.full[s], (uint32_t)(it / p.stages) & 1u, a.status));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int at = 0; at < kMaxAtoms; ++at) {
                    if (at >= here) break;
#pragma unroll
                    for (int kk = 0; kk < kAtom / 32; ++kk)  // descriptors count 16-byte units
                        tc_mma_i8(one, tmem_base + (uint32_t)(acc * p.nt), ad + (at * kATile + kk * 32) / 16,
                                  bd + (at * rows * kAtom + kk * 32) / 16, idesc,
                                  (kb != kb0 || at != 0 || kk != 0) ? 1u : 0u);
                }
                if (one) tc_commit(&bar.empty[s]);
            }
            if (!ok) {
                atomicExch(&bar.abort_flag, 1);
                break;
            }
            if (one) tc_commit(&bar.acc_full[acc]);
        }
        if (one) tc_commit(&bar.drain);  // completes once every MMA issued above has
        mbar_wait(&bar.drain, 0u, a.status);
        __syncwarp();
    } else {
        // ---------------- epilogue warps ----------------
        const int q = warp & 3;            // tensor memory lanes this warp may read
        const int ch = q * 32 + lane;      // channel within the tile
        const int et = threadIdx.x - 64;   // 0 .. 127
        bool waited = a.offsets != nullptr, joined = p.split == 1;
        int ti = 0;
        for (int t = worker; t < total; t += workers, ++ti) {
            const TokenTile w = find_tile(t, p.n_ct, a.E, off, cum, 16);
            const int acc = ti & 1;
            const int c = w.ct * kCh + ch;
            const bool cv = c < a.N;
            // groups of 4 columns: group g belongs to CTA g % split of the cluster
            const int groups = (w.n + 3) >> 2;
            const int pitch = (groups + p.split - 1) / p.split;  // groups kept per sender
            const int own = rank < groups ? (groups - rank + p.split - 1) / p.split : 0;
            if (!joined) {
                if (et == 0) mbar_arrive_expect_tx(&bar.recv, (uint32_t)((p.split - 1) * own * kCh * 16));
                cluster_wait();  // the others' barriers are initialised
                joined = true;
            }
            if (!waited) {
                pdl_wait_prior();
                waited = true;
            }
            const float sw = cv ? __half2float(__ushort_as_half(a.ws[(int64_t)w.e * a.N + c])) : 0.0f;
            float* rs = row_scale + acc * p.nt;
            if (et < w.n) rs[et] = a.xs[w.row0 + et];
            if (!named_sync_and(1, 128, !*abort_flag)) break;
            const bool ok = __all_sync(0xffffffffu, mbar_wait(&bar.acc_full[acc], (uint32_t)(ti >> 1) & 1u, a.status));
            tc_fence_after();
            if (!ok) {
                atomicExch(&bar.abort_flag, 1);
                continue;  // the next barrier ends the loop for all warps
            }
            const uint32_t dcol = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * p.nt);
            if (p.split == 1) {
                for (int c0 = 0; c0 < w.n; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(dcol + (uint32_t)c0, v);
                    tc_wait_ld();
                    if (cv)
                        w8a8_store_cols(a.Y, a.y_fp32, (int64_t)(w.row0 + c0) * a.N + c, a.N, sw, rs + c0, v, w.n - c0);
                }
            } else {
                const uint32_t recv_bar = smem_u32(&bar.recv);
                uint32_t slot = smem_u32(recv) + (uint32_t)((rank * pitch * kCh + ch) * 16);
                int r = 0;
                for (int c0 = 0; c0 < w.n; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(dcol + (uint32_t)c0, v);
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        if (c0 + j < w.n) {
                            if (r == rank)
                                recv[(slot - smem_u32(recv)) / 16] = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                            else
                                st_async_v4(map_rank(slot, (uint32_t)r), v[j], v[j + 1], v[j + 2], v[j + 3],
                                            map_rank(recv_bar, (uint32_t)r));
                            if (++r == p.split) {
                                r = 0;
                                slot += kCh * 16;
                            }
                        }
                    }
                }
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(&bar.recv, 0u, a.status))) {
                    atomicExch(&bar.abort_flag, 1);
                    continue;
                }
                for (int g = 0; g < own; ++g) {
                    int sum[4] = {0, 0, 0, 0};
                    for (int s = 0; s < p.split; ++s) {
                        const uint4 v = recv[(s * pitch + g) * kCh + ch];
                        sum[0] += (int)v.x;
                        sum[1] += (int)v.y;
                        sum[2] += (int)v.z;
                        sum[3] += (int)v.w;
                    }
                    const int col = (g * p.split + rank) * 4;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (cv && col + j < w.n)
                            w8a8_store(a.Y, a.y_fp32, (int64_t)(w.row0 + col + j) * a.N + c,
                                       w8a8_value(sum[j], sw, rs[col + j]));
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
    tc_fence_before();
    __syncthreads();
    if (p.split > 1) {
        if (warp < 2) cluster_wait();
        // All that the others send here has arrived, unless a wait gave up: then
        // this CTA stays until they have ended or come here too.
        if (*abort_flag) {
            cluster_arrive();
            cluster_wait();
        }
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, (uint32_t)tmem_cols);
    }
}

constexpr int kCtaSmem = 112 * 1024;  // two CTAs per SM

}  // namespace

cudaError_t launch_w8a8_stream(const W8A8Args& a, int num_sms, bool pdl, cudaStream_t stream) {
    StreamPlan p = {};
    p.n_ct = ceil_div(a.N, kCh);
    const int experts = a.E < a.R ? a.E : a.R;  // that can have rows
    const int per_expert = ceil_div(a.R, experts);
    // rows per tile: what an expert holds, with room for an uneven share
    p.nt = 16;
    while (p.nt < kMaxRows && p.nt < (a.offsets ? 2 * per_expert : per_expert)) p.nt *= 2;
    const int64_t tiles = (a.offsets ? (int64_t)experts + a.R / p.nt : ceil_div(a.R, p.nt)) * p.n_ct;
    if (tiles > 0x3fffffff) return cudaErrorNotSupported;  // tile numbers stay far from overflow
    const int atoms = ceil_div(a.K, kAtom);
    const int64_t slots = 2 * (int64_t)num_sms;
    // Clusters that all fit at once: a cluster stays within one GPC, so not every
    // slot can be used (12288 x 4096, M = 1: 288 CTAs in clusters of 3 took 16.7 us,
    // 192 in clusters of 2 take 12.6; 258 of 296 still fit).
    p.split = 1;
    while (p.split < kMaxSplit && tiles * (p.split + 1) * 10 <= slots * 9 && atoms >= kMaxAtoms * (p.split + 1)) ++p.split;
    const int tail = 1024 + tail_bytes(p.nt, p.split, a.E);
    p.atoms = kMaxAtoms;
    if ((kCtaSmem - tail) / (p.atoms * (kATile + p.nt * kAtom)) < 2) p.atoms = 1;
    const int stage = p.atoms * (kATile + p.nt * kAtom);
    p.stages = (kCtaSmem - tail) / stage;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    if (p.stages < 1) return cudaErrorInvalidConfiguration;
    p.smem = tail + p.stages * stage;
    p.grid = (int)(p.split > 1 || tiles < slots ? tiles : slots) * p.split;

    RowMaps tx = {};
    CUtensorMap tw;
    CUresult cr = encode_tensor_map_k_atoms(&tw, a.qweight, (uint64_t)a.K, (uint64_t)a.E * (uint64_t)a.N, kCh, p.atoms);
    // one matrix: no tile has more rows than the first
    const int most = ceil_div(ceil_div(a.R, ceil_div(a.R, p.nt)), 16) * 16;
    for (int rows = 16; rows <= p.nt && cr == CUDA_SUCCESS; rows += 16)
        if (a.offsets || rows <= most)
            cr = encode_tensor_map_k_atoms(&tx.m[rows / 16 - 1], a.Xq, (uint64_t)a.K, (uint64_t)a.R, rows, p.atoms);
    if (cr != CUDA_SUCCESS) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(w8a8_stream_kernel), kCtaSmem, allowed);
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
