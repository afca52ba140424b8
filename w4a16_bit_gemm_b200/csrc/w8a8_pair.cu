// w8a8_pair.cu -- INT8 x INT8 linear layer, many rows per weight matrix
// (sm_100a): prefill, long chunks, loaded experts.
//
// Y[m, n] = s_m w_n sum_k Xq[m, k] q[n, k] on pairs of SMs: one
// tcgen05.mma.cta_group::2 (kind::i8, M = 256, K = 32) multiplies 256 output
// channels, 128 from each CTA's shared memory, with up to 256 rows, half of
// them from each CTA.  A 1-SM tile of 128 x 256 needs 48 KB of operands per
// 128 k; a pair needs 32 KB per SM for twice the product.
//
// Rows are the N side, so a tile with few rows (the last one of a prompt, a
// lightly loaded expert) costs its own rows rounded up to 32, not a full tile.
// The accumulator is int32 in tensor memory, two of 256 columns: the epilogue
// of a tile runs under the products of the next.  Or both belong to one tile of
// 512 channels, which reads a quarter less from L2 (13 to 14 TB/s into the SMs
// was the bound of 256-channel tiles at full clock).  Persistent: each pair walks
// the tiles in steps of the number of pairs.  Every wait on an mbarrier is
// bounded (WQ_DEVFLAG_TIMEOUT); the cluster's barriers are reached by all threads
// on every path.
//
// No programmatic dependent launch, on either side: a quantizer's blocks beside
// this kernel as it starts are the common part of three chains that did not
// finish, when the collective allocation of tensor memory still came before the
// first cluster barrier.  It costs 2.5 to 3 us behind a quantizer (512 x 4096 x
// 4096 from bf16 15.1 -> 17.8 us, 128 x 11008 x 4096 15.7 -> 18.7, 512 x 8192 x
// 8192 31.4 -> 34.0) and 1 to 4 us for a call with experts by itself.
//
// Bound by the tensor pipe (84 to 88 % of active cycles) and, in long runs, by
// the power cap: 2048 x 8192 x 8192 91 us (3020 TOPS, 91 % of twice the bf16
// rate of cuBLAS), 8192 x 28672 x 8192 1.22 to 1.24 ms in a burst, 1.33 to 1.36
// ms back to back, 8192 x 1024 x 8192 46.5 us.  On the way: 1-SM tiles 153 us and
// 1.82 ms; pairs 103 us and 1.37 ms; two atoms per stage and copy, so that the
// issuing threads keep up, and an epilogue of eight warps without a test per
// column 89 us and 1.24 ms (1.45 back to back); tiles of 512 channels; waits that
// acquire from the cluster 1 % more.  Small products add about 9 us of start,
// last epilogue and hand-off (512 x 8192 x 8192 30 us).
#include <stdint.h>

#include "w8a8.h"
#include "w8a8_device.cuh"
#include "wq_kernels.h"

namespace wq {
namespace {

constexpr int kKB = 128;                 // k per swizzle atom
constexpr int kMaxRows = 256;            // rows per tile
constexpr int kBTile = 128 * kKB;        // bytes of rows per CTA and atom
constexpr int kEpiWarps = 8;             // per accumulator of a tile
constexpr int kTmemCols = 2 * kMaxRows;

// kSub = 1: tiles of 256 channels, 128 per CTA; the two accumulators belong to
// successive tiles.  kSub = 2: tiles of 512 channels, 256 per CTA; each
// accumulator takes 128 of them, and a row is fetched once for both.
template <int kSub>
struct Shape {
    static constexpr int kCh = 256 * kSub;           // channels per tile
    static constexpr int kCtaCh = 128 * kSub;        // channels per CTA
    static constexpr int kAtoms = kSub == 1 ? 2 : 1; // atoms per stage
    static constexpr int kStages = kSub == 1 ? 3 : 4;
    static constexpr int kATile = kCtaCh * kKB;      // bytes of weights per CTA and atom
    static constexpr int kEpi = 32 * kEpiWarps * kSub;  // epilogue threads
    static constexpr int kThreads = 64 + kEpi;       // copy warp, MMA warp, epilogue warps
};
constexpr int kMostStages = 4;

struct PairPlan {
    int step;   // most rows of a tile, a multiple of 32
    int n_ct;   // channel tiles
};

// Boxes of 16, 32, ... 128 rows: the half of a tile's rows that a CTA brings, in
// one copy.
struct RowMaps {
    CUtensorMap m[8];
};

struct PairBars {
    uint64_t full[kMostStages];   // leader: both CTAs' bytes
    uint64_t empty[kMostStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];    // leader: the epilogue warps of both CTAs
    uint64_t drain;           // leader
    uint32_t tmem_slot;
    int abort_flag;
};

__host__ __device__ constexpr int table_ints(int E) { return (E + 1 + 3) & ~3; }
template <int kSub>
__host__ __device__ constexpr int pair_smem(int E) {
    using S = Shape<kSub>;
    return 1024 + S::kStages * S::kAtoms * (S::kATile + kBTile) + 2 * kMaxRows * 4 + 2 * table_ints(E) * 4 + 64 * 4 +
           (int)sizeof(PairBars);
}
static_assert(pair_smem<1>(WQ_INT8_MAX_EXPERTS) <= 227 * 1024 && pair_smem<2>(WQ_INT8_MAX_EXPERTS) <= 227 * 1024,
              "pair kernel shared memory");

__device__ __forceinline__ void tc_mma_i8_pair(bool one, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"((int)one)
        : "memory");
}

// Arrive on this barrier in the CTAs of `mask` once the MMAs issued so far are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(mask)
        : "memory");
}

// 3-D tiled load into this CTA's shared memory, its bytes counted on a barrier
// of the pair's leader (cluster_bar).
__device__ __forceinline__ void tma_load_3d_pair(bool one, uint32_t smem_dst, const void* tmap, uint32_t cluster_bar,
                                                 int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(smem_dst),
        "l"(tmap), "r"(cluster_bar), "r"(x), "r"(y), "r"(z), "r"((int)one)
        : "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

template <int kSub>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<kSub>::kThreads, 1)
    w8a8_pair_kernel(const __grid_constant__ RowMaps tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                     const W8A8Args a, const PairPlan p) {
    using S = Shape<kSub>;
    constexpr int kCh = S::kCh, kAtoms = S::kAtoms, kStages = S::kStages, kATile = S::kATile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* smem_a = smem;
    uint8_t* smem_b = smem + kStages * kAtoms * kATile;
    float* row_scale = reinterpret_cast<float*>(smem_b + kStages * kAtoms * kBTile);  // [2][kMaxRows]
    int* off = reinterpret_cast<int*>(row_scale + 2 * kMaxRows);
    int* cum = off + table_ints(a.E);
    int* warp_part = cum + table_ints(a.E);
    PairBars& bar = *reinterpret_cast<PairBars*>(warp_part + 64);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x & 1u);
    const int worker = (int)(blockIdx.x >> 1), workers = (int)(gridDim.x >> 1);
    const int atoms = (a.K + kKB - 1) / kKB, nkb = (atoms + kAtoms - 1) / kAtoms;
    const bool whole = a.K % kKB == 0;  // two atoms per copy

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmap_w);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar.acc_full[s], 1);
            mbar_init(&bar.acc_empty[s], 2 * kEpiWarps);
        }
        mbar_init(&bar.drain, 1);
        bar.abort_flag = 0;
        fence_mbar_init();
    }
    // Both CTAs run before either allocates: the allocation is one operation of
    // the two, made by a warp of each, and has no limit.  A CTA's blocks start
    // when its SM gets to them, which other kernels' blocks can put off.
    cluster_arrive();
    cluster_wait();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bar.tmem_slot)),
                     "r"((uint32_t)kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    build_tiles(a.offsets, a.E, a.R, p.step, off, cum, warp_part, S::kThreads, a.status);  // ends with __syncthreads
    cluster_arrive();
    cluster_wait();  // both CTAs' barriers are initialised, both have their tensor memory
    tc_fence_after();
    const uint32_t tmem_base = bar.tmem_slot;
    const int total = cum[a.E] * p.n_ct;
    volatile int* abort_flag = &bar.abort_flag;

    if (warp == 0) {
        // ---------------- copy warp (both CTAs) ----------------
        const bool one = elect_one();
        const uint32_t a0 = smem_u32(smem_a), b0 = smem_u32(smem_b);
        const uint32_t full0 = map_rank(smem_u32(bar.full), 0);  // the leader's
        int it = 0;
        for (int t = worker; t < total && !__any_sync(0xffffffffu, *abort_flag); t += workers) {
            const TokenTile w = find_tile(t, p.n_ct, a.E, off, cum, 32);
            const int half = ceil_div(w.n, 32) * 16;  // rows this CTA brings
            const int wrow = w.e * a.N + w.ct * kCh + rank * S::kCtaCh;
            const int xrow = w.row0 + rank * half;
            const CUtensorMap* tx = &tmap_x.m[half / 16 - 1];
            const auto expect = [&](int s, int kb) {
                const int here = whole ? kAtoms : min(kAtoms, atoms - kb * kAtoms);
                if (rank == 0 && one) mbar_arrive_expect_tx(&bar.full[s], (uint32_t)(2 * here * (kATile + half * kKB)));
            };
            const auto load = [&](uint32_t dst, int atom_bytes, const CUtensorMap* map, int s, int kb, int row) {
                if (whole) {
                    tma_load_3d_pair(one, dst, map, full0 + 8 * s, 0, row, kb * kAtoms);
                } else {
                    for (int at = 0; at < kAtoms && kb * kAtoms + at < atoms; ++at)
                        tma_load_3d_pair(one, dst + at * atom_bytes, map, full0 + 8 * s, (kb * kAtoms + at) * kKB, row, 0);
                }
            };
            for (int kb = 0; kb < nkb; ++kb, ++it) {
                const int s = it % kStages;
                if (it >= kStages &&
                    !__all_sync(0xffffffffu, mbar_wait_cluster(&bar.empty[s], (uint32_t)(it / kStages - 1) & 1u, a.status))) {
                    atomicExch(&bar.abort_flag, 1);
                    break;
                }
                expect(s, kb);
                load(a0 + s * kAtoms * kATile, kATile, &tmap_w, s, kb, wrow);
                load(b0 + s * kAtoms * kBTile, half * kKB, tx, s, kb, xrow);
            }
        }
        // before the pair ends, the loads in flight (of both CTAs) land in the
        // leader's count and the leader's last arrivals reach both CTAs
        for (int j = max(0, it - kStages); j < it; ++j) {
            const uint32_t parity = (uint32_t)(j / kStages) & 1u;
            if (rank == 0) mbar_wait_cluster(&bar.full[j % kStages], parity, a.status);
            mbar_wait_cluster(&bar.empty[j % kStages], parity, a.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA warp (leader) ----------------
        if (rank == 0) {
            const bool one = elect_one();
            int it = 0, ti = 0;
            for (int t = worker; t < total && !__any_sync(0xffffffffu, *abort_flag); t += workers, ++ti) {
                const TokenTile w = find_tile(t, p.n_ct, a.E, off, cum, 32);
                const int half = ceil_div(w.n, 32) * 16;
                const uint32_t idesc = mma_idesc_s8(256, 2 * half);
                // accumulator of the tile's (sub)tile j, and how often it was used before
                const auto acc_of = [&](int j) { return kSub == 1 ? ti & 1 : j; };
                const int uses = kSub == 1 ? ti >> 1 : ti;
                bool ok = true;
                for (int kb = 0; ok && kb < nkb; ++kb, ++it) {
                    const int s = it % kStages;
                    ok = __all_sync(0xffffffffu, mbar_wait_cluster(&bar.full[s], (uint32_t)(it / kStages) & 1u, a.status));
                    const uint64_t ad = sw128_kmajor_desc(smem_u32(smem_a + s * kAtoms * kATile));
                    const uint64_t bd = sw128_kmajor_desc(smem_u32(smem_b + s * kAtoms * kBTile));
                    const int here = min(kAtoms, atoms - kb * kAtoms);
#pragma unroll
                    for (int j = 0; j < kSub; ++j) {
                        const int acc = acc_of(j);
                        if (kb == 0 && uses > 0)
                            ok = ok && __all_sync(0xffffffffu, mbar_wait_cluster(&bar.acc_empty[acc], (uint32_t)(uses - 1) & 1u, a.status));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int at = 0; at < kAtoms; ++at) {
                            if (at >= here) break;
#pragma unroll
                            for (int kk = 0; kk < kKB / 32; ++kk)  // descriptors count 16-byte units
                                tc_mma_i8_pair(one, tmem_base + (uint32_t)(acc * kMaxRows),
                                               ad + (at * kATile + j * 128 * kKB + kk * 32) / 16,
                                               bd + (at * half * kKB + kk * 32) / 16, idesc, (kb | at | kk) != 0 ? 1u : 0u);
                        }
                        if (kb == nkb - 1 && one) tc_commit_pair(&bar.acc_full[acc], 3);
                    }
                    if (ok && one) tc_commit_pair(&bar.empty[s], 3);
                }
                if (!ok) {
                    atomicExch(&bar.abort_flag, 1);
                    break;
                }
            }
            if (one) tc_commit_pair(&bar.drain, 1);  // completes once every MMA issued above has
            mbar_wait(&bar.drain, 0u, a.status);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue warps (both CTAs) ----------------
        const int q = warp & 3;            // tensor memory lanes this warp may read
        const int et = threadIdx.x - 64;
        const int part = ((warp - 2) >> 2) & 1;                  // which half of the 64-column groups
        const int j = kSub == 1 ? 0 : (warp - 2) / kEpiWarps;    // which 128 of the CTA's channels
        int ti = 0;
        for (int t = worker; t < total; t += workers, ++ti) {
            const TokenTile w = find_tile(t, p.n_ct, a.E, off, cum, 32);
            const int acc = kSub == 1 ? ti & 1 : j, uses = kSub == 1 ? ti >> 1 : ti;
            float* rs = row_scale + (ti & 1) * kMaxRows;
            for (int i = et; i < w.n; i += S::kEpi) rs[i] = a.xs[w.row0 + i];
            const int c = w.ct * kCh + rank * S::kCtaCh + j * 128 + q * 32 + lane;
            const bool cv = c < a.N;
            const float sw = cv ? __half2float(__ushort_as_half(a.ws[(int64_t)w.e * a.N + c])) : 0.0f;
            if (!named_sync_and(1, S::kEpi, !*abort_flag)) break;
            const bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(&bar.acc_full[acc], (uint32_t)uses & 1u, a.status));
            tc_fence_after();
            if (!ok) {
                atomicExch(&bar.abort_flag, 1);
                continue;  // the next barrier ends the loop for all warps
            }
            const uint32_t dcol = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * kMaxRows);
            for (int c0 = 32 * part; c0 < w.n; c0 += 64) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(dcol + (uint32_t)c0, v);
                tc_wait_ld();
                if (cv)
                    w8a8_store_cols(a.Y, a.y_fp32, (int64_t)(w.row0 + c0) * a.N + c, a.N, sw, rs + c0, v, w.n - c0);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&bar.acc_empty[acc]), 0));
        }
        __syncwarp();
    }

    // ---------------- teardown ----------------
    // the leader's MMAs read both CTAs' shared memory and arrive on both CTAs'
    // barriers: neither ends before the other is done
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"((uint32_t)kTmemCols)
                     : "memory");
    }
}

int max_of(int a, int b) { return a > b ? a : b; }

template <int kSub>
cudaError_t launch_shape(const W8A8Args& a, int step, int pairs, cudaStream_t stream) {
    using S = Shape<kSub>;
    PairPlan p = {};
    p.step = step;
    p.n_ct = ceil_div(a.N, S::kCh);
    const int64_t token_tiles = a.offsets ? (int64_t)(a.E < a.R ? a.E : a.R) + a.R / step : ceil_div(a.R, step);
    const int64_t tiles = token_tiles * p.n_ct;
    if (tiles > 0x3fffffff) return cudaErrorNotSupported;  // tile numbers stay far from overflow

    RowMaps tx = {};
    CUtensorMap tw;
    CUresult cr = encode_tensor_map_k_atoms(&tw, a.qweight, (uint64_t)a.K, (uint64_t)a.E * (uint64_t)a.N, S::kCtaCh, S::kAtoms);
    // one matrix: no tile has more rows than the first
    const int most = ceil_div(ceil_div(a.R, ceil_div(a.R, step)), 32) * 16;
    for (int half = 16; half <= step / 2 && cr == CUDA_SUCCESS; half += 16)
        if (a.offsets || half <= most)
            cr = encode_tensor_map_k_atoms(&tx.m[half / 16 - 1], a.Xq, (uint64_t)a.K, (uint64_t)a.R, half, S::kAtoms);
    if (cr != CUDA_SUCCESS) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> allowed{0};
    const auto kernel = w8a8_pair_kernel<kSub>;
    cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kernel), 227 * 1024, allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = (size_t)pair_smem<kSub>(a.E);
    cfg.stream = stream;
    // no launch attribute: it starts once the kernel ahead has ended (see the top)
    return cudaLaunchKernelEx(&cfg, kernel, tx, tw, a, p);
}

}  // namespace

cudaError_t launch_w8a8_pair(const W8A8Args& a, int num_sms, cudaStream_t stream) {
    // Channels and rows per tile, by the time of all waves.  A k atom of a tile
    // takes as long as its reads from L2 (per CTA 128 bytes per channel, 64 per
    // row) or as its MMAs, 124 of those bytes per row and 256 channels of the
    // tile, whichever is longer.  Wide tiles read less but leave the tensor pipe
    // idle between tiles, and a coarser last wave: for one deep matrix only.
    // (us, narrow / wide: 8192 x 1024 x 8192 50.7 / 45.1, 4096 x 4096 x 11008
    // 122 / 117, 8192 x 28672 x 8192 back to back 1416 / 1328; but 4096 x 11008 x
    // 4096 118 / 121, and 8 experts of 4096 x 11008 with 2048 rows each 543 / 555.)
    // Fewer rows than the most have to win by 3 %: they read more for the same
    // MMAs, which the power limit charges (8192 x 28672 x 8192 in wide tiles of
    // 224 / 256 rows: 1180 / 1203 from rest, 1360 / 1325 back to back).
    const int pairs = num_sms / 2;
    int sub = 1, step = kMaxRows;
    int64_t best = -1;
    for (int u = 1; u <= 2 && !a.offsets; ++u)
        for (int rows = kMaxRows; rows >= 32 && (u == 1 || a.K >= 8192); rows -= 32) {
            const int64_t tiles = (int64_t)ceil_div(a.R, rows) * ceil_div(a.N, 256 * u);
            const int64_t atom = max_of(128 * 128 * u + 64 * rows, 124 * rows * u);
            const int64_t cost = (tiles + pairs - 1) / pairs * atom;
            if (best < 0 || cost * 100 < best * (rows == kMaxRows ? 100 : 97)) {
                best = cost;
                sub = u;
                step = rows;
            }
        }
    return sub == 1 ? launch_shape<1>(a, step, pairs, stream) : launch_shape<2>(a, step, pairs, stream);
}

}  // namespace wq
