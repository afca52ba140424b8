// w8a8_device.cuh -- device pieces shared by the W8A8 kernels (sm_100a only):
// INT8 tcgen05.mma, cluster and distributed shared memory helpers, and the
// table that turns a tile number into rows and channels of an expert.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/wq_int8.h"
#include "wq_device.cuh"
#include "wq_tcgen05.cuh"

namespace wq {

// Instruction descriptor: D int32, A and B signed 8 bit, both K-major, N, M.
__host__ __device__ constexpr uint32_t mma_idesc_s8(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_i8(bool one, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"((int)one)
        : "memory");
}

// One lane of a converged warp.  The copy and MMA warps run their loops as whole
// warps and let this lane's predicate pick the thread that issues: addresses and
// descriptors then stay in uniform registers (a loop inside "if (lane == 0)"
// took 90 to 135 cycles per MMA and about 200 per copy).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// ------------------------------------------------------------------------
// Clusters and distributed shared memory
// ------------------------------------------------------------------------

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t smem_addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
    return r;
}

// 16-byte store into another CTA's shared memory, counted on its mbarrier.
__device__ __forceinline__ void st_async_v4(uint32_t cluster_addr, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3,
                                            uint32_t cluster_bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     cluster_addr),
                 "r"(v0), "r"(v1), "r"(v2), "r"(v3), "r"(cluster_bar)
                 : "memory");
}

// Bounded wait on an mbarrier that another CTA of the cluster arrives on, or
// whose bytes or commits come from one: what that CTA wrote before is seen
// (mbar_wait acquires from this CTA's own threads only).
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}

// (as mbar_test_wait: a completed phase is seen at once)
__device__ __forceinline__ bool mbar_test_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint32_t* status) {
    if (mbar_test_wait_cluster(bar, parity)) return true;
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        for (int i = 0; i < 16; ++i)
            if (mbar_try_wait_cluster(bar, parity)) return true;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            raise_flag(status, kFlagTimeout);
            return false;
        }
    }
}

// 3-D tiled load global -> shared, completion counted on `bar` (bytes).
__device__ __forceinline__ void tma_load_3d(bool one, uint32_t smem_dst, const void* tmap, uint32_t bar, int32_t x,
                                            int32_t y, int32_t z) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];\n\t}" ::"r"(smem_dst),
        "l"(tmap), "r"(bar), "r"(x), "r"(y), "r"(z), "r"((int)one)
        : "memory");
}

// The same box into L2 only.  L2 is where all SMs' writes meet, so what another
// kernel writes there later is still read fresh.
__device__ __forceinline__ void tma_prefetch_3d(bool one, const void* tmap, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n\t}" ::"l"(tmap),
        "r"(x), "r"(y), "r"(z), "r"((int)one)
        : "memory");
}

// named_sync that tells every thread whether `go` held in all of them: warps
// that may have given up at different times leave a loop together.
__device__ __forceinline__ bool named_sync_and(int id, int nthreads, bool go) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
        "bar.red.and.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(all)
        : "r"(id), "r"(nthreads), "r"((uint32_t)go)
        : "memory");
    return all != 0;
}

// ------------------------------------------------------------------------
// Tiles.  Expert e holds rows off[e] .. off[e+1] - 1 in cum[e+1] - cum[e]
// token tiles; tile t of the product is one token tile times one channel
// tile, the experts in order, an expert's token tiles next to each other (they
// read the same weights).
// ------------------------------------------------------------------------

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

struct TokenTile {
    int row0;   // first row
    int n;      // rows, >= 1
    int ct;     // channel tile
    int e;      // expert
};

// off/cum: shared memory, E + 1 entries each.  Built by all `nthreads` threads
// of the block (a multiple of 32, at most 1024); ends with a __syncthreads.
// step: most rows of a tile.
__device__ __forceinline__ void build_tiles(const int32_t* offsets, int E, int R, int step, int* off, int* cum,
                                            int* warp_part, int nthreads, uint32_t* status) {
    if (!offsets) {
        if (threadIdx.x == 0) {
            off[0] = 0;
            off[1] = R;
            cum[0] = 0;
            cum[1] = ceil_div(R, step);
        }
        __syncthreads();
        return;
    }
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nwarps = nthreads >> 5;
    const int per = (E + nthreads) / nthreads;  // ceil((E + 1) / nthreads)
    const int i0 = t * per, i1 = min(i0 + per, E + 1);
    // running maximum of the clamped offsets: they never decrease below
    int m = 0;
    bool bad = false;
    for (int i = i0; i < i1; ++i) {
        const int v = offsets[i];
        const int c = min(max(v, 0), R);
        bad |= v != c || c < m;
        m = max(m, c);
        off[i] = m;
    }
    int inc = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc = max(inc, u);
    }
    int before = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) before = 0;
    if (lane == 31) warp_part[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before = max(before, warp_part[w]);
    for (int i = i0; i < i1; ++i) {
        bad |= off[i] < before;
        off[i] = max(off[i], before);
    }
    if (bad && blockIdx.x == 0) raise_flag(status, WQ_DEVFLAG_INDEX);
    __syncthreads();
    // prefix sums of the experts' tile counts (entry i: tiles of experts < i)
    int s = 0;
    for (int i = i0; i < i1 && i < E; ++i) s += ceil_div(off[i + 1] - off[i], step);
    inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    before = inc - s;
    if (lane == 31) warp_part[nwarps + warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += warp_part[nwarps + w];
    for (int i = i0; i < i1; ++i) {
        cum[i] = before;
        if (i < E) before += ceil_div(off[i + 1] - off[i], step);
    }
    __syncthreads();
}

// Tile t (0 <= t < cum[E] * n_ct).  An expert's rows are spread evenly over its
// token tiles, in multiples of `unit` rows.
__device__ __forceinline__ TokenTile find_tile(int t, int n_ct, int E, const int* off, const int* cum, int unit) {
    const int q = t / n_ct;
    int lo = 0, hi = E;  // cum[lo] <= q < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= q)
            lo = mid;
        else
            hi = mid;
    }
    const int mt = cum[lo + 1] - cum[lo];
    const int l = t - cum[lo] * n_ct;
    TokenTile r;
    r.e = lo;
    r.ct = l / mt;
    const int tt = l - r.ct * mt;
    const int cnt = off[lo + 1] - off[lo];
    const int each = ceil_div(ceil_div(cnt, mt), unit) * unit;  // <= step, so no tile is empty
    r.row0 = off[lo] + tt * each;
    r.n = min(each, off[lo + 1] - r.row0);
    return r;
}

// The output value: exact integer sum, weight scale, token scale.
__device__ __forceinline__ float w8a8_value(int sum, float w, float s) {
    return __fmul_rn(__fmul_rn(__int2float_rn(sum), w), s);
}

__device__ __forceinline__ void w8a8_store(void* Y, int y_fp32, int64_t i, float y) {
    if (y_fp32)
        static_cast<float*>(Y)[i] = y;
    else
        static_cast<__nv_bfloat16*>(Y)[i] = __float2bfloat16_rn(y);
}

// The first n of COLS columns (rows of the output) of this thread's channel:
// sums v, row scales rs in shared memory, first output at index `at`.  A warp
// writes 32 neighbouring channels of a row per column.
template <int COLS, typename T>
__device__ __forceinline__ void w8a8_store_typed(T* p, int N, float sw, const float* rs, const uint32_t (&v)[COLS],
                                                 int n) {
    if (n >= COLS) {  // no test per column: 75 -> about 10 cycles per column and warp
        float s[COLS];
#pragma unroll
        for (int j = 0; j < COLS; j += 4) *reinterpret_cast<float4*>(s + j) = *reinterpret_cast<const float4*>(rs + j);
#pragma unroll
        for (int j = 0; j < COLS; ++j, p += N) {
            const float y = w8a8_value((int)v[j], sw, s[j]);
            if constexpr (sizeof(T) == 4)
                *p = y;
            else
                *p = __float2bfloat16_rn(y);
        }
    } else {
#pragma unroll
        for (int j = 0; j < COLS; ++j, p += N) {
            if (j < n) {
                const float y = w8a8_value((int)v[j], sw, rs[j]);
                if constexpr (sizeof(T) == 4)
                    *p = y;
                else
                    *p = __float2bfloat16_rn(y);
            }
        }
    }
}

template <int COLS>
__device__ __forceinline__ void w8a8_store_cols(void* Y, int y_fp32, int64_t at, int N, float sw, const float* rs,
                                                const uint32_t (&v)[COLS], int n) {
    if (y_fp32)
        w8a8_store_typed(static_cast<float*>(Y) + at, N, sw, rs, v, n);
    else
        w8a8_store_typed(static_cast<__nv_bfloat16*>(Y) + at, N, sw, rs, v, n);
}

}  // namespace wq
