// NVFP4 product for large batches: CTA pairs on 256 x 256 tiles.
//
// What bounds it is the FP4 rate of the tensor cores, so the design keeps
// them fed: a pair of CTAs issues one 256 x 256 x 64 product over both SMs
// (each reads half of the weight tile, which halves the traffic into shared
// memory), five stages of 256 elements of K are in flight, CTAs are
// persistent, and the sums of one tile leave tensor memory while the next
// tile is computed.
//
// Tensor memory (512 columns): the sums of even tiles in columns 0-255, of
// odd tiles in 192-447, the scales behind.  Two whole tiles and the scales do
// not fit, so neighbours share 64 columns: the epilogue takes those first and
// the next tile starts as soon as they are out, long before the rest is.
//
// Warps of a CTA: 0 copies, 1 issues products (in the pair's first CTA),
// 2-5 take sums out (32 rows each).
#include <algorithm>

#include "gemma_nq.h"
#include "gnq_linear.cuh"

namespace gnq {
namespace {

constexpr int kPairTile = 256;
constexpr int kPairStages = 5;
constexpr uint32_t kHalf = 128 * kStageK / 2;                       // 128 rows of codes of one stage
constexpr uint32_t kPairStage = 2 * kHalf + 3 * kBytesSf;           // per CTA
constexpr uint32_t kAccCols = 192, kSfxCol = 448, kSfwCol = 464;    // second tile, scales

struct PairParams {
    LinearParams p;
    int m_tiles, n_tiles;
    int vec;  // bytes of an output row's widest aligned store: 32, 16 or 0 (single values)
};

__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Tile load into this CTA, completing on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Arrives on the barrier at this offset in both CTAs of the pair once every
// copy and product issued so far is done.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 32 sums of one row to y[n .. n + 32): alpha, bias, one rounding.
template <typename O, typename B>
__device__ __forceinline__ void store_row32(const PairParams &pp, int64_t m, int n, const uint32_t (&acc)[32],
                                            float alpha) {
    const LinearParams &p = pp.p;
    if (m >= p.M || n >= p.N) return;
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float b = p.bias && n + i < p.N ? OutType<B>::bias(__ldg(p.bias + n + i)) : 0.f;
        v[i] = fmaf(__uint_as_float(acc[i]), alpha, b);
    }
    constexpr int PER = 4 / sizeof(O);  // values per 32-bit word
    uint32_t w[32 / PER];
#pragma unroll
    for (int i = 0; i < 32 / PER; ++i) {
        if constexpr (PER == 1) w[i] = __float_as_uint(v[i]);
        else w[i] = Act<O>::pack2(v[2 * i], v[2 * i + 1]);
    }
    O *o = static_cast<O *>(p.y) + m * p.N + n;
    if (pp.vec && n + 32 <= p.N) {
#pragma unroll
        for (int i = 0; i < 32 / PER; i += 8) {
            const uint4 a = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            const uint4 b = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
            if (pp.vec == 32) {
                st_v8(reinterpret_cast<uint32_t *>(o) + i, a, b);
            } else {
                st_v4(reinterpret_cast<uint32_t *>(o) + i, a);
                st_v4(reinterpret_cast<uint32_t *>(o) + i + 4, b);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (n + i < p.N) {
                if constexpr (PER == 1) o[i] = v[i];
                else o[i] = OutType<O>::round(v[i]);
            }
    }
}

template <typename O, typename B>
__global__ void __launch_bounds__(192) linear_pair_kernel(
    const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
    const __grid_constant__ CUtensorMap map_xs, const __grid_constant__ CUtensorMap map_ws,
    const __grid_constant__ PairParams pp) {
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kPairStages + 3];
    __shared__ __align__(16) uint4 topup[kPairStages];
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;

    const LinearParams &p = pp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t base = ((uint32_t)__cvta_generic_to_shared(dyn) + 1023u) & ~1023u;
    const uint32_t bar0 = (uint32_t)__cvta_generic_to_shared(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };                   // first CTA's: both halves landed
    auto empty = [&](int s) { return bar0 + 8u * (kPairStages + s); };  // each CTA's: products done with it
    const uint32_t acc_full = bar0 + 8u * (2 * kPairStages);            // each CTA's: a tile's sums are ready
    const uint32_t shared_free = acc_full + 8;                          // first CTA's: the shared columns are out
    const uint32_t done = acc_full + 16;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(shared_free, 8);
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        failed = 0;
    }
    if (warp == 1) {
        tmem_alloc<2>((uint32_t)__cvta_generic_to_shared(&tmem_slot), 512);
        tmem_relinquish<2>();
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait();  // the peer's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    pdl_wait();  // inputs may come from the preceding grid, outputs may still be read by it
    pdl_trigger();

    const int KT = (p.K64 + 3) / 4;
    const int tiles = pp.m_tiles * pp.n_tiles, G = gridDim.x / 2;
    // Bands of 8 tile rows, walked column by column: the tiles in flight at
    // one time share few rows and columns.
    auto tile_at = [&](int i, int &mt, int &nt) {
        const int band = i / (8 * pp.n_tiles), in = i - band * 8 * pp.n_tiles;
        const int rows = min(8, pp.m_tiles - 8 * band);
        nt = in / rows;
        mt = 8 * band + in - nt * rows;
    };
    auto gave_up = [&] { return *(volatile int *)&failed != 0; };
    auto give_up = [&] {
        atomicOr(p.err, (unsigned)DEVERR_WAIT_TIMEOUT);
        *(volatile int *)&failed = 1;
    };

    if (warp == 0) {
        // ---- copies ----
        int it = 0;
        for (int i = blockIdx.x / 2; i < tiles && !gave_up(); i += G) {
            int mt, nt;
            tile_at(i, mt, nt);
            for (int kt = 0; kt < KT; ++kt, ++it) {
                const int s = it % kPairStages;
                if (it >= kPairStages && !mbar_wait_bounded(empty(s), (it / kPairStages - 1) & 1, p.wait_limit)) {
                    give_up();
                    break;
                }
                if (elect_one()) {
                    const uint32_t at = base + kPairStage * s, bar = map_to_cta(full(s), 0);
                    if (rank == 0) mbar_expect_tx(full(s), 2 * kPairStage + p.tx_extra);
                    tma_load_pair(at, &map_x, kt * 128, mt * kPairTile + 128 * rank, bar);
                    tma_load_pair(at + kHalf, &map_w, kt * 128, nt * kPairTile + 128 * rank, bar);
                    tma_load_pair(at + 2 * kHalf, &map_xs, 0, (2 * mt + rank) * p.K64 + 4 * kt, bar);
                    tma_load_pair(at + 2 * kHalf + kBytesSf, &map_ws, 0, 2 * nt * p.K64 + 4 * kt, bar);
                    tma_load_pair(at + 2 * kHalf + 2 * kBytesSf, &map_ws, 0, (2 * nt + 1) * p.K64 + 4 * kt, bar);
                }
                __syncwarp();
            }
        }
        // Every copy has landed before the shared memory goes away (test
        // hook: with the bytes that its announcement lacks).
        if (rank == 0 && lane == 0)
            for (int j = max(0, it - kPairStages); j < it; ++j) {
                const int s = j % kPairStages;
                if (mbar_wait_bounded(full(s), (j / kPairStages) & 1, p.wait_limit)) continue;
                give_up();
                if (p.tx_extra) bulk_g2s((uint32_t)__cvta_generic_to_shared(&topup[s]), p.w_sf, p.tx_extra, full(s));
                mbar_wait_bounded(full(s), (j / kPairStages) & 1, p.wait_limit);
            }
    } else if (warp == 1 && rank == 0) {
        // ---- products ----
        constexpr uint32_t idesc = idesc_nvfp4(256, 256);
        int it = 0, j = 0;
        bool good = true;
        for (int i = blockIdx.x / 2; good && i < tiles; i += G, ++j) {
            if (j > 0 && !mbar_wait_bounded(shared_free, (j - 1) & 1, p.wait_limit)) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + kAccCols * (j & 1);
            for (int kt = 0; kt < KT; ++kt, ++it) {
                const int s = it % kPairStages;
                if (!mbar_wait_bounded(full(s), (it / kPairStages) & 1, p.wait_limit) || gave_up()) {
                    give_up();
                    good = false;
                    break;
                }
                tc_fence_after();
                const int nk = p.K64 - 4 * kt;
                if (elect_one()) {
                    const uint32_t at = base + kPairStage * s, sf = at + 2 * kHalf;
                    const uint64_t a = desc_sw128(at), b = desc_sw128(at + kHalf);
                    const uint64_t sx = desc_scales(sf), sw0 = desc_scales(sf + kBytesSf),
                                   sw1 = desc_scales(sf + 2 * kBytesSf);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k < nk) {
                            cp_scales<2>(tmem + kSfxCol + 4 * k, sx + 32 * k);
                            cp_scales<2>(tmem + kSfwCol + 8 * k, sw0 + 32 * k);
                            cp_scales<2>(tmem + kSfwCol + 8 * k + 4, sw1 + 32 * k);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < nk)
                            mma_nvfp4<2>(acc, a + 2 * k, b + 2 * k, idesc, tmem + kSfxCol + 4 * k,
                                         tmem + kSfwCol + 8 * k, kt > 0 || k > 0);
                    tc_commit_pair(empty(s));
                    if (kt == KT - 1) tc_commit_pair(acc_full);
                }
                __syncwarp();
            }
        }
        // every product is done before tensor memory goes away
        if (elect_one()) tc_commit_pair(done);
        __syncwarp();
        if (!mbar_wait_bounded(done, 0, p.wait_limit)) give_up();
    } else if (warp == 1) {
        if (!mbar_wait_bounded(done, 0, 4 * p.wait_limit)) give_up();  // the first CTA's last arrival here
    } else if (warp >= 2) {
        // ---- sums out ----
        const float alpha = __ldg(p.alpha);
        const int quad = warp & 3;
        const uint32_t lanes = (uint32_t)quad << 21;  // 32 lanes per warp, lane number in bits 16-31
        const uint32_t free_bar = map_to_cta(shared_free, 0);
        int j = 0;
        for (int i = blockIdx.x / 2; i < tiles; i += G, ++j) {
            int mt, nt;
            tile_at(i, mt, nt);
            const bool ok = mbar_wait_bounded(acc_full, j & 1, 2 * p.wait_limit) && !gave_up();
            if (!__all_sync(0xffffffffu, ok)) {
                give_up();
                break;
            }
            tc_fence_after();
            const int64_t m = (int64_t)mt * kPairTile + 128 * rank + 32 * quad + lane;
            const int n0 = nt * kPairTile;
            const uint32_t acc = tmem + kAccCols * (j & 1) + lanes;
            const int first = j & 1 ? 0 : 192;  // the tile's columns that it shares
            uint32_t v[32], u[32];
            tmem_ld32(acc + first, v);
            tmem_ld32(acc + first + 32, u);
            tmem_wait(v);
            tmem_wait(u);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_remote(free_bar);
            store_row32<O, B>(pp, m, n0 + first, v, alpha);
            store_row32<O, B>(pp, m, n0 + first + 32, u, alpha);
            const int rest = j & 1 ? 64 : 0;
            for (int c = rest; c < rest + 192; c += 32) {
                __syncwarp();
                tmem_ld32(acc + c, v);
                tmem_wait(v);
                store_row32<O, B>(pp, m, n0 + c, v, alpha);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait();  // the peer's copies and barriers are no longer in use
    if (warp == 1) tmem_dealloc<2>(tmem, 512);
}

template <typename O, typename B>
cudaError_t launch_pair(const CUtensorMap (&m)[4], const PairParams &pp, int64_t grid, cudaStream_t s) {
    auto fn = linear_pair_kernel<O, B>;
    const cudaError_t e = opt_in_dynamic_smem(reinterpret_cast<const void *>(fn));
    if (e != cudaSuccess) return e;
    return launch(fn, grid, 192, 1024 + kPairStages * kPairStage, 2, s, m[0], m[1], m[2], m[3], pp);
}

}  // namespace

cudaError_t launch_linear_pair(const LinearParams &p, const void *q, const void *w_q, int out_type, int bias_type,
                               int sms, cudaStream_t s) {
    PairParams pp = {p, 0, 0, 0};
    const int64_t K = (int64_t)p.K64 * 64;
    const int64_t mt = (p.M + kPairTile - 1) / kPairTile, nt = (p.N + kPairTile - 1) / kPairTile;
    const int64_t x_rows = (p.M + 127) / 128 * p.K64, w_rows = (p.N + 127) / 128 * (int64_t)p.K64;
    if (mt * nt > 0x3FFFFFFF || x_rows > 0x7FFFFFFF || w_rows > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    pp.m_tiles = (int)mt;
    pp.n_tiles = (int)nt;
    const int64_t row_bytes = (int64_t)p.N * (out_type == GNQ_FP32 ? 4 : 2);
    pp.vec = row_bytes % 32 == 0 && aligned(p.y, 32) ? 32 : row_bytes % 16 == 0 ? 16 : 0;
    CUtensorMap m[4];
    if (!encode_codes(&m[0], q, p.M, K, 128) || !encode_codes(&m[1], w_q, p.N, K, 128) ||
        !encode_scales(&m[2], p.x_sf, x_rows) || !encode_scales(&m[3], p.w_sf, w_rows))
        return cudaErrorInvalidValue;
    const int64_t grid = 2 * std::min<int64_t>(mt * nt, sms / 2);
    if (out_type == GNQ_BF16) return launch_pair<__nv_bfloat16, __nv_bfloat16>(m, pp, grid, s);
    if (out_type == GNQ_FP16) return launch_pair<__half, __half>(m, pp, grid, s);
    if (bias_type == GNQ_FP16) return launch_pair<float, __half>(m, pp, grid, s);
    return launch_pair<float, __nv_bfloat16>(m, pp, grid, s);
}

}  // namespace gnq
