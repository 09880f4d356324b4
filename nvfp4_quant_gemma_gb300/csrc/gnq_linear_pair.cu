// NVFP4 product for large batches: CTA pairs on 256 x 256 tiles.
//
// A pair of CTAs issues one 256 x 256 x 64 product over both SMs, each with
// half of the weight tile in its shared memory; five stages of 256 elements of
// K are in flight, CTAs are persistent, and the sums of one tile leave tensor
// memory while the next tile is computed.
//
// What bounds it: a stage is 512 cycles of the tensor cores but 38 912 bytes
// into each SM, and 608 cycles at 64 bytes a cycle is what a stage takes with
// the scale copies into tensor memory left out (650 with them; on 40 pairs as
// on 76, so it is the SM's intake, not the L2).  A 256 x 384 tile would take in 768
// cycles' worth for 768 of products; with its scales it needs 448 columns of
// tensor memory, so one fits, but not the next tile's sums beside those on their
// way out.  Which of the two costs more has not been measured.  The rest is the
// hand-over between tiles, about 1300 cycles.  4864 x 8192 x 16384: 188 us, 6.9
// PFLOP/s; 8192 x 8192 x 5120 (14 rounds for 13.5 of tiles): 114 us, 6.0 PFLOP/s.
//
// Tensor memory (512 columns): the sums of even tiles in columns 0-255, of
// odd tiles in 192-447, the scales behind.  Two whole tiles and the scales do
// not fit, so neighbours share 64 columns: the epilogue takes those first and
// the next tile starts as soon as they are out, long before the rest is.
//
// A row of the output tile is 128 bytes at a time: each of the eight epilogue
// warps packs 32 rows of a chunk into shared memory and a tile store writes
// it as whole lines (stores straight from the registers touch 32 rows per
// instruction: 4864 x 8192 x 512 took 58 us with them).  An output whose rows
// are not 16-byte aligned leaves from there row by row.
//
// Warps of a CTA: 0 copies, 1 issues products (in the pair's first CTA),
// 2-9 take sums out: two warps for each 32 rows, chunks in turn.
#include <algorithm>

#include "gemma_nq.h"
#include "gnq_linear.cuh"

namespace gnq {
namespace {

constexpr int kPairTile = 256;   // tokens and weight rows of a tile
constexpr int kPairStages = 5;
constexpr int kBand = 4;                                            // tile rows of a band
constexpr uint32_t kHalf = 128 * kStageK / 2;                       // 128 rows of codes of one stage
constexpr uint32_t kPairStage = 2 * kHalf + 3 * kBytesSf;           // per CTA
constexpr uint32_t kChunk = 32 * 128;                               // 32 rows x 128 bytes of output
constexpr uint32_t kPairSmem = 1024 + kPairStages * kPairStage + 8 * kChunk;
constexpr uint32_t kAccCols = 192, kSfxCol = 448, kSfwCol = 464;    // second tile, scales

struct PairParams {
    LinearParams p;
    int m_tiles, n_tiles;
    bool tiled;     // rows of y are 16-byte aligned: tile stores
    bool bias16;    // the bias is 16-byte aligned
};

// Result of 32 sums of one row at columns n .. n + 31: alpha and bias.
template <typename B>
__device__ __forceinline__ void scale_bias32(const PairParams &pp, int n, const uint32_t (&acc)[32], float alpha,
                                             float *v) {
    const LinearParams &p = pp.p;
    if (!p.bias) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(acc[i]) * alpha;
        return;
    }
    float b[32];
    if (pp.bias16 && n + 32 <= p.N) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) Act<B>::unpack(ld_weight(p.bias + n + i), &b[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) b[i] = n + i < p.N ? OutType<B>::bias(ld_u16(p.bias + n + i)) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(acc[i]), alpha, b[i]);
}

// One chunk: 32 rows (one per lane) x 128 bytes of y from column n, of the
// sums in `acc` (32 or 64 columns).  buf: this warp's shared memory chunk.
template <typename O, typename B, int COLS>
__device__ __forceinline__ void store_chunk(const PairParams &pp, const CUtensorMap *map_y, uint32_t buf, int64_t m0,
                                            int n, const uint32_t (*acc)[32], float alpha, int lane) {
    const LinearParams &p = pp.p;
    float v[COLS];
#pragma unroll
    for (int h = 0; h < COLS / 32; ++h) scale_bias32<B>(pp, n + 32 * h, acc[h], alpha, v + 32 * h);
    constexpr int PER = COLS / 8;  // values per 16 bytes
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint4 w;
        if constexpr (PER == 8) w = pack8<O>(&v[8 * i]);
        else w = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                            __float_as_uint(v[4 * i + 3]));
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(buf + 128u * lane + 16u * (i ^ (lane & 7))),
                     "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                     : "memory");
    }
    if (pp.tiled) {
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (m0 < p.M && n < p.N) tma_store_2d(map_y, n, (int)m0, buf);
            tma_store_commit();  // a group per chunk, empty or not: the buffer is free by count
        }
    } else {
        // rows of y that a tile store cannot take: each in one go of the warp,
        // a word per lane (two values that are stored apart where N is odd)
        __syncwarp();
        constexpr int W = 4 / sizeof(O);  // values per word
        const int col = n + W * lane, live = (int)min((int64_t)32, p.M - m0);
        O *o = static_cast<O *>(p.y) + m0 * p.N + col;
        for (int r0 = 0; r0 < live; r0 += 4) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + k;
                asm volatile("ld.shared.u32 %0, [%1];"
                             : "=r"(w[k])
                             : "r"(buf + 128u * r + 16u * ((lane >> 2) ^ (r & 7)) + 4u * (lane & 3)));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k, o += p.N) {
                if (r0 + k >= live) break;
                if (W == 1 || p.N % 2 == 0) {
                    if (col < p.N) *reinterpret_cast<uint32_t *>(o) = w[k];
                } else {
                    uint16_t *h = reinterpret_cast<uint16_t *>(o);
                    if (col < p.N) h[0] = (uint16_t)w[k];
                    if (col + 1 < p.N) h[1] = (uint16_t)(w[k] >> 16);
                }
            }
        }
    }
    __syncwarp();
}

template <typename O, typename B>
__global__ void __launch_bounds__(320) linear_pair_kernel(
    const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
    const __grid_constant__ CUtensorMap map_xs, const __grid_constant__ CUtensorMap map_ws,
    const __grid_constant__ CUtensorMap map_y, const __grid_constant__ PairParams pp) {
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
        mbar_init(shared_free, 16);
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
    // Bands of tile rows, walked column by column: the tiles in flight at one
    // time share few rows and columns.
    auto tile_at = [&](int i, int &mt, int &nt) {
        const int band = i / (kBand * pp.n_tiles), in = i - band * kBand * pp.n_tiles;
        const int rows = min(kBand, pp.m_tiles - kBand * band);
        nt = in / rows;
        mt = kBand * band + in - nt * rows;
    };
    auto gave_up = [&] { return *(volatile int *)&failed != 0; };
    auto give_up = [&] {
        atomicOr(p.err, (unsigned)DEVERR_WAIT_TIMEOUT);
        *(volatile int *)&failed = 1;
    };

    if (warp == 0) {
        // ---- copies ----
        int it = 0, s = 0;
        uint32_t parity = 1;  // of the wait on `empty`: passes at once in the first round
        const uint32_t x_row = 128 * rank;
        for (int i = blockIdx.x / 2; i < tiles && !__any_sync(0xffffffffu, gave_up()); i += G) {
            int mt, nt;
            tile_at(i, mt, nt);
            const int x0 = mt * kPairTile + x_row, w0 = nt * kPairTile + x_row;
            const int xs = (2 * mt + rank) * p.K64, ws = 2 * nt * p.K64;
            for (int kt = 0; kt < KT; ++kt, ++it) {
                if (!warp_wait_bounded(empty(s), parity, p.wait_limit)) {
                    give_up();
                    break;
                }
                if (elect_one()) {
                    const uint32_t at = base + kPairStage * s, bar = map_to_cta(full(s), 0);
                    if (rank == 0) mbar_expect_tx(full(s), 2 * kPairStage + p.tx_extra);
                    tma_load_pair(at, &map_x, kt * 128, x0, bar);
                    tma_load_pair(at + kHalf, &map_w, kt * 128, w0, bar);
                    tma_load_pair(at + 2 * kHalf, &map_xs, 0, xs + 4 * kt, bar);
                    tma_load_pair(at + 2 * kHalf + kBytesSf, &map_ws, 0, ws + 4 * kt, bar);
                    tma_load_pair(at + 2 * kHalf + 2 * kBytesSf, &map_ws, 0, ws + p.K64 + 4 * kt, bar);
                }
                __syncwarp();
                if (++s == kPairStages) s = 0, parity ^= 1;
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
        int j = 0, s = 0;
        uint32_t parity = 0;
        bool good = true;
        for (int i = blockIdx.x / 2; good && i < tiles; i += G, ++j) {
            if (j > 0 && !warp_wait_bounded(shared_free, (j - 1) & 1, p.wait_limit)) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + kAccCols * (j & 1);
            for (int kt = 0; kt < KT; ++kt) {
                // (under the test hook a stage may complete late, by the copy
                // that makes up for the announcement)
                if (!warp_wait_bounded(full(s), parity, p.wait_limit) ||
                    (p.tx_extra && __any_sync(0xffffffffu, gave_up()))) {
                    give_up();
                    good = false;
                    break;
                }
                tc_fence_after();
                const int nk = p.K64 - 4 * kt;
                if (elect_one()) {
                    const uint32_t at = (base >> 4) + (kPairStage >> 4) * s;
                    auto step = [&](int k) {
                        cp_scales<2>(tmem + kSfxCol + 4 * k, desc_scales(at + (2 * kHalf + 512 * k) / 16));
                        cp_scales<2>(tmem + kSfwCol + 8 * k, desc_scales(at + (2 * kHalf + kBytesSf + 512 * k) / 16));
                        cp_scales<2>(tmem + kSfwCol + 8 * k + 4,
                                     desc_scales(at + (2 * kHalf + 2 * kBytesSf + 512 * k) / 16));
                        mma_nvfp4<2>(acc, desc_sw128(at + 2 * k), desc_sw128(at + kHalf / 16 + 2 * k), idesc,
                                     tmem + kSfxCol + 4 * k, tmem + kSfwCol + 8 * k, kt > 0 || k > 0);
                    };
                    if (nk >= 4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) step(k);
                    } else {
                        for (int k = 0; k < nk; ++k) step(k);
                    }
                    tc_commit_pair(empty(s));
                    if (kt == KT - 1) tc_commit_pair(acc_full);
                }
                __syncwarp();
                if (++s == kPairStages) s = 0, parity ^= 1;
            }
        }
        // every product is done before tensor memory goes away
        if (elect_one()) tc_commit_pair(done);
        __syncwarp();
        if (!mbar_wait_bounded(done, 0, p.wait_limit)) give_up();
    } else if (warp >= 2) {
        // ---- sums out ----
        // Warps 2-5 take the shared columns of a tile first and then the
        // third chunk of 64, warps 6-9 the second and the fourth.
        const float alpha = ld_f32(p.alpha);
        const int quad = warp & 3, set = (warp - 2) >> 2;
        const uint32_t lanes = (uint32_t)quad << 21;  // 32 lanes per warp, lane number in bits 16-31
        const uint32_t free_bar = map_to_cta(shared_free, 0);
        const uint32_t buf = base + kPairStages * kPairStage + kChunk * (warp - 2);
        auto out_chunk = [&](int64_t m0, int n, const uint32_t (*acc)[32], auto cols) {
            if (lane == 0) tma_store_wait<0>();
            __syncwarp();
            store_chunk<O, B, decltype(cols)::value>(pp, &map_y, buf, m0, n, acc, alpha, lane);
        };
        int j = 0;
        for (int i = blockIdx.x / 2; i < tiles; i += G, ++j) {
            int mt, nt;
            tile_at(i, mt, nt);
            // the tile's bias on its way while the products finish
            if (p.bias && lane < 4 && nt * kPairTile + 64 * lane < p.N)
                prefetch_l1_line(p.bias + nt * kPairTile + 64 * lane);
            const bool ok = mbar_wait_bounded(acc_full, j & 1, 2 * p.wait_limit) && !(p.tx_extra && gave_up());
            if (!__all_sync(0xffffffffu, ok)) {
                give_up();
                break;
            }
            tc_fence_after();
            const int64_t m0 = (int64_t)mt * kPairTile + 128 * rank + 32 * quad;
            const int n0 = nt * kPairTile;
            const uint32_t acc = tmem + kAccCols * (j & 1) + lanes;
            // the next tile may start once the shared columns of this one are
            // out (first set) and all of the one before, whose place it takes
            // (second set: it has come here)
            if (set == 1 && lane == 0) arrive_remote(free_bar);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int turn = 2 * h + set;  // chunk in the order of taking: the shared one is the first
                const int c = j & 1 ? 64 * turn : 64 * ((turn + 3) & 3);
                uint32_t v[2][32];
                tmem_ld32(acc + c, v[0]);
                tmem_ld32(acc + c + 32, v[1]);
                tmem_wait(v[0]);
                tmem_wait(v[1]);
                if (turn == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_remote(free_bar);
                }
                if constexpr (sizeof(O) == 2) {
                    out_chunk(m0, n0 + c, v, std::integral_constant<int, 64>{});
                } else {
                    out_chunk(m0, n0 + c, v, std::integral_constant<int, 32>{});
                    out_chunk(m0, n0 + c + 32, v + 1, std::integral_constant<int, 32>{});
                }
            }
            tc_fence_before();  // this tile's reads are done before the arrival at the next
            __syncwarp();
        }
        tma_store_wait<0>();  // shared memory is read before it goes away
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // the first CTA's last arrival here, before these barriers go away
    if (rank == 1 && warp == 1 && !mbar_wait_bounded(done, 0, p.wait_limit)) give_up();
    __syncwarp();
    cluster_arrive_release();
    cluster_wait();  // the peer's copies and barriers are no longer in use
    if (warp == 1) tmem_dealloc<2>(tmem, 512);
}

template <typename O, typename B>
cudaError_t launch_pair(const CUtensorMap (&m)[5], const PairParams &pp, int64_t grid, cudaStream_t s) {
    auto fn = linear_pair_kernel<O, B>;
    const cudaError_t e = opt_in_dynamic_smem(reinterpret_cast<const void *>(fn));
    if (e != cudaSuccess) return e;
    return launch(fn, grid, 320, kPairSmem, 2, s, m[0], m[1], m[2], m[3], m[4], pp);
}

}  // namespace

cudaError_t launch_linear_pair(const LinearParams &p, const void *q, const void *w_q, int out_type, int bias_type,
                               int sms, cudaStream_t s) {
    PairParams pp = {p, 0, 0, false, false};
    const int64_t K = (int64_t)p.K64 * 64;
    const int64_t mt = (p.M + kPairTile - 1) / kPairTile, nt = (p.N + kPairTile - 1) / kPairTile;
    const int64_t x_rows = (p.M + 127) / 128 * p.K64, w_rows = (p.N + 127) / 128 * (int64_t)p.K64;
    if (mt * nt > 0x3FFFFFFF || x_rows > 0x7FFFFFFF || w_rows > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    pp.m_tiles = (int)mt;
    pp.n_tiles = (int)nt;
    const int size = out_type == GNQ_FP32 ? 4 : 2;
    pp.tiled = (int64_t)p.N * size % 16 == 0;
    pp.bias16 = p.bias && aligned(p.bias, 16);
    CUtensorMap m[5] = {};
    if (!encode_codes(&m[0], q, p.M, K, 128) || !encode_codes(&m[1], w_q, p.N, K, 128) ||
        !encode_scales(&m[2], p.x_sf, x_rows) || !encode_scales(&m[3], p.w_sf, w_rows) ||
        (pp.tiled && !encode_output(&m[4], p.y, p.M, p.N, size)))
        return cudaErrorInvalidValue;
    const int64_t grid = 2 * std::min<int64_t>(mt * nt, sms / 2);
    if (out_type == GNQ_BF16) return launch_pair<__nv_bfloat16, __nv_bfloat16>(m, pp, grid, s);
    if (out_type == GNQ_FP16) return launch_pair<__half, __half>(m, pp, grid, s);
    if (bias_type == GNQ_FP16) return launch_pair<float, __half>(m, pp, grid, s);
    return launch_pair<float, __nv_bfloat16>(m, pp, grid, s);
}

}  // namespace gnq
