// Products grouped by expert on CTA pairs: tiles of 256 weight rows and up to
// 256 rows of one expert.
//
// As in the pair kernel of one weight, a pair of CTAs issues one product over
// both SMs and the sums of a tile leave tensor memory while the next tile's
// come in.  Here the weight takes the M side (256 rows, 128 per CTA) and the
// expert's rows the N side, as many as there are (rounded up to 32): a ragged
// last tile costs what its rows take in, not a whole tile.  Tensor memory (512
// columns): sums of even tiles in columns 0-255, of odd tiles in 192-447, the
// scales behind; neighbours share 64 columns, which the epilogue takes first.
//
// A lane holds one weight row, so a warp's store is 64 bytes of each of two
// rows of y (128 of one in fp32): whole sectors straight from registers.
//
// Warps of a CTA: 0 copies, 1 issues products (in the pair's first CTA), 2-9
// take sums out: two warps for each 32 weight rows, chunks of 64 rows in turn.
#include <algorithm>

#include "gemma_nq.h"
#include "gnq_expert_linear.cuh"

namespace gnq {
namespace {

constexpr int kRows = 256;        // rows of an expert, and weight rows, of a tile
constexpr int kStages = 5;
constexpr int kPairWarps = 10;
constexpr uint32_t kHalf = 128 * kStageK / 2;              // 128 rows of codes of one stage
constexpr uint32_t kStage = 2 * kHalf + 3 * kBytesSf;      // per CTA: weight, rows, scales of both
constexpr uint32_t kAccCols = 192, kSfwCol = 448, kSfxCol = 464;  // second tile, scales

// y of up to 64 rows (columns of `acc`) x this lane's weight row n.
template <typename O>
__device__ __forceinline__ void store_rows(O *y, int64_t stride, int n, int N, int live, const uint32_t (*acc)[32],
                                           float alpha, float bias, int lane) {
    auto result = [&](uint32_t v) { return fmaf(__uint_as_float(v), alpha, bias); };
    // Two 16-bit columns per lane: neighbouring lanes exchange, the even one
    // stores row i, the odd one i + 1.
    if constexpr (sizeof(O) == 2) {
        if (N % 2 == 0) {
            const int odd = lane & 1;
            O *o = y + n + (odd ? stride - 1 : 0);
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
                const uint32_t own = Act<O>::pack2(result(acc[i / 32][i % 32]), result(acc[i / 32][i % 32 + 1]));
                const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
                if (n < N && i + odd < live)
                    *reinterpret_cast<uint32_t *>(o) =
                        odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
                o += 2 * stride;
            }
            return;
        }
    }
    if (n < N) {
        O *o = y + n;
#pragma unroll
        for (int i = 0; i < 64; ++i, o += stride)
            if (i < live) {
                const float v = result(acc[i / 32][i % 32]);
                if constexpr (std::is_same<O, float>::value) *o = v;
                else *o = OutType<O>::round(v);
            }
    }
}

// map_x: boxes of 128 rows, map_x32: of 32.
template <typename O, typename B>
__global__ void __launch_bounds__(32 * kPairWarps) expert_linear_pair_kernel(
    const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
    const __grid_constant__ CUtensorMap map_x32, const __grid_constant__ CUtensorMap map_ws,
    const __grid_constant__ CUtensorMap map_xs, const __grid_constant__ ExpertLinearParams x) {
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 3];
    __shared__ __align__(16) uint4 topup[kStages];
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;

    const LinearParams &p = x.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t dyn0 = (uint32_t)__cvta_generic_to_shared(dyn), base = (dyn0 + 1023u) & ~1023u;
    const uint32_t bar0 = (uint32_t)__cvta_generic_to_shared(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };               // first CTA's: both halves landed
    auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };  // each CTA's: products done with it
    const uint32_t acc_full = bar0 + 8u * (2 * kStages);            // each CTA's: a tile's sums are ready
    const uint32_t shared_free = acc_full + 8;                      // first CTA's: the shared columns are out
    const uint32_t done = acc_full + 16;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
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
    const TileList list = build_tiles(x, kRows, reinterpret_cast<int *>(dyn + (base - dyn0) + kStages * kStage), kPairWarps);

    const int KT = (p.K64 + 3) / 4;
    const int64_t first = blockIdx.x / 2, G = gridDim.x / 2;
    auto gave_up = [&] { return *(volatile int *)&failed != 0; };
    auto give_up = [&] {
        atomicOr(p.err, (unsigned)DEVERR_WAIT_TIMEOUT);
        *(volatile int *)&failed = 1;
    };
    // Rows that each CTA of the pair holds of a tile: half of them, rounded up
    // to 16.
    auto half_rows = [](int rows) { return (rows + 31) / 32 * 16; };

    if (warp == 0) {
        // ---- copies ----
        int it = 0, s = 0, e = 0;
        uint32_t parity = 1;  // of the wait on `empty`: passes at once in the first round
        const int sf_rows = (p.N + 127) / 128;
        for (int64_t i = first; i < list.count && !__any_sync(0xffffffffu, gave_up()); i += G) {
            const TileList::Tile tile = list.at(i, e, lane);
            e = tile.e;
            const int half = half_rows(tile.rows), x0 = tile.row + half * rank;
            const int boxes = half > 64 ? 0 : (half + 31) / 32;  // 0: one of 128 rows
            const bool second = tile.rows > 128;                 // rows of a second scale tile
            const uint32_t bytes = kHalf + (boxes ? 4096u * boxes : kHalf) + (second ? 3 : 2) * kBytesSf;
            const int w0 = tile.e * p.N + tile.n * kRows + 128 * rank;
            const int ws = (tile.e * sf_rows + 2 * tile.n + rank) * p.K64;
            const int xs = ((tile.start >> 7) + tile.e + ((tile.row - tile.start) >> 7)) * p.K64;
            for (int kt = 0; kt < KT; ++kt, ++it) {
                if (!warp_wait_bounded(empty(s), parity, p.wait_limit)) {
                    give_up();
                    break;
                }
                if (elect_one()) {
                    const uint32_t at = base + kStage * s, bar = map_to_cta(full(s), 0);
                    if (rank == 0) mbar_expect_tx(full(s), 2 * bytes + p.tx_extra);
                    tma_load_pair(at, &map_w, kt * 128, w0, bar);
                    if (boxes == 0) {
                        tma_load_pair(at + kHalf, &map_x, kt * 128, x0, bar);
                    } else {
                        tma_load_pair(at + kHalf, &map_x32, kt * 128, x0, bar);
                        if (boxes == 2) tma_load_pair(at + kHalf + 4096, &map_x32, kt * 128, x0 + 32, bar);
                    }
                    tma_load_pair(at + 2 * kHalf, &map_ws, 0, ws + 4 * kt, bar);
                    tma_load_pair(at + 2 * kHalf + kBytesSf, &map_xs, 0, xs + 4 * kt, bar);
                    if (second) tma_load_pair(at + 2 * kHalf + 2 * kBytesSf, &map_xs, 0, xs + p.K64 + 4 * kt, bar);
                }
                __syncwarp();
                if (++s == kStages) s = 0, parity ^= 1;
            }
        }
        // Every copy has landed before the shared memory goes away (test
        // hook: with the bytes that its announcement lacks).
        if (rank == 0 && lane == 0)
            for (int j = max(0, it - kStages); j < it; ++j) {
                const int s = j % kStages;
                if (mbar_wait_bounded(full(s), (j / kStages) & 1, p.wait_limit)) continue;
                give_up();
                if (p.tx_extra) bulk_g2s((uint32_t)__cvta_generic_to_shared(&topup[s]), p.w_sf, p.tx_extra, full(s));
                mbar_wait_bounded(full(s), (j / kStages) & 1, p.wait_limit);
            }
    } else if (warp == 1 && rank == 0) {
        // ---- products ----
        int j = 0, s = 0, e = 0;
        uint32_t parity = 0;
        bool good = true;
        for (int64_t i = first; good && i < list.count; i += G, ++j) {
            const TileList::Tile tile = list.at(i, e, lane);
            e = tile.e;
            const uint32_t idesc = idesc_nvfp4(256, 2 * half_rows(tile.rows));
            const bool second = tile.rows > 128;
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
                    const uint32_t at = (base >> 4) + (kStage >> 4) * s;
                    auto step = [&](int k) {
                        cp_scales<2>(tmem + kSfwCol + 4 * k, desc_scales(at + (2 * kHalf + 512 * k) / 16));
                        cp_scales<2>(tmem + kSfxCol + 8 * k, desc_scales(at + (2 * kHalf + kBytesSf + 512 * k) / 16));
                        if (second)
                            cp_scales<2>(tmem + kSfxCol + 8 * k + 4,
                                         desc_scales(at + (2 * kHalf + 2 * kBytesSf + 512 * k) / 16));
                        mma_nvfp4<2>(acc, desc_sw128(at + 2 * k), desc_sw128(at + kHalf / 16 + 2 * k), idesc,
                                     tmem + kSfwCol + 4 * k, tmem + kSfxCol + 8 * k, kt > 0 || k > 0);
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
                if (++s == kStages) s = 0, parity ^= 1;
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
        const int quad = warp & 3, set = (warp - 2) >> 2;
        const uint32_t lanes = (uint32_t)quad << 21;  // 32 lanes per warp, lane number in bits 16-31
        const uint32_t free_bar = map_to_cta(shared_free, 0);
        int j = 0, e = 0;
        for (int64_t i = first; i < list.count; i += G, ++j) {
            const TileList::Tile tile = list.at(i, e, lane);
            e = tile.e;
            const int n = tile.n * kRows + 128 * rank + 32 * quad + lane;
            const float alpha = ld_f32(p.alpha + e * x.alpha_stride);
            const float bias = p.bias && n < p.N ? OutType<B>::bias(ld_u16(p.bias + (int64_t)e * p.N + n)) : 0.f;
            const bool ok = mbar_wait_bounded(acc_full, j & 1, 2 * p.wait_limit) && !(p.tx_extra && gave_up());
            if (!__all_sync(0xffffffffu, ok)) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + kAccCols * (j & 1) + lanes;
            // the next tile may start once the shared columns of this one are
            // out (first set) and all of the one before, whose place it takes
            // (second set: it has come here)
            if (set == 1 && lane == 0) arrive_remote(free_bar);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int turn = 2 * h + set;  // chunk in the order of taking: the shared one is the first
                const int c = j & 1 ? 64 * turn : 64 * ((turn + 3) & 3);
                const int live = tile.rows - c;
                uint32_t v[2][32];
                if (live > 0) {
                    tmem_ld32(acc + c, v[0]);
                    tmem_ld32(acc + c + 32, v[1]);
                    tmem_wait(v[0]);
                    tmem_wait(v[1]);
                }
                if (turn == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_remote(free_bar);
                }
                if (live > 0)
                    store_rows<O>(static_cast<O *>(p.y) + (int64_t)(tile.row + c) * p.N, p.N, n, p.N, live, v, alpha, bias,
                                  lane);
                __syncwarp();
            }
            tc_fence_before();  // this tile's reads are done before the arrival at the next
            __syncwarp();
        }
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
cudaError_t launch_pair(const CUtensorMap (&m)[5], const ExpertLinearParams &x, int64_t grid, size_t smem, cudaStream_t s) {
    auto fn = expert_linear_pair_kernel<O, B>;
    const cudaError_t e = opt_in_dynamic_smem(reinterpret_cast<const void *>(fn));
    if (e != cudaSuccess) return e;
    return launch(fn, grid, 32 * kPairWarps, smem, 2, s, m[0], m[1], m[2], m[3], m[4], x);
}

}  // namespace

cudaError_t launch_expert_linear_pair(ExpertLinearParams x, const void *q, const void *w_q, int out_type, int bias_type,
                                      int sms, cudaStream_t s) {
    LinearParams &p = x.p;
    p.n_tiles = (p.N + kRows - 1) / kRows;
    const int64_t K = (int64_t)p.K64 * 64, E = x.E, R = p.M;
    const int64_t x_rows = (R / 128 + E) * p.K64, w_rows = E * ((p.N + 127) / 128) * p.K64;
    if (x_rows > 0x7FFFFFFF || w_rows > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    CUtensorMap m[5] = {};
    if (!encode_codes(&m[0], w_q, E * p.N, K, 128) || !encode_codes(&m[1], q, R, K, 128) ||
        !encode_codes(&m[2], q, R, K, 32) || !encode_scales(&m[3], p.w_sf, w_rows) || !encode_scales(&m[4], p.x_sf, x_rows))
        return cudaErrorInvalidValue;
    const int64_t tiles = (R / kRows + std::min(E, R)) * p.n_tiles;  // at most
    const int64_t grid = 2 * std::min<int64_t>(tiles, sms / 2);
    const size_t smem = 1024 + kStages * kStage + TileList::bytes(x.E, kPairWarps);
    if (out_type == GNQ_BF16) return launch_pair<__nv_bfloat16, __nv_bfloat16>(m, x, grid, smem, s);
    if (out_type == GNQ_FP16) return launch_pair<__half, __half>(m, x, grid, smem, s);
    if (bias_type == GNQ_FP16) return launch_pair<float, __half>(m, x, grid, smem, s);
    return launch_pair<float, __nv_bfloat16>(m, x, grid, smem, s);
}

}  // namespace gnq
