// Products of NVFP4 rows with the NVFP4 weight of each row's expert.  The
// contract is in include/gemma_nq.h.
//
//   y[r, n] = alpha[e] * sum_k a[r, k] sa[r, k/16] w[e, n, k] sw[e, n, k/16] + bias[e, n]
//
// e being the expert whose rows offsets[e] .. offsets[e + 1] - 1 hold r.  The
// arithmetic is that of nvfp4_linear: products of codes and scales exact,
// sums in fp32 in tensor memory, one rounding.
//
// The weight takes the tensor core's M side (128 rows), the rows of one expert
// its N side, as many as there are (rounded up to 16): an expert with few rows
// wastes neither tensor time nor row copies.  CTAs are persistent; each walks
// the list of tiles, which it builds itself from the offsets, with one warp
// copying, one issuing products and four taking sums out while the next tile's
// products run.  (K-splitting clusters for a handful of rows, as the product of
// one weight has them, gained only below 64 tiles: one token to 8 of 128 experts,
// N = 2048, K = 4096, 11.2 us against 10.8.)
//
// What bounds it: the bytes of the weights that have rows, each read once.  64
// tokens to 8 of 128 experts, N = 4096, K = 2048: 77 us of 73.7 at the copy rate (105
// experts have rows), to fp32 78 of 75; one token, N = 2048, K = 4096: 10.4 us of 5.6,
// launch, offsets, first copy and last store; 301 tokens to 4 of 60, 1000 x 1088: 11.5
// of 5.8, 480 tiles on 304 CTAs.
#include <algorithm>

#include "gemma_nq.h"
#include "gnq_expert_linear.cuh"

namespace gnq {
namespace {

// 64 rows a tile leave tensor memory (twice 64 sums and the scales) and shared
// memory (three stages) for two CTAs on an SM, one of which computes while the
// other starts or ends a tile: 77.1 us for 64 tokens to 8 of 128 experts, N = 4096,
// K = 2048 (79.2 with one CTA and 128 rows); 128 experts of 200 rows, N = 2048, K =
// 512: 40.9 (51.0); of 16 rows, N = 4096, K = 2048: 89.8 (94.0).
constexpr int kTileRows = 64;
constexpr int kPerSm = 2;
constexpr uint32_t kTmemCols = 256;
constexpr int kRowBox = 32;  // rows of one tile copy of activations
constexpr uint32_t kBytesX = kTileRows * 128, kStage = kBytesW + kBytesX + 2 * kBytesSf;
constexpr int kWarps = 6;

template <typename O, typename B>
__global__ void __launch_bounds__(32 * kWarps) expert_linear_kernel(const __grid_constant__ CUtensorMap map_w,
                                                                    const __grid_constant__ CUtensorMap map_x,
                                                                    const __grid_constant__ ExpertLinearParams x) {
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5];
    __shared__ __align__(16) uint4 topup[kMaxStages];
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;

    const LinearParams &p = x.p;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const uint32_t dyn0 = (uint32_t)__cvta_generic_to_shared(dyn), base = (dyn0 + 1023u) & ~1023u;
    const uint32_t bar0 = (uint32_t)__cvta_generic_to_shared(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * kMaxStages + 2 + b); };
    const uint32_t done = bar0 + 8u * (2 * kMaxStages + 4);
    if (warp == 0 && lane == 0) {
        prefetch_map(&map_w);
        prefetch_map(&map_x);
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 4);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        failed = 0;
    }
    if (warp == 1) {
        tmem_alloc<1>((uint32_t)__cvta_generic_to_shared(&tmem_slot), kTmemCols);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t sfw_col = tmem + 2 * kTileRows, sfx_col = sfw_col + 16;

    pdl_wait();  // inputs may come from the preceding grid, outputs may still be read by it
    pdl_trigger();
    const TileList list = build_tiles(x, kTileRows, reinterpret_cast<int *>(dyn + (base - dyn0) + kStage * p.stages), kWarps);

    const int KT = (p.K64 + 3) / 4;
    auto give_up = [&] {
        atomicOr(p.err, (unsigned)DEVERR_WAIT_TIMEOUT);
        *(volatile int *)&failed = 1;
    };
    auto gave_up = [&] { return *(volatile int *)&failed != 0; };
    if (warp == 0) {
        // ---- copies ----
        int it = 0, s = 0, e = 0;
        uint32_t parity = 1;  // of the wait on `empty`: passes at once in the first round
        const int sf_rows = (p.N + 127) / 128;
        bool good = true;
        for (int i = blockIdx.x; good && i < list.count; i += (int)gridDim.x) {
            const TileList::Tile tile = list.at(i, e, lane);
            e = tile.e;
            const int w0 = tile.e * p.N + tile.n * kTileN, boxes = (tile.rows + kRowBox - 1) / kRowBox;
            const uint8_t *const w_sf = p.w_sf + ((int64_t)tile.e * sf_rows + tile.n) * p.K64 * 512;
            const uint8_t *const x_sf =
                p.x_sf + ((int64_t)(tile.start >> 7) + tile.e + ((tile.row - tile.start) >> 7)) * p.K64 * 512;
            for (int kt = 0; kt < KT; ++kt, ++it) {
                if (!warp_wait_bounded(empty(s), parity, p.wait_limit)) {
                    give_up();
                    good = false;
                    break;
                }
                if (elect_one()) {
                    const uint32_t at = base + kStage * s, sf_bytes = 512u * min(4, p.K64 - 4 * kt);
                    mbar_expect_tx(full(s), kBytesW + boxes * (kRowBox * 128) + 2 * sf_bytes + p.tx_extra);
                    tma_load_2d(at, &map_w, kt * 128, w0, full(s));
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(at + kBytesW + b * (kRowBox * 128), &map_x, kt * 128, tile.row + b * kRowBox, full(s));
                    bulk_g2s(at + kBytesW + kBytesX, w_sf + kt * 2048, sf_bytes, full(s));
                    bulk_g2s(at + kBytesW + kBytesX + kBytesSf, x_sf + kt * 2048, sf_bytes, full(s));
                }
                __syncwarp();
                if (++s == p.stages) s = 0, parity ^= 1;
            }
        }
        // Every copy has landed before the shared memory goes away: the last
        // use of each stage (test hook: with the bytes that its announcement
        // lacks).
        if (lane == 0)
            for (int j = max(0, it - p.stages); j < it; ++j) {
                const int s = j % p.stages;
                if (mbar_wait_bounded(full(s), (j / p.stages) & 1, p.wait_limit)) continue;
                give_up();
                if (p.tx_extra) bulk_g2s((uint32_t)__cvta_generic_to_shared(&topup[s]), p.w_sf, p.tx_extra, full(s));
                mbar_wait_bounded(full(s), (j / p.stages) & 1, p.wait_limit);
            }
    } else if (warp == 1) {
        // ---- products ----
        int s = 0, j = 0, e = 0;
        uint32_t parity = 0;
        bool good = true;
        for (int i = blockIdx.x; good && i < list.count; i += gridDim.x, ++j) {
            const TileList::Tile tile = list.at(i, e, lane);
            e = tile.e;
            const uint32_t idesc = idesc_nvfp4(kTileN, (tile.rows + 15) & ~15);
            // 32 rows of a scale tile are one column of tensor memory.  A tile
            // starts 0 or 64 rows into it: the column has to be even.
            const uint32_t acc = tmem + kTileRows * (j & 1), sfx = sfx_col + (((tile.row - tile.start) & 127) >> 5);
            if (!warp_wait_bounded(acc_empty(j & 1), ((j >> 1) & 1) ^ 1, p.wait_limit)) {
                give_up();
                break;
            }
            tc_fence_after();
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
                const int nk = min(4, p.K64 - 4 * kt);
                if (elect_one()) {
                    const uint32_t at = (base + kStage * s) >> 4, sf = at + ((kBytesW + kBytesX) >> 4);
                    auto step = [&](int k) {
                        cp_scales<1>(sfw_col + 4 * k, desc_scales(sf + 32 * k));
                        cp_scales<1>(sfx_col + 4 * k, desc_scales(sf + kBytesSf / 16 + 32 * k));
                        mma_nvfp4<1>(acc, desc_sw128(at + 2 * k), desc_sw128(at + kBytesW / 16 + 2 * k), idesc,
                                     sfw_col + 4 * k, sfx + 4 * k, kt > 0 || k > 0);
                    };
                    if (nk == 4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) step(k);
                    } else {
                        for (int k = 0; k < nk; ++k) step(k);
                    }
                    tc_commit(empty(s));
                    if (kt == KT - 1) tc_commit(acc_full(j & 1));
                }
                __syncwarp();
                if (++s == p.stages) s = 0, parity ^= 1;
            }
        }
        // every product is done before tensor memory goes away
        if (elect_one()) tc_commit(done);
        __syncwarp();
        if (!warp_wait_bounded(done, 0, p.wait_limit)) give_up();
    } else {
        // ---- sums out: warp by warp 32 weight rows, one per lane ----
        const int quad = warp & 3, row = 32 * quad + lane;
        const uint32_t lanes = (uint32_t)quad << 21;  // 32 lanes per warp, lane number in bits 16-31
        int j = 0, e = 0;
        for (int i = blockIdx.x; i < list.count; i += gridDim.x, ++j) {
            const TileList::Tile tile = list.at(i, e, lane);
            e = tile.e;
            const int n = tile.n * kTileN + row;
            const float alpha = ld_f32(p.alpha + e * x.alpha_stride);
            const float bias = p.bias && n < p.N ? OutType<B>::bias(ld_u16(p.bias + (int64_t)e * p.N + n)) : 0.f;
            if (!warp_wait_bounded(acc_full(j & 1), (j >> 1) & 1, 2 * p.wait_limit) ||
                (p.tx_extra && __any_sync(0xffffffffu, gave_up()))) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + kTileRows * (j & 1) + lanes;
            auto result = [&](uint32_t v) { return fmaf(__uint_as_float(v), alpha, bias); };
            // Two 16-bit columns per lane: neighbouring lanes exchange, the
            // even one stores row c + i, the odd one c + i + 1.
            const bool pairs = sizeof(O) == 2 && p.N % 2 == 0;
            for (int c = 0; c < tile.rows; c += 16) {
                uint32_t v[16];
                __syncwarp();
                tmem_ld16(acc + c, v);
                tmem_wait(v);
                O *o = static_cast<O *>(p.y) + (int64_t)(tile.row + c) * p.N + n;
                const int live = tile.rows - c;
                if constexpr (sizeof(O) == 2) {
                    if (pairs) {
                        const int odd = lane & 1;
                        o += odd ? (int64_t)p.N - 1 : 0;
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const uint32_t own = Act<O>::pack2(result(v[i]), result(v[i + 1]));
                            const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
                            if (n < p.N && i + odd < live)
                                *reinterpret_cast<uint32_t *>(o) =
                                    odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
                            o += 2 * (int64_t)p.N;
                        }
                        continue;
                    }
                }
                if (n < p.N)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < live) {
                            if constexpr (std::is_same<O, float>::value) o[i * (int64_t)p.N] = result(v[i]);
                            else o[i * (int64_t)p.N] = OutType<O>::round(result(v[i]));
                        }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(acc_empty(j & 1)) : "memory");
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc<1>(tmem, kTmemCols);
}

template <typename O, typename B>
cudaError_t launch_expert_linear(const CUtensorMap &mw, const CUtensorMap &mx, const ExpertLinearParams &x, int64_t grid,
                                 size_t smem, cudaStream_t s) {
    auto fn = expert_linear_kernel<O, B>;
    const cudaError_t e = opt_in_dynamic_smem(reinterpret_cast<const void *>(fn));
    if (e != cudaSuccess) return e;
    return launch(fn, grid, 32 * kWarps, smem, 1, s, mw, mx, x);
}

// Whether CTA pairs take the call.  Their tile is eight times the other
// kernel's and pays from about 120 rows an expert on, where there are enough of
// them to go round and K is deep enough for the hand-over between tiles; with
// many, from 96 rows on.  Of 668 shapes timed in both kernels (2 to 128 experts, 64
// to 1000 rows each, N of 512 to 8192, K of 512 to 4096) the choice loses 0.4 % on
// average against the faster one, and more than 10 % on 3 (2 experts of 380 rows,
// N = K = 4096: 17.4 us on single CTAs, 15.8 on pairs; 16 of 200 rows, N = 1024,
// K = 2048: 11.3 and 12.4).  R, the rows that the buffers have room for, stands for
// the rows that there are, which the host does not know: in all shapes timed the two
// were the same, and a batch most of whose slots are -1 is taken for a full one.
bool pairs_take(int64_t E, int64_t R, int64_t N, int64_t K) {
    if (K < 768) return false;
    const int64_t tiles = (N + 255) / 256 * std::max(E, R / 224);
    return R >= 120 * E ? tiles >= (K >= 1536 ? 64 : 300) : R >= 96 * E && tiles >= 500;
}

}  // namespace
}  // namespace gnq

extern "C" int nvfp4_expert_linear(const void *q, const void *block_scale, const void *w_q, const void *w_block_scale,
                                   const float *alpha, int alpha_stride, const void *bias, const int32_t *offsets,
                                   int64_t E, void *y, int64_t R, int64_t N, int64_t K, int out_type, int bias_type,
                                   void *stream) {
    using namespace gnq;
    if (out_type < GNQ_BF16 || out_type > GNQ_FP32) return GNQ_ERR_DTYPE;
    if (bias && bias_type != GNQ_BF16 && bias_type != GNQ_FP16) return GNQ_ERR_DTYPE;
    if (bias && out_type != GNQ_FP32 && bias_type != out_type) return GNQ_ERR_DTYPE;
    if (alpha_stride != 0 && alpha_stride != 1) return GNQ_ERR_MODE;
    if (E < 1 || E > kMaxExperts || R < 0 || R > kMaxM) return GNQ_ERR_SHAPE;
    if (N <= 0 || N > kMaxM || N * E > kMaxM || K <= 0 || K > kMaxH || K % 64 != 0) return GNQ_ERR_SHAPE;
    if (R == 0) return GNQ_OK;
    if (!q || !block_scale || !w_q || !w_block_scale || !alpha || !offsets || !y) return GNQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(block_scale, 16) || !aligned(w_q, 16) || !aligned(w_block_scale, 16) ||
        !aligned(y, 16) || !aligned(alpha, 4) || !aligned(offsets, 4) || !aligned(bias, 2))
        return GNQ_ERR_ALIGN;
    const Extent written[] = {extent(y, R * N * (out_type == GNQ_FP32 ? 4 : 2))};
    const Extent read[] = {extent(q, code_bytes(GNQ_NVFP4, R, K)), extent(block_scale, (R / 128 + E) * 8 * K),
                           extent(w_q, code_bytes(GNQ_NVFP4, E * N, K)),
                           extent(w_block_scale, E * scale_bytes(GNQ_NVFP4, N, K)),
                           extent(alpha, 4 * (alpha_stride ? E : 1)), extent(offsets, 4 * (E + 1)),
                           extent(bias, 2 * E * N)};
    if (outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
    for (const void *buf : {q, block_scale, w_q, w_block_scale, static_cast<const void *>(y)})
        if (!on_device(buf, d->dev)) return GNQ_ERR_MEMORY;
    ExpertLinearParams x = {};
    x.offsets = offsets;
    x.E = (int)E;
    x.alpha_stride = alpha_stride;
    LinearParams &p = x.p;
    p.w_sf = static_cast<const uint8_t *>(w_block_scale);
    p.x_sf = static_cast<const uint8_t *>(block_scale);
    p.alpha = alpha;
    p.bias = static_cast<const uint16_t *>(bias);
    p.y = y;
    p.M = R;
    p.N = (int)N;
    p.K64 = (int)(K / 64);
    p.err = d->err;
    p.wait_limit = wait_limit_cycles();
    p.tx_extra = inject_timeout_on() ? 16u : 0u;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int forced = linear_policy();
    if (forced ? forced == 2 : pairs_take(E, R, N, K)) return status_of(launch_expert_linear_pair(x, q, w_q, out_type, bias_type, d->sms, s));
    p.n_tiles = (int)((N + kTileN - 1) / kTileN);
    const int64_t tiles = (R / kTileRows + std::min(E, R)) * p.n_tiles;  // at most
    if (tiles > 0x3FFFFFFF) return GNQ_ERR_SHAPE;
    const int64_t lists = TileList::bytes((int)E, kWarps);
    // (each CTA: 1 KB of the system's, its static part, and what alignment takes)
    const int64_t room = (tiles <= d->sms ? d->smem_optin : d->smem_sm / kPerSm - 1024) - 1024 - 1024 - lists;
    p.stages = (int)std::min<int64_t>(kMaxStages, room / kStage);
    const size_t smem = (size_t)(1024 + p.stages * kStage + lists);
    const int64_t grid = std::min<int64_t>(tiles, kPerSm * d->sms);
    CUtensorMap mw, mx;
    if (!encode_codes(&mw, w_q, E * N, K, kTileN) || !encode_codes(&mx, q, R, K, kRowBox)) return GNQ_ERR_CUDA;
    if (out_type == GNQ_BF16) return status_of(launch_expert_linear<__nv_bfloat16, __nv_bfloat16>(mw, mx, x, grid, smem, s));
    if (out_type == GNQ_FP16) return status_of(launch_expert_linear<__half, __half>(mw, mx, x, grid, smem, s));
    if (bias_type == GNQ_FP16) return status_of(launch_expert_linear<float, __half>(mw, mx, x, grid, smem, s));
    return status_of(launch_expert_linear<float, __nv_bfloat16>(mw, mx, x, grid, smem, s));
}
