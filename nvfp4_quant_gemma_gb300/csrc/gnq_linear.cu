// Product of an NVFP4 activation with an NVFP4 weight.  The contract is in
// include/gemma_nq.h.
//
//   y[m, n] = alpha * sum_k a[m, k] sa[m, k/16] w[n, k] sw[n, k/16] + bias[n]
//
// a, w: E2M1 codes, two per byte; sa, sw: E4M3 block scales in the 128x4
// layout.  Every product of two codes and two scales is exact in fp32; the
// tensor cores accumulate in fp32 (tensor memory) and the result is rounded
// once to the output type.
//
// The weight takes the tensor core's M side (128 rows), the tokens its N
// side (16 to 256), so a decode batch wastes no rows.  A scale tile of the
// 128x4 layout is 512 contiguous bytes for 128 rows x 64 elements, exactly
// what one copy into tensor memory takes, so scales are fetched by plain bulk
// copies.  K advances by 256 elements (128 bytes, one swizzle row) a stage.
#include <algorithm>
#include <atomic>

#include "gemma_nq.h"
#include "gnq_linear.cuh"

namespace gnq {
namespace {

// O: output type; B: type of the bias (bf16 or fp16).
template <typename O, typename B>
__global__ void __launch_bounds__(128) linear_kernel(const __grid_constant__ CUtensorMap map_w,
                                                     const __grid_constant__ CUtensorMap map_x,
                                                     const __grid_constant__ LinearParams p) {
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 1];
    __shared__ __align__(16) uint4 topup[kMaxStages];
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;

    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const uint32_t base = ((uint32_t)__cvta_generic_to_shared(dyn) + 1023u) & ~1023u;
    const uint32_t bar0 = (uint32_t)__cvta_generic_to_shared(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    const uint32_t acc_bar = bar0 + 8u * (2 * kMaxStages);

    const int S = p.split, ks = blockIdx.x % S, tile = blockIdx.x / S;
    const int nt = tile % p.n_tiles, n0 = nt * kTileN;
    const int64_t tt = tile / p.n_tiles, t0 = tt * p.T;
    const int KT = (p.K64 + 3) / 4;
    const int k_begin = KT * ks / S, n_k = KT * (ks + 1) / S - k_begin;
    const uint32_t bytes_x = (uint32_t)p.T * 128;
    const uint32_t stage_bytes = kBytesW + bytes_x + 2 * kBytesSf;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(acc_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        failed = 0;
    }
    if (warp == 1) {
        tmem_alloc<1>((uint32_t)__cvta_generic_to_shared(&tmem_slot), p.tmem_cols);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t sfw_col = tmem + p.T, sfx_col = sfw_col + 16;

    pdl_wait();  // inputs may come from the preceding grid, outputs may still be read by it
    pdl_trigger();

    auto give_up = [&] {
        atomicOr(p.err, (unsigned)DEVERR_WAIT_TIMEOUT);
        *(volatile int *)&failed = 1;
    };

    auto gave_up = [&] { return *(volatile int *)&failed != 0; };
    if (warp == 0) {
        // ---- copies ----
        int i = 0;
        for (; i < n_k; ++i) {
            const int s = i % p.stages;
            if (i >= p.stages && !mbar_wait_bounded(empty(s), (i / p.stages - 1) & 1, p.wait_limit)) {
                give_up();
                break;
            }
            const int kt = k_begin + i, nk = min(4, p.K64 - 4 * kt);
            if (elect_one()) {
                const uint32_t at = base + stage_bytes * s, sf_bytes = 512u * nk;
                mbar_expect_tx(full(s), kBytesW + bytes_x + 2 * sf_bytes + p.tx_extra);
                tma_load_2d(at, &map_w, kt * 128, n0, full(s));
                tma_load_2d(at + kBytesW, &map_x, kt * 128, (int)t0, full(s));
                const uint32_t sf = at + kBytesW + bytes_x;
                bulk_g2s(sf, p.w_sf + ((int64_t)nt * p.K64 + 4 * kt) * 512, sf_bytes, full(s));
                bulk_g2s(sf + kBytesSf, p.x_sf + (t0 / 128 * p.K64 + 4 * kt) * 512, sf_bytes, full(s));
            }
            __syncwarp();
        }
        // Every copy has landed before the shared memory goes away or is
        // used again: the last use of each stage (test hook: with the bytes
        // that its announcement lacks).
        if (lane == 0)
            for (int j = max(0, i - p.stages); j < i; ++j) {
                const int s = j % p.stages;
                if (mbar_wait_bounded(full(s), (j / p.stages) & 1, p.wait_limit)) continue;
                give_up();
                if (p.tx_extra) bulk_g2s((uint32_t)__cvta_generic_to_shared(&topup[s]), p.w_sf, p.tx_extra, full(s));
                mbar_wait_bounded(full(s), (j / p.stages) & 1, p.wait_limit);
            }
    } else if (warp == 1) {
        // ---- products ----
        const uint32_t idesc = idesc_nvfp4(kTileN, p.T);
        for (int i = 0; i < n_k; ++i) {
            const int s = i % p.stages;
            if (!mbar_wait_bounded(full(s), (i / p.stages) & 1, p.wait_limit) || (p.tx_extra && gave_up())) {
                give_up();
                break;
            }
            tc_fence_after();
            const int nk = p.K64 - 4 * (k_begin + i);
            if (elect_one()) {
                const uint32_t at = (base + stage_bytes * s) >> 4, sf = at + ((kBytesW + bytes_x) >> 4);
                auto step = [&](int k) {
                    cp_scales<1>(sfw_col + 4 * k, desc_scales(sf + 32 * k));
                    cp_scales<1>(sfx_col + 4 * k, desc_scales(sf + kBytesSf / 16 + 32 * k));
                    mma_nvfp4<1>(tmem, desc_sw128(at + 2 * k), desc_sw128(at + kBytesW / 16 + 2 * k), idesc,
                                 sfw_col + 4 * k, sfx_col + 4 * k, i > 0 || k > 0);
                };
                if (nk >= 4) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) step(k);
                } else {
                    for (int k = 0; k < nk; ++k) step(k);
                }
                tc_commit(empty(s));
            }
            __syncwarp();
        }
        if (elect_one()) tc_commit(acc_bar);
    }
    __syncwarp();

    // ---- epilogue ----
    if (!mbar_wait_bounded(acc_bar, 0, 2 * p.wait_limit)) give_up();
    tc_fence_after();
    __syncthreads();  // `failed` agreed on, every copy landed
    const bool good = !failed;
    const float alpha = __ldg(p.alpha);
    const int row = warp * 32 + lane, n = n0 + row;
    const int rows = (int)min((int64_t)p.T, p.M - t0);  // tokens in the tile
    const float bias = p.bias && n < p.N ? OutType<B>::bias(__ldg(p.bias + n)) : 0.f;
    auto store = [&](int64_t m, float v) {
        const float r = fmaf(v, alpha, bias);
        const int64_t at = m * p.N + n;
        if constexpr (std::is_same<O, float>::value) static_cast<float *>(p.y)[at] = r;
        else static_cast<O *>(p.y)[at] = OutType<O>::round(r);
    };
    const uint32_t lane_base = (uint32_t)warp << 21;  // 32 lanes per warp, lane number in bits 16-31
    if (S == 1) {
        if (good)
            for (int c = 0; c < rows; c += 16) {
                uint32_t v[16];
                __syncwarp();
                tmem_ld16(tmem + lane_base + c, v);
                tmem_wait(v);
                if (n < p.N)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < rows) store(t0 + c + j, __uint_as_float(v[j]));
            }
    } else {
        // The cluster's partial sums meet in shared memory, [token][weight row]
        // in fp32, and each CTA adds every S-th token's in rank order.
        float *part = reinterpret_cast<float *>(dyn + (base - (uint32_t)__cvta_generic_to_shared(dyn)));
        if (good)
            for (int c = 0; c < rows; c += 16) {
                uint32_t v[16];
                tmem_ld16(tmem + lane_base + c, v);
                tmem_wait(v);
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(c + j) * kTileN + row] = __uint_as_float(v[j]);
            }
        cluster_arrive_release();
        cluster_wait();
        if (good && n < p.N)
            for (int c0 = ks; c0 < rows; c0 += 8 * S) {  // 8 tokens at a time: their reads overlap
                float v[8] = {};
                for (int r = 0; r < S; ++r)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] += ld_peer_f32(part + min(c0 + j * S, rows - 1) * kTileN + row, r);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + j * S < rows) store(t0 + c0 + j * S, v[j]);
            }
        cluster_arrive_release();
        cluster_wait();  // peers may still be reading this CTA's sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc<1>(tmem, p.tmem_cols);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static std::atomic<EncodeFn> cached{nullptr};
    EncodeFn f = cached.load();
    if (!f) {
        void *sym = nullptr;
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &st) !=
                cudaSuccess || st != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<EncodeFn>(sym);
        cached.store(f);
    }
    return f;
}

bool encode_tiles(CUtensorMap *map, CUtensorMapDataType type, const void *base, const cuuint64_t (&dims)[2],
                  cuuint64_t stride, const cuuint32_t (&box)[2], CUtensorMapSwizzle swizzle) {
    const EncodeFn f = encode_fn();
    const cuuint32_t step[2] = {1, 1};
    return f && f(map, type, 2, const_cast<void *>(base), dims, &stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool encode_codes(CUtensorMap *map, const void *codes, int64_t rows, int64_t K, int box) {
    return encode_tiles(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, {(cuuint64_t)(K / 2), (cuuint64_t)rows},
                        (cuuint64_t)(K / 2), {128, (cuuint32_t)box}, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool encode_scales(CUtensorMap *map, const void *scales, int64_t rows) {
    return encode_tiles(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales, {128, (cuuint64_t)rows}, 512, {128, 4},
                        CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool encode_output(CUtensorMap *map, void *y, int64_t M, int64_t N, int size) {
    return encode_tiles(map, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, y,
                        {(cuuint64_t)N, (cuuint64_t)M}, (cuuint64_t)N * size, {(cuuint32_t)(128 / size), 32},
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

namespace {

// Tile and split of a call.  The smallest tile that holds the tokens (above
// 128, tiles of 256); K is split over a cluster while the grid is smaller
// than the SMs and every CTA keeps a stage of it.
bool shape_of(const DevInfo &d, int64_t M, int64_t N, int64_t K, LinearParams &p, int64_t &grid, size_t &smem) {
    p.T = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    p.n_tiles = (int)((N + kTileN - 1) / kTileN);
    const int KT = (p.K64 + 3) / 4;
    const int64_t tiles = p.n_tiles * ((M + p.T - 1) / p.T);
    p.split = (int)std::max<int64_t>(1, std::min<int64_t>({8, d.sms / tiles, KT}));
    grid = tiles * p.split;
    if (grid > 0x7FFFFFFF) return false;
    const int64_t stage = kBytesW + p.T * 128 + 2 * kBytesSf;
    p.tmem_cols = p.T <= 32 ? 64 : p.T == 64 ? 128 : 256;
    // two CTAs per SM where the grid has them and half of each memory does
    const int64_t limit = d.smem_optin - 1024 - 512;
    const int64_t room = grid > d.sms ? limit / 2 - 1024 : limit;
    p.stages = (int)std::min<int64_t>({kMaxStages, room / stage, (KT + p.split - 1) / p.split});
    p.stages = std::max(p.stages, 1);
    smem = (size_t)(1024 + std::max<int64_t>(p.stages * stage, p.split > 1 ? p.T * kTileN * 4 : 0));
    return true;
}

template <typename O, typename B>
cudaError_t launch_linear(const CUtensorMap &mw, const CUtensorMap &mx, const LinearParams &p, int64_t grid,
                          size_t smem, cudaStream_t s) {
    auto fn = linear_kernel<O, B>;
    const cudaError_t e = opt_in_dynamic_smem(reinterpret_cast<const void *>(fn));
    if (e != cudaSuccess) return e;
    return launch(fn, grid, 128, smem, p.split, s, mw, mx, p);
}

}  // namespace
}  // namespace gnq

extern "C" int nvfp4_linear(const void *q, const void *block_scale, const void *w_q, const void *w_block_scale,
                            const float *alpha, const void *bias, void *y, int64_t M, int64_t N, int64_t K,
                            int out_type, int bias_type, void *stream) {
    using namespace gnq;
    if (out_type < GNQ_BF16 || out_type > GNQ_FP32) return GNQ_ERR_DTYPE;
    if (bias && bias_type != GNQ_BF16 && bias_type != GNQ_FP16) return GNQ_ERR_DTYPE;
    if (bias && out_type != GNQ_FP32 && bias_type != out_type) return GNQ_ERR_DTYPE;
    if (M < 0 || M > kMaxM || N <= 0 || N > kMaxM || K <= 0 || K > kMaxH || K % 64 != 0) return GNQ_ERR_SHAPE;
    if (M == 0) return GNQ_OK;
    if (!q || !block_scale || !w_q || !w_block_scale || !alpha || !y) return GNQ_ERR_NULL;
    if (y == q || y == block_scale || y == w_q || y == w_block_scale || (bias && y == bias)) return GNQ_ERR_ALIAS;
    if (!aligned(q, 16) || !aligned(block_scale, 16) || !aligned(w_q, 16) || !aligned(w_block_scale, 16) ||
        !aligned(y, 16) || !aligned(alpha, 4) || (bias && !aligned(bias, 2)))
        return GNQ_ERR_ALIGN;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
    if (!in_device_memory(q) || !in_device_memory(block_scale) || !in_device_memory(w_q) ||
        !in_device_memory(w_block_scale))
        return GNQ_ERR_MEMORY;
    LinearParams p = {};
    p.w_sf = static_cast<const uint8_t *>(w_block_scale);
    p.x_sf = static_cast<const uint8_t *>(block_scale);
    p.alpha = alpha;
    p.bias = static_cast<const uint16_t *>(bias);
    p.y = y;
    p.M = M;
    p.N = (int)N;
    p.K64 = (int)(K / 64);
    p.err = d->err;
    p.wait_limit = wait_limit_cycles();
    p.tx_extra = inject_timeout_on() ? 16u : 0u;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (M > 128) {
        e = launch_linear_pair(p, q, w_q, out_type, bias_type, d->sms, s);
        if (e == cudaSuccess) return GNQ_OK;
        cudaGetLastError();
        return GNQ_ERR_CUDA;
    }
    int64_t grid = 0;
    size_t smem = 0;
    if (!shape_of(*d, M, N, K, p, grid, smem)) return GNQ_ERR_SHAPE;
    CUtensorMap mw, mx;
    if (!encode_codes(&mw, w_q, N, K, kTileN) || !encode_codes(&mx, q, M, K, p.T)) return GNQ_ERR_CUDA;
    if (out_type == GNQ_BF16) e = launch_linear<__nv_bfloat16, __nv_bfloat16>(mw, mx, p, grid, smem, s);
    else if (out_type == GNQ_FP16) e = launch_linear<__half, __half>(mw, mx, p, grid, smem, s);
    else if (bias_type == GNQ_FP16) e = launch_linear<float, __half>(mw, mx, p, grid, smem, s);
    else e = launch_linear<float, __nv_bfloat16>(mw, mx, p, grid, smem, s);
    if (e == cudaSuccess) return GNQ_OK;
    cudaGetLastError();
    return GNQ_ERR_CUDA;
}
