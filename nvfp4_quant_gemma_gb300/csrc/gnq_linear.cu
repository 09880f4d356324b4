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
// side (16 to 128), so a decode batch wastes no rows.  A scale tile of the
// 128x4 layout is 512 contiguous bytes for 128 rows x 64 elements, exactly
// what one copy into tensor memory takes, so scales are fetched by plain bulk
// copies.  K advances by 256 elements (128 bytes, one swizzle row) a stage.
//
// A decode batch is bound by the weight's bytes and, at these sizes, by
// latency: launch, the first copy, the join and the stores are 3.5 us of the
// 5.4 us of M = 16, N = 8192, K = 5120 (23.9 MB, 3.5 us at 6.8 TB/s; M = 1,
// N = 4096, K = 2048: 3.5 us).  So K is split until one round of CTAs fills
// the SMs, and the split is joined in shared memory across a cluster.
#include <algorithm>
#include <atomic>

#include "gemma_nq.h"
#include "gnq_linear.cuh"

namespace gnq {
namespace {

// Tokens of a tile that one CTA of a split adds: whole groups of four.
__host__ __device__ constexpr int join_block(int T, int split) { return ((T + split - 1) / split + 3) / 4 * 4; }

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
    __shared__ uint32_t cta_failed[kMaxSplit];  // of each CTA of the split, by its own account

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
    const uint32_t tx_extra = p.tx_cta < 0 || p.tx_cta == ks ? p.tx_extra : 0;

    // No CTA waits for another between taking tensor memory and giving it
    // back, so CTAs of several grids that share SMs cannot block each other:
    // the arrival that lets peers store here comes before, the join after.
    if (S > 1) cluster_arrive_relaxed();
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

    // Copies of the k-th 256 elements into stage s: the weight's tile and
    // scales, then the tokens'.  (The stage and its phase are counted, not
    // divided out: one warp issues every copy, and its loop is what limits a
    // CTA at these sizes.)
    const uint8_t *const w_sf = p.w_sf + ((int64_t)nt * p.K64 + 4 * k_begin) * 512;
    const uint8_t *const x_sf = p.x_sf + (t0 / 128 * p.K64 + 4 * k_begin) * 512;
    const int k64 = p.K64 - 4 * k_begin;  // 64-element steps from this CTA's first
    auto copy_w = [&](int k, int s) {
        const uint32_t at = base + stage_bytes * s, sf_bytes = 512u * min(4, k64 - 4 * k);
        mbar_expect_tx(full(s), kBytesW + bytes_x + 2 * sf_bytes + tx_extra);
        tma_load_2d(at, &map_w, (k_begin + k) * 128, n0, full(s));
        bulk_g2s(at + kBytesW + bytes_x, w_sf + k * 2048, sf_bytes, full(s));
    };
    auto copy_x = [&](int k, int s) {
        const uint32_t at = base + stage_bytes * s, sf_bytes = 512u * min(4, k64 - 4 * k);
        tma_load_2d(at + kBytesW, &map_x, (k_begin + k) * 128, (int)t0, full(s));
        bulk_g2s(at + kBytesW + bytes_x + kBytesSf, x_sf + k * 2048, sf_bytes, full(s));
    };
    // Constant weights (gnq_set_constant_weights): the first stages' come in
    // while the preceding grid drains.
    const int early = p.early_w ? min(n_k, p.stages) : 0;
    if (warp == 0 && elect_one())
        for (int i = 0; i < early; ++i) copy_w(i, i);
    __syncwarp();

    pdl_wait();  // inputs may come from the preceding grid, outputs may still be read by it
    pdl_trigger();

    // read now, used at the end
    const int row = warp * 32 + lane, n = n0 + row;
    const float alpha = ld_f32(p.alpha);
    const uint16_t bias16 = p.bias && n < p.N ? ld_u16(p.bias + n) : 0;

    auto give_up = [&] {
        atomicOr(p.err, (unsigned)DEVERR_WAIT_TIMEOUT);
        *(volatile int *)&failed = 1;
    };
    auto gave_up = [&] { return *(volatile int *)&failed != 0; };
    if (warp == 0) {
        // ---- copies ----
        int i = 0, s = 0;
        uint32_t parity = 1;  // of the wait on `empty`: passes at once in the first round
        for (; i < n_k; ++i) {
            if (!warp_wait_bounded(empty(s), parity, p.wait_limit)) {
                give_up();
                break;
            }
            if (elect_one()) {
                if (i >= early) copy_w(i, s);
                copy_x(i, s);
            }
            __syncwarp();
            if (++s == p.stages) s = 0, parity ^= 1;
        }
        // Every copy has landed before the shared memory goes away: the last
        // use of each stage (test hook: with the bytes that its announcement
        // lacks).
        if (lane == 0)
            for (int j = max(0, i - p.stages); j < max(i, early); ++j) {
                const int s = j % p.stages;
                if (mbar_wait_bounded(full(s), (j / p.stages) & 1, p.wait_limit)) continue;
                give_up();
                if (tx_extra) bulk_g2s((uint32_t)__cvta_generic_to_shared(&topup[s]), p.w_sf, tx_extra, full(s));
                mbar_wait_bounded(full(s), (j / p.stages) & 1, p.wait_limit);
            }
    } else if (warp == 1) {
        // ---- products ----
        const uint32_t idesc = idesc_nvfp4(kTileN, p.T);
        int s = 0;
        uint32_t parity = 0;
        for (int i = 0; i < n_k; ++i) {
            // (under the test hook a stage may complete late, by the copy that
            // makes up for the announcement)
            if (!warp_wait_bounded(full(s), parity, p.wait_limit) ||
                (tx_extra && __any_sync(0xffffffffu, gave_up()))) {
                give_up();
                break;
            }
            tc_fence_after();
            const int nk = k64 - 4 * i;
            if (elect_one()) {
                const uint32_t at = (base + stage_bytes * s) >> 4, sf = at + ((kBytesW + bytes_x) >> 4);
                auto scales = [&](int k) {
                    cp_scales<1>(sfw_col + 4 * k, desc_scales(sf + 32 * k));
                    cp_scales<1>(sfx_col + 4 * k, desc_scales(sf + kBytesSf / 16 + 32 * k));
                };
                auto product = [&](int k) {
                    mma_nvfp4<1>(tmem, desc_sw128(at + 2 * k), desc_sw128(at + kBytesW / 16 + 2 * k), idesc,
                                 sfw_col + 4 * k, sfx_col + 4 * k, i > 0 || k > 0);
                };
                if (nk >= 4) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) scales(k);
#pragma unroll
                    for (int k = 0; k < 4; ++k) product(k);
                } else {
                    for (int k = 0; k < nk; ++k) scales(k);
                    for (int k = 0; k < nk; ++k) product(k);
                }
                tc_commit(empty(s));
            }
            __syncwarp();
            if (++s == p.stages) s = 0, parity ^= 1;
        }
        if (elect_one()) tc_commit(acc_bar);
    }
    __syncwarp();

    // ---- epilogue ----
    if (!mbar_wait_bounded(acc_bar, 0, 2 * p.wait_limit)) give_up();
    tc_fence_after();
    __syncthreads();  // `failed` agreed on, every copy landed
    const bool good = !failed;
    const int rows = (int)min((int64_t)p.T, p.M - t0);  // tokens in the tile
    const float bias = OutType<B>::bias(bias16);  // bits 0: +0
    auto result = [&](float v) { return fmaf(v, alpha, bias); };
    auto store = [&](int64_t m, float v) {
        O *const o = static_cast<O *>(p.y) + m * p.N + n;
        if constexpr (std::is_same<O, float>::value) *o = result(v);
        else *o = OutType<O>::round(result(v));
    };
    auto free_tmem = [&] {
        tc_fence_before();
        __syncthreads();
        if (warp == 1) tmem_dealloc<1>(tmem, p.tmem_cols);
        __syncwarp();
    };
    const uint32_t lane_base = (uint32_t)warp << 21;  // 32 lanes per warp, lane number in bits 16-31
    if (S == 1) {
        // Two 16-bit columns per lane: neighbouring lanes exchange, the even
        // one stores token c + j, the odd one c + j + 1.
        const bool pairs = sizeof(O) == 2 && p.N % 2 == 0;
        if (good)
            for (int c = 0; c < rows; c += 16) {
                uint32_t v[16];
                __syncwarp();
                tmem_ld16(tmem + lane_base + c, v);
                tmem_wait(v);
                if constexpr (sizeof(O) == 2) {
                    if (pairs && c + 16 <= rows) {
                        const int odd = lane & 1;
                        O *o = static_cast<O *>(p.y) + (t0 + c + odd) * p.N + (n - odd);
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const uint32_t own = Act<O>::pack2(result(__uint_as_float(v[j])), result(__uint_as_float(v[j + 1])));
                            const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
                            if (n < p.N)
                                *reinterpret_cast<uint32_t *>(o) =
                                    odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
                            o += 2 * (int64_t)p.N;
                        }
                        continue;
                    }
                }
                if (n < p.N)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < rows) store(t0 + c + j, __uint_as_float(v[j]));
            }
        free_tmem();
    } else {
        // Join: CTA r adds the r-th block of tokens.  Every CTA stores its
        // partial sums of a block into the shared memory of the CTA that adds
        // it, [source][token / 4][weight row][token % 4], then each adds in
        // source order: one way across the cluster and one barrier, and the
        // order of the sum is fixed.  Each CTA tells the others along with the
        // sums whether it gave up: nobody stores a sum that lacks a part.
        const int blk = join_block(p.T, S);
        const uint32_t part = base + stage_bytes * p.stages + 16u * row;
        const uint32_t src = 16u * kTileN * (blk / 4);  // bytes of one source
        cluster_wait();
        if (t < S) st_cluster_u32(map_to_cta((uint32_t)__cvta_generic_to_shared(&cta_failed[ks]), t), !good);
        if (good) {
            int dst = -1, left = 0;
            uint32_t to = 0;
            for (int c = 0; c < rows; c += 16) {
                uint32_t v[16];
                __syncwarp();
                tmem_ld16(tmem + lane_base + c, v);
                tmem_wait(v);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    if (left == 0) {
                        left = blk;
                        to = map_to_cta(part + src * ks, ++dst);
                    }
                    if (c + j < rows) st_cluster_v4(to, v[j], v[j + 1], v[j + 2], v[j + 3]);
                    to += 16u * kTileN;
                    left -= 4;
                }
            }
        }
        free_tmem();
        cluster_arrive_release();
        cluster_wait();
        bool whole = true;
        for (int r = 0; r < S; ++r) whole &= cta_failed[r] == 0;
        if (whole && n < p.N)
            for (int i = 0; i < blk; i += 4) {
                const int c = ks * blk + i;
                if (c >= rows) break;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int r = 0; r < S; ++r) {
                    const uint4 u = lds_v4(part + src * r + 16u * kTileN * (i / 4));
                    v.x += __uint_as_float(u.x);
                    v.y += __uint_as_float(u.y);
                    v.z += __uint_as_float(u.z);
                    v.w += __uint_as_float(u.w);
                }
                store(t0 + c, v.x);
                if (c + 1 < rows) store(t0 + c + 1, v.y);
                if (c + 2 < rows) store(t0 + c + 2, v.z);
                if (c + 3 < rows) store(t0 + c + 3, v.w);
            }
    }
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

bool encode_scale_tiles(CUtensorMap *map, const void *scales, int64_t tiles, int64_t K64, int box) {
    const EncodeFn f = encode_fn();
    const cuuint64_t dims[3] = {128, (cuuint64_t)K64, (cuuint64_t)tiles}, strides[2] = {512, (cuuint64_t)K64 * 512};
    const cuuint32_t boxes[3] = {128, 4, (cuuint32_t)box}, step[3] = {1, 1, 1};
    return f && f(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(scales), dims, strides, boxes, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_output(CUtensorMap *map, void *y, int64_t M, int64_t N, int size) {
    return encode_tiles(map, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, y,
                        {(cuuint64_t)N, (cuuint64_t)M}, (cuuint64_t)N * size, {(cuuint32_t)(128 / size), 32},
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

bool encode_output_half(CUtensorMap *map, void *y, int64_t R, int64_t N) {
    return encode_tiles(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, y, {(cuuint64_t)N, (cuuint64_t)R}, (cuuint64_t)N * 2, {32, 32},
                        CU_TENSOR_MAP_SWIZZLE_NONE);
}

namespace {

// Shared memory of a split: half of an SM's where two stages fit it (two CTAs
// of one grid run there, or the next grid's start up beside the last ones of
// this one), else all.  Up to 64 tokens three stages are as many as help (M =
// 16, N = 8192, K = 5120 in four parts: 5.5, 5.3, 5.6 us with 2, 3, 4).
struct SplitShape {
    int stages;
    size_t smem;
};
SplitShape split_shape(const DevInfo &d, int T, int split, int KT) {
    const int64_t stage = kBytesW + T * 128 + 2 * kBytesSf;
    const int64_t join = split > 1 ? (int64_t)join_block(T, split) * split * kTileN * 4 : 0;
    const int64_t whole = d.smem_optin - 1024 - 512 - join, half = (d.smem_optin - 1024 - 512) / 2 - 1024 - join;
    const int64_t room = half >= 2 * stage ? half : whole;
    const int stages = std::max(
        1, (int)std::min<int64_t>({T <= 64 ? 3 : kMaxStages, room / stage, (KT + split - 1) / split}));
    return {stages, (size_t)(1024 + stages * stage + join)};
}

// Clusters of `split` CTAs that the device runs at a time with one CTA per SM
// (0 on error, for this call), asked once per device: SMs of a processing
// cluster that do not make a whole one stay idle (GB300: 76, 46, 36, 28, 23, 15,
// 15 for 2 to 8).
int resident_clusters(const DevInfo &d, int split) {
    static std::atomic<int> cached[kMaxDevices][kMaxSplit + 1];  // clusters + 1
    const int n = answer_once(cached[d.dev][split], [&] {
        auto fn = linear_kernel<__nv_bfloat16, __nv_bfloat16>;
        if (opt_in_dynamic_smem(reinterpret_cast<const void *>(fn)) != cudaSuccess) return -1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(split * d.sms), 1, 1);
        cfg.blockDim = dim3(128, 1, 1);
        cfg.dynamicSmemBytes = (size_t)d.smem_optin / 2 + 4096;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)split;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.numAttrs = 1;
        cfg.attrs = &attr;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg) == cudaSuccess) return clusters;
        cudaGetLastError();
        return -1;
    });
    return std::max(n, 0);
}

// Tile and split of a call: the smallest tile that holds the tokens (128 at
// most), and K split over the largest cluster of which all run at a time, each
// CTA keeping two stages of K or more.  A further round of CTAs costs more
// than a deeper split gives (M = 16, N = 8192, K = 5120: 7.8, 6.1, 5.8, 5.3 us
// for 1 to 4 parts, then 8.8 us for 6, in two rounds; N = 5120: 4.9 us for 6,
// 8.0 for 8).  At 64 tokens a join of more than six parts costs more too (N =
// 2048: 5.45 us for 6, 6.0 for 8).
void shape_of(const DevInfo &d, int64_t M, int64_t N, LinearParams &p, int64_t &grid, size_t &smem) {
    p.T = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    p.n_tiles = (int)((N + kTileN - 1) / kTileN);
    const int KT = (p.K64 + 3) / 4;
    const int64_t tiles = p.n_tiles * ((M + p.T - 1) / p.T);
    p.split = 1;
    if (tiles <= d.sms)
        for (int c = std::min(p.T >= 64 ? 6 : kMaxSplit, KT / 2); c > 1 && p.split == 1; --c) {
            const int64_t per_sm = d.smem_sm / ((int64_t)split_shape(d, p.T, c, KT).smem + 1024 + 512);
            if (resident_clusters(d, c) * per_sm >= tiles) p.split = c;
        }
    grid = tiles * p.split;
    const SplitShape ss = split_shape(d, p.T, p.split, KT);
    p.stages = ss.stages;
    smem = ss.smem;
    p.tmem_cols = p.T <= 32 ? 64 : p.T == 64 ? 128 : 256;
}

// Whether CTA pairs on 256 x 256 tiles take the call (more than 64 tokens).
// Both times follow the rounds of CTAs and the depth of K.  A round of the other
// kernel holds up to two CTAs per SM where their shared and tensor memory fit;
// with more CTAs than SMs two share what an SM takes in, and a stage of theirs
// costs 0.455 us against 0.37 alone.  Unsplit tiles of 4-byte outputs, or of odd rows, are stored value by
// value; pairs store an output with rows off 16 bytes, and 4-byte ones, more
// slowly.  The constants, in microseconds, are fits to shapes of 65 to 4096 tokens,
// 32 to 16384 outputs and a K of 64 to 8192, each timed in both kernels; on 2917
// such shapes, 843 of them with 4-byte outputs, the choice loses 0.6 % on average
// against the faster kernel, and more than 10 % on 69 (300 x 5000 x 4096: 7.9 us
// on 120 single CTAs, 10.6 on 40 pairs; 512 x 4096 x 4096: 8.0 on 128, 10.2; 2048 x
// 2048 x 1024, two per SM: 5.7 and 7.4; 128 x 2048 x 5120, split six ways: 7.8 and
// 10.9; 256 x 8192 x 5120: 12.9 and 12.0; 8192 x 8192 x 5120: 160 and 114).
bool pairs_take(const DevInfo &d, int64_t M, int64_t N, int out_size, const LinearParams &p, int64_t grid,
                size_t smem) {
    if (M <= 64) return false;
    const int KT = (p.K64 + 3) / 4, ks = (KT + p.split - 1) / p.split;
    const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256), pairs = d.sms / 2;
    const double rounds = (double)((tiles + pairs - 1) / pairs);
    const double pair = 3.2 + rounds * (2.2 + 0.31 * KT + (N * out_size % 16 ? 2.1 : 0.0) + (out_size == 4 ? 1.1 : 0.0));
    const bool share = 2 * (smem + 1024 + 512) <= (size_t)d.smem_sm && p.tmem_cols <= 256;
    const int64_t wave = share ? 2 * d.sms : d.sms, rest = grid % wave;
    const double whole = (double)(grid / wave) + (rest > (share ? d.sms : 0));  // rounds of `wave` CTAs
    const double one = share ? (double)(rest > 0 && rest <= d.sms) : whole, two = share ? whole : 0.0;
    const double slow = p.split == 1 && (out_size == 4 || N % 2) ? 2.1 : 0.0;
    const double single = 1.2 + one * (1.9 + 0.37 * ks + slow) + two * (2.8 + 0.455 * ks + 2 * slow) +
                          (p.split > 1 ? 3.0 : 0.0);
    return pair < single;
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

extern "C" int gnq_query_linear(int64_t M, int64_t N, int64_t K, int out_type, int *kernel, int *tokens, int *split) {
    using namespace gnq;
    if (!kernel || !tokens || !split) return GNQ_ERR_NULL;
    if (out_type < GNQ_BF16 || out_type > GNQ_FP32) return GNQ_ERR_DTYPE;
    if (M < 1 || M > kMaxM || N <= 0 || N > kMaxM || K <= 0 || K > kMaxH || K % 64 != 0) return GNQ_ERR_SHAPE;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
    LinearParams p = {};
    p.K64 = (int)(K / 64);
    int64_t grid = 0;
    size_t smem = 0;
    shape_of(*d, M, N, p, grid, smem);
    const bool pairs = grid > 0x7FFFFFFF || pairs_take(*d, M, N, out_type == GNQ_FP32 ? 4 : 2, p, grid, smem);
    *kernel = pairs ? 2 : 1;
    *tokens = pairs ? 256 : p.T;
    *split = pairs ? 1 : p.split;
    return GNQ_OK;
}

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
    if (!aligned(q, 16) || !aligned(block_scale, 16) || !aligned(w_q, 16) || !aligned(w_block_scale, 16) ||
        !aligned(y, 16) || !aligned(alpha, 4) || (bias && !aligned(bias, 2)))
        return GNQ_ERR_ALIGN;
    const Extent written[] = {extent(y, M * N * (out_type == GNQ_FP32 ? 4 : 2))};
    const Extent read[] = {extent(q, code_bytes(GNQ_NVFP4, M, K)),   extent(block_scale, scale_bytes(GNQ_NVFP4, M, K)),
                           extent(w_q, code_bytes(GNQ_NVFP4, N, K)), extent(w_block_scale, scale_bytes(GNQ_NVFP4, N, K)),
                           extent(alpha, 4),                         extent(bias, 2 * N)};
    if (outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
    for (const void *buf : {q, block_scale, w_q, w_block_scale, static_cast<const void *>(y)})
        if (!on_device(buf, d->dev)) return GNQ_ERR_MEMORY;
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
    p.tx_cta = -1;
    p.early_w = constant_weights_on();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    int64_t grid = 0;
    size_t smem = 0;
    shape_of(*d, M, N, p, grid, smem);
    const int forced = linear_policy();
    if (grid > 0x7FFFFFFF ||
        (forced ? forced == 2 : pairs_take(*d, M, N, out_type == GNQ_FP32 ? 4 : 2, p, grid, smem))) {
        e = launch_linear_pair(p, q, w_q, out_type, bias_type, d->sms, s);
        if (e == cudaSuccess) return GNQ_OK;
        cudaGetLastError();
        return GNQ_ERR_CUDA;
    }
    if (const int cta = inject_split_timeout(); cta >= 0 && cta < p.split && p.split > 1 && !p.tx_extra) {
        p.wait_limit = kTestWaitLimit;
        p.tx_extra = 16u;
        p.tx_cta = cta;
    }
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
