// Router of a mixture of experts: the k largest logits of each token, their
// softmax weights, and the rows of the chosen experts.  The contract is in
// include/gemma_nq.h.
//
//   experts[t, j]  index of the j-th largest logit of token t, equal ones by
//                  index; -1 where only -inf is left
//   weights[t, j]  scale * exp(l_j - l_0) / sum, over the chosen or over all
//   slots[t, j]    row of (t, j) in expert order: by expert, then by token
//   offsets[e]     first row of expert e
//
// Two steps.  A warp per token picks and weighs.  Then the M k choices are
// placed by counting: each warp counts a contiguous stretch of them in its own
// histogram, a prefix over warps, CTAs of a cluster and experts gives every
// warp the first row of its choices of each expert, and a second pass over
// the same stretch places them.  No atomics: the rows of an expert are in
// token order whatever the timing.
#include "gemma_nq.h"
#include "gnq_expert.cuh"
#include "gnq_host.cuh"
#include "gnq_launch.cuh"
#include "gnq_tcgen05.cuh"

namespace gnq {
namespace {

struct RouteParams {
    const void *logits;
    int64_t row_stride;
    int M, E, k;
    bool renormalize;
    float scale;
    int32_t *experts, *offsets, *slots;
    float *weights;
};

constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // order_key(-inf)

// Unsigned order of fp32 values: equal zeros, NaN above all.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 -> +0
    if (v != v) return 0xFFFFFFFFu;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {  // of a key that is not NaN's
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

template <typename L> __device__ __forceinline__ float load_logit(const void *p, int64_t i);
template <> __device__ __forceinline__ float load_logit<float>(const void *p, int64_t i) {
    return ld_f32(static_cast<const float *>(p) + i);
}
template <> __device__ __forceinline__ float load_logit<__nv_bfloat16>(const void *p, int64_t i) {
    return __uint_as_float((uint32_t)ld_u16(static_cast<const uint16_t *>(p) + i) << 16);
}
template <> __device__ __forceinline__ float load_logit<__half>(const void *p, int64_t i) {
    return __half2float(__ushort_as_half(ld_u16(static_cast<const uint16_t *>(p) + i)));
}

// One token by one warp; lane l holds the logits of experts l, l + 32, ...
template <typename L, int NV> __device__ __forceinline__ void pick_token(const RouteParams &p, int t, int lane) {
    uint32_t key[NV];
    const int64_t row = (int64_t)t * p.row_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = 32 * i + lane;
        key[i] = e < p.E ? order_key(load_logit<L>(p.logits, row + e)) : 0u;
    }
    auto value = [&](uint32_t u) { return u == 0xFFFFFFFFu ? __int_as_float(0x7FC00000) : key_value(u); };
    uint32_t all[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) all[i] = key[i];

    // lane j keeps the j-th choice
    uint32_t mine = 0;
    int choice = -1;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top <= kKeyNegInf) break;
        const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)(32 * at + lane) : 0x7FFFFFFFu);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (e == 32 * i + lane) key[i] = 0;
        if (lane == j) mine = top, choice = e;
    }
    const uint32_t first = __shfl_sync(0xffffffffu, mine, 0);
    float w = 0.f;
    if (first != 0) {  // (warp-uniform)
        const float peak = value(first);
        w = choice >= 0 ? expf(value(mine) - peak) : 0.f;
        float part = w;
        if (!p.renormalize) {
            part = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (all[i] > 0) part += expf(value(all[i]) - peak);
        }
        const float total = warp_sum(part);
        if (choice >= 0) w = __fmul_rn(__fdiv_rn(w, total), p.scale);
    }
    if (lane < p.k) {
        const int64_t at = (int64_t)t * p.k + lane;
        p.experts[at] = choice;
        p.weights[at] = w;
    }
}

// Rows of the M k choices, by a cluster of CTAs (or one) of 1024 threads.
// hist: per warp and expert; totals: per CTA and expert.
__device__ __forceinline__ void place_choices(const RouteParams &p, int32_t *hist, int32_t *totals, int32_t *sums) {
    constexpr int W = 32;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const uint32_t C = cluster_size(), rank = C > 1 ? cluster_rank() : 0;
    const int64_t n = (int64_t)p.M * p.k;
    const int64_t per = ((n + C * W - 1) / (C * W) + 31) / 32 * 32;
    const int64_t begin = min(n, (int64_t)(rank * W + warp) * per), end = min(n, begin + per);
    int32_t *const h = hist + warp * p.E;

    for (int i = t; i < W * p.E; i += 1024) hist[i] = 0;
    __syncthreads();
    const uint32_t below = (1u << lane) - 1;
    // place < 0: counts; else hands out rows
    auto pass = [&](bool place) {
        for (int64_t i = begin + lane; i - lane < end; i += 32) {
            const int e = i < end ? p.experts[i] : -1;
            const uint32_t peers = __match_any_sync(0xffffffffu, e);
            const int before = __popc(peers & below);
            int row = -1;
            if (e >= 0) row = h[e] + before;
            __syncwarp();
            if (e >= 0 && before == 0) h[e] += __popc(peers);
            __syncwarp();
            if (place && i < end) p.slots[i] = row;
        }
    };
    pass(false);
    __syncthreads();
    // counts -> prefix over the warps; one expert per thread
    int total = 0;
    if (t < p.E)
        for (int w = 0; w < W; ++w) {
            const int c = hist[w * p.E + t];
            hist[w * p.E + t] = total;
            total += c;
        }
    int before = 0;
    if (C > 1) {
        cluster_wait();  // every CTA exists
        if (t < p.E)
            for (uint32_t r = 0; r < C; ++r)
                st_cluster_u32(map_to_cta((uint32_t)__cvta_generic_to_shared(totals + rank * p.E + t), r), (uint32_t)total);
        cluster_arrive_release();
        cluster_wait();
        if (t < p.E) {
            total = 0;
            for (uint32_t r = 0; r < C; ++r) {
                const int c = totals[r * p.E + t];
                if (r < rank) before += c;
                total += c;
            }
        }
    }
    // prefix over the experts
    int sum = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += sums[w];
    const int offset = base + sum - total;
    if (t < p.E) {
        for (int w = 0; w < W; ++w) hist[w * p.E + t] += offset + before;
        if (rank == 0) {
            p.offsets[t] = offset;
            if (t == p.E - 1) p.offsets[p.E] = offset + total;
        }
    }
    __syncthreads();
    pass(true);
}

template <typename L, int NV> __global__ void __launch_bounds__(256) route_pick_kernel(const __grid_constant__ RouteParams p) {
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t < p.M) pick_token<L, NV>(p, t, threadIdx.x & 31);
}

__global__ void __launch_bounds__(1024) route_place_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ int32_t counts[];
    __shared__ int32_t sums[32];
    if (cluster_size() > 1) cluster_arrive_relaxed();
    pdl_wait();
    pdl_trigger();
    place_choices(p, counts, counts + 32 * p.E, sums);
}

// Both steps in one CTA.
template <typename L, int NV> __global__ void __launch_bounds__(1024) route_small_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ int32_t counts[];
    __shared__ int32_t sums[32];
    pdl_wait();
    pdl_trigger();
    for (int t = threadIdx.x >> 5; t < p.M; t += 32) pick_token<L, NV>(p, t, threadIdx.x & 31);
    __syncthreads();
    place_choices(p, counts, nullptr, sums);
}

constexpr int kPlaceCluster = 8;

template <typename L, int NV> cudaError_t launch_route(const RouteParams &p, cudaStream_t s) {
    const size_t hist = (size_t)32 * p.E * 4;
    if (p.M <= 64) {
        auto fn = route_small_kernel<L, NV>;
        const cudaError_t e = opt_in_dynamic_smem(reinterpret_cast<const void *>(fn));
        return e != cudaSuccess ? e : launch(fn, 1, 1024, hist, 1, s, p);
    }
    cudaError_t e = opt_in_dynamic_smem(reinterpret_cast<const void *>(route_place_kernel));
    if (e != cudaSuccess) return e;
    if ((e = launch(route_pick_kernel<L, NV>, (p.M + 7) / 8, 256, 0, 1, s, p)) != cudaSuccess) return e;
    return launch(route_place_kernel, kPlaceCluster, 1024, hist + (size_t)kPlaceCluster * p.E * 4, kPlaceCluster, s, p);
}

template <typename L> cudaError_t launch_route_experts(const RouteParams &p, cudaStream_t s) {
    if (p.E <= 32) return launch_route<L, 1>(p, s);
    if (p.E <= 64) return launch_route<L, 2>(p, s);
    if (p.E <= 128) return launch_route<L, 4>(p, s);
    if (p.E <= 256) return launch_route<L, 8>(p, s);
    if (p.E <= 512) return launch_route<L, 16>(p, s);
    return launch_route<L, 32>(p, s);
}

}  // namespace
}  // namespace gnq

extern "C" int gnq_expert_route(const void *logits, int64_t row_stride, int logits_type, int64_t M, int64_t E, int k,
                                int renormalize, float scale, int32_t *experts, float *weights, int32_t *offsets,
                                int32_t *slots, void *stream) {
    using namespace gnq;
    if (logits_type < GNQ_BF16 || logits_type > GNQ_FP32) return GNQ_ERR_DTYPE;
    if (E < 1 || E > kMaxExperts || k < 1 || k > kMaxTopK || k > E) return GNQ_ERR_SHAPE;
    if (M < 0 || M > kMaxM || M * k > 0x7FFFFFFF) return GNQ_ERR_SHAPE;
    const int64_t size = logits_type == GNQ_FP32 ? 4 : 2;
    if (row_stride < E || row_stride > (int64_t)1 << 32) return GNQ_ERR_ALIGN;
    if (!offsets || (M > 0 && (!logits || !experts || !weights || !slots))) return GNQ_ERR_NULL;
    if (!aligned(logits, size) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(slots, 4))
        return GNQ_ERR_ALIGN;
    const Extent written[] = {extent(experts, 4 * M * k), extent(weights, 4 * M * k), extent(slots, 4 * M * k),
                              extent(offsets, 4 * (E + 1))};
    const Extent read[] = {{logits, M, size * row_stride, size * E}};
    if (outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    RouteParams p = {};
    p.logits = logits;
    p.row_stride = row_stride;
    p.M = (int)M;
    p.E = (int)E;
    p.k = k;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    p.experts = experts;
    p.weights = weights;
    p.offsets = offsets;
    p.slots = slots;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (logits_type == GNQ_BF16) return status_of(launch_route_experts<__nv_bfloat16>(p, s));
    if (logits_type == GNQ_FP16) return status_of(launch_route_experts<__half>(p, s));
    return status_of(launch_route_experts<float>(p, s));
}
