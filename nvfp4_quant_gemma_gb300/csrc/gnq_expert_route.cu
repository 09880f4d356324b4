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
// A warp per token picks and weighs.  The M k choices are then placed by
// counting, without atomics on memory: an expert's rows are in token order
// whatever the timing.  Up to 4096 choices one CTA does it: each warp counts a
// contiguous stretch in a histogram of its own, a prefix over warps and
// experts gives its first row of each expert.  More are cut into chunks of
// tokens: the CTA that picks a chunk leaves its counts in the slots that the
// chunk will have (it has at least as many choices as there are experts), a
// cluster turns them into first rows, an expert's slice per CTA, and a CTA per
// chunk places its choices as above.  (Where that makes fewer chunks than SMs,
// the counting is a step of its own.)
//
// What bounds it: picking is the integer pipes (420 warp instructions a token of 256
// fp32 logits, 5.7 us for 16384 tokens at every issue slot, take 10: 58 % of the slots,
// and a full pipe is what warps wait for most), placing latency.  16384 tokens: 256 fp32
// logits, 8 choices 20 us, 128 bf16 logits 17, 64 and 2 choices 13.9; 65536 of the first
// 56 us (1.2 TB/s of logits); one token 2.4 us.  One CTA or cluster that places all
// 131072 choices took 22 us by itself, the chunks' two steps take 9.
#include <algorithm>

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

// Unsigned order of a type's values, in the upper bits of a word: equal zeros,
// NaN above all.  The inverse gives a NaN for NaN's key.
template <typename L> struct Logit;
template <> struct Logit<float> {
    static constexpr uint32_t kNegInf = 0x007FFFFFu;
    static __device__ __forceinline__ uint32_t key(uint32_t b) {
        const float v = __uint_as_float(b) + 0.f;  // -0 -> +0
        return v != v ? 0xFFFFFFFFu : number_key(v);
    }
    static __device__ __forceinline__ uint32_t number_key(float v) {
        const uint32_t b = __float_as_uint(v);
        return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    }
    static __device__ __forceinline__ float value(uint32_t key) {
        return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
    }
};
template <typename L, uint32_t INF> struct Logit16 {
    static constexpr uint32_t kNegInf = (0xFFFFu - (INF | 0x8000u)) << 16;
    static __device__ __forceinline__ uint32_t key(uint32_t b) {
        if ((b & 0x7FFFu) > INF) return 0xFFFF0000u;
        if (b == 0x8000u) b = 0;
        return (b & 0x8000u ? 0xFFFFu - b : b | 0x8000u) << 16;
    }
    static __device__ __forceinline__ uint16_t bits(uint32_t key) {
        key >>= 16;
        return (uint16_t)(key & 0x8000u ? key & 0x7FFFu : 0xFFFFu - key);
    }
};
template <> struct Logit<__nv_bfloat16> : Logit16<__nv_bfloat16, 0x7F80u> {
    static __device__ __forceinline__ float value(uint32_t key) { return __uint_as_float((uint32_t)bits(key) << 16); }
};
template <> struct Logit<__half> : Logit16<__half, 0x7C00u> {
    static __device__ __forceinline__ float value(uint32_t key) { return __half2float(__ushort_as_half(bits(key))); }
};

// A logit's key and its expert, in order: by key, equal keys by falling index.
struct Ranked {
    uint32_t v, e;
    static __device__ __forceinline__ bool less(const Ranked &a, const Ranked &b) {
        return a.v < b.v || (a.v == b.v && a.e > b.e);
    }
};

// Bits of a lane's logits: experts lane * NV + i in wide loads (WIDE: E = 32 NV,
// rows 16-byte aligned), else 32 i + lane, 0 behind the last.
template <typename L, int NV, bool WIDE>
__device__ __forceinline__ void load_logits(const RouteParams &p, int t, int lane, uint32_t (&b)[NV]) {
    constexpr int S = sizeof(L), BYTES = NV * S;
    const uint8_t *row = static_cast<const uint8_t *>(p.logits) + (int64_t)t * p.row_stride * S;
    if constexpr (WIDE && BYTES >= 4) {
        uint32_t w[BYTES / 4];
        const uint8_t *at = row + lane * BYTES;
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                const uint4 v = ld_stream(at + 16 * i);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < BYTES / 4; ++i) w[i] = __float_as_uint(ld_f32(reinterpret_cast<const float *>(at) + i));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) b[i] = S == 4 ? w[i] : (w[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = WIDE ? lane * NV + i : 32 * i + lane;
            b[i] = 0;
            if (e < p.E) {
                if constexpr (S == 4) b[i] = __float_as_uint(ld_f32(reinterpret_cast<const float *>(row) + e));
                else b[i] = ld_u16(row + 2 * e);
            }
        }
    }
}

// The choices of a token from exact keys, the lane-th to each lane: a search
// through all of them for each.
template <int NV>
__device__ __noinline__ int pick_exact(const uint32_t (&key)[NV], int e0, int de, int k, uint32_t none, int lane) {
    uint32_t taken = 0;
    int choice = -1;
    for (int j = 0; j < k; ++j) {
        Ranked h = {0, 0x7FFFFFFFu};
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Ranked o = {taken >> i & 1 ? 0u : key[i], (uint32_t)(e0 + de * i)};
            if (Ranked::less(h, o)) h = o, at = i;
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, h.v);
        if (top <= none) break;
        const uint32_t e = __reduce_min_sync(0xffffffffu, h.v == top ? h.e : 0x7FFFFFFFu);
        if (h.v == top && h.e == e) taken |= 1u << at;
        if (lane == j) choice = (int)e;
    }
    return choice;
}

// One token by one warp.  A logit's key and all ones less its index share a
// word, the index in the low bits, so that one comparison orders both, ties by
// index, and a maximum names the expert.  16-bit keys fit beside the index;
// fp32 ones lose their low 8 bits (10 from 512 experts on): if two neighbours
// in the order, down to the first that is not chosen, are equal in what is
// left, the token is picked again from exact keys (16384 x 256 fp32 logits:
// 15.5 us with exact keys throughout).  So is one with a
// NaN, whose key the first look does not make (their sum is one, too).
// `b` holds the lane's logits.  Up to eight a lane are put in falling order (Batcher's merge
// exchange), so that a choice is a maximum over the lanes' first ones and a
// step in one lane; more are searched at each choice.  Returns the lane-th
// choice (-1: none).
template <typename L, int NV, bool WIDE>
__device__ __forceinline__ int pick_token(const RouteParams &p, int t, int lane, const uint32_t (&b)[NV]) {
    constexpr bool SORT = NV <= 8, EXACT = sizeof(L) == 2;
    constexpr uint32_t MASK = EXACT ? 0xFFFFu : NV <= 8 ? 0xFFu : 0x3FFu;
    constexpr uint32_t NONE = Logit<L>::kNegInf | MASK;  // up to here: -inf, or no expert
    const int e0 = WIDE ? lane * NV : lane;
    constexpr int DE = WIDE ? 1 : 32;
    uint32_t r[NV];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = e0 + DE * i;
        uint32_t key;
        if constexpr (EXACT) {
            key = Logit<L>::key(b[i]);
        } else {
            const float v = __uint_as_float(b[i]) + 0.f;  // -0 -> +0
            sum += v;
            key = Logit<float>::number_key(v);
        }
        r[i] = WIDE || e < p.E ? (key & ~MASK) | (MASK - e) : 0u;
    }
    auto order = [&](uint32_t &x, uint32_t &y) {
        const uint32_t m = max(x, y);
        y = min(x, y);
        x = m;
    };
    if constexpr (SORT) {
#pragma unroll
        for (int q = 1; q < NV; q *= 2)
#pragma unroll
            for (int d = q; d >= 1; d /= 2)
#pragma unroll
                for (int i = d % q; i + d < NV; i += 2 * d)
#pragma unroll
                    for (int c = 0; c < d; ++c)
                        if (i + c + d < NV && (i + c) / (2 * q) == (i + c + d) / (2 * q)) order(r[i + c], r[i + c + d]);
    }
    auto first = [&] {
        uint32_t h = r[0];
        if constexpr (!SORT) {
#pragma unroll
            for (int i = 1; i < NV; ++i) h = max(h, r[i]);
        }
        return __reduce_max_sync(0xffffffffu, h);
    };
    uint32_t mine = 0, last = 0;  // lane j keeps the j-th choice
    bool again = !EXACT && __any_sync(0xffffffffu, sum != sum);
    for (int j = 0;; ++j) {
        const uint32_t top = first();
        again |= !EXACT && ((top ^ last) & ~MASK) == 0;
        if (top <= NONE || j == p.k) break;
        last = top;
        if (lane == j) mine = top;
        if (EXACT && j + 1 == p.k) break;
        if constexpr (SORT) {
            const bool step = r[0] == top;
#pragma unroll
            for (int i = 0; i + 1 < NV; ++i) r[i] = step ? r[i + 1] : r[i];
            r[NV - 1] = step ? 0u : r[NV - 1];
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) r[i] = r[i] == top ? 0u : r[i];
        }
    }
    int choice = mine ? (int)(MASK - (mine & MASK)) : -1;
    if constexpr (!EXACT) {
        if (again) {  // (the same for the whole warp)
            uint32_t key[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) key[i] = WIDE || e0 + DE * i < p.E ? Logit<L>::key(b[i]) : 0u;
            choice = pick_exact<NV>(key, e0, DE, p.k, Logit<L>::kNegInf, lane);
        }
    }
    float v = 0.f;
    if (choice >= 0) {
        if constexpr (EXACT) v = Logit<L>::value(mine);
        else v = ld_f32(static_cast<const float *>(p.logits) + (int64_t)t * p.row_stride + choice);
    }
    const float peak = __shfl_sync(0xffffffffu, v, 0);
    float w = choice >= 0 ? expf(v - peak) : 0.f;
    float part = w;
    if (!p.renormalize) {
        part = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (WIDE || e0 + DE * i < p.E) part += expf(Logit<L>::value(Logit<L>::key(b[i])) - peak);
    }
    const float total = warp_sum(part);
    if (choice >= 0) w = __fmul_rn(__fdiv_rn(w, total), p.scale);
    if (lane < p.k) {
        const int64_t at = (int64_t)t * p.k + lane;
        p.experts[at] = choice;
        p.weights[at] = w;
    }
    return choice;
}

// Tokens first, first + step, ... before `end` by one warp, the next one's
// logits on their way meanwhile; `done` gets the lane-th choice of each.
template <typename L, int NV, bool WIDE, typename Done>
__device__ __forceinline__ void pick_tokens(const RouteParams &p, int first, int end, int step, int lane, const Done &done) {
    if (first >= end) return;
    uint32_t b[NV];
    load_logits<L, NV, WIDE>(p, first, lane, b);
    for (int t = first; t < end; t += step) {
        uint32_t next[NV];
        if (t + step < end) load_logits<L, NV, WIDE>(p, t + step, lane, next);
        done(pick_token<L, NV, WIDE>(p, t, lane, b));
#pragma unroll
        for (int i = 0; i < NV; ++i) b[i] = next[i];
    }
}

constexpr int kKeep = 4;        // groups of 32 choices whose place a warp keeps in registers
// One launch up to so many tokens and logits: more are picked faster by several
// SMs (E = 128: 16 tokens 3.3 us in one launch and 3.8 in two, 64 tokens 6.3 and 4.7).
constexpr int kSmallTokens = 32, kSmallLogits = 4096;
// Choices that one CTA places: 4096 take 8.7 us with the picks (E = 128, k = 8), 8192
// took 12.7, and in chunks 16384 take 9.2.
constexpr int kOneCta = 32 * 32 * kKeep;
constexpr int kScanCtas = 8;
constexpr int kPickWarps = 18;

// Choices begin .. end - 1 by one CTA: the place of each among those of its
// expert, plus first(expert).  hist: E words per warp, and E more.  `first` is called by
// thread e for expert e (at least E threads) with the expert's count, by all
// threads together.
template <typename First>
__device__ __forceinline__ void place_choices(const RouteParams &p, int begin, int end, int32_t *hist, const First &first) {
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, W = blockDim.x >> 5;
    const int per = ((end - begin + W - 1) / W + 31) / 32 * 32;  // choices of a warp
    const int busy = per ? (end - begin + per - 1) / per : 0;    // warps that have some
    const int from = min(end, begin + warp * per), to = min(end, from + per);
    int32_t *const h = hist + warp * p.E;
    for (int i = t; i < busy * p.E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    const uint32_t below = (1u << lane) - 1;
    int e[kKeep], at[kKeep];
    auto read = [&](int base) {
#pragma unroll
        for (int g = 0; g < kKeep; ++g) {
            const int i = base + 32 * g + lane;
            e[g] = i < to ? p.experts[i] : -1;
        }
    };
    const bool kept = per <= 32 * kKeep;  // else the places wait in the slots
    for (int base = from; base < to; base += 32 * kKeep) {
        read(base);
#pragma unroll
        for (int g = 0; g < kKeep; ++g) {
            if (base + 32 * g >= to) break;
            const uint32_t peers = __match_any_sync(0xffffffffu, e[g]);
            const int before = __popc(peers & below);
            at[g] = e[g] >= 0 ? h[e[g]] + before : 0;
            __syncwarp();
            if (e[g] >= 0 && before == 0) h[e[g]] = at[g] + __popc(peers);
            __syncwarp();
            if (!kept && base + 32 * g + lane < to) p.slots[base + 32 * g + lane] = at[g];
        }
    }
    __syncthreads();
    // counts -> prefix over the warps; one expert per thread, eight reads on
    // their way at a time
    int total = 0;
    if (t < p.E)
        for (int w = 0; w < busy; w += 8) {
            int c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = w + i < busy ? hist[(w + i) * p.E + t] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (w + i < busy) hist[(w + i) * p.E + t] = total;
                total += c[i];
            }
        }
    int32_t *const row0 = hist + W * p.E;
    const int row = first(total);
    if (t < p.E) row0[t] = row;
    __syncthreads();
    for (int base = from; base < to; base += 32 * kKeep) {
        if (!kept) read(base);
#pragma unroll
        for (int g = 0; g < kKeep; ++g) {
            const int i = base + 32 * g + lane;
            if (i < to) p.slots[i] = e[g] < 0 ? -1 : row0[e[g]] + h[e[g]] + (kept ? at[g] : p.slots[i]);
        }
    }
}

// Sum of `v` over the threads before this one (of at most 1024), and over all.
__device__ __forceinline__ int prefix(int v, int32_t *sums, int &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    const int u = lane < W ? sums[lane] : 0;
    all = __reduce_add_sync(0xffffffffu, u);
    return __reduce_add_sync(0xffffffffu, lane < warp ? u : 0) + sum - v;
}

// All choices by one CTA, offsets included.
__device__ __forceinline__ void place_all(const RouteParams &p, int32_t *hist, int32_t *sums) {
    place_choices(p, 0, p.M * p.k, hist, [&](int total) {
        int all;
        const int row = prefix(total, sums, all), t = threadIdx.x;
        if (t < p.E) p.offsets[t] = row;
        if (t == 0) p.offsets[p.E] = all;
        return row;
    });
}

// Few tokens: everything in one CTA.
template <typename L, int NV, bool WIDE>
__global__ void __launch_bounds__(1024) route_small_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ int32_t counts[];
    __shared__ int32_t sums[32];
    pdl_wait();
    pdl_trigger();
    const int W = blockDim.x >> 5;
    pick_tokens<L, NV, WIDE>(p, threadIdx.x >> 5, p.M, W, threadIdx.x & 31, [](int) {});
    __syncthreads();
    place_all(p, counts, sums);
}

__global__ void __launch_bounds__(1024) route_place_all_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ int32_t counts[];
    __shared__ int32_t sums[32];
    pdl_wait();
    pdl_trigger();
    place_all(p, counts, sums);
}

// The choices of `chunk` tokens (the last chunk: of what is left, less than
// twice as many), and their counts where the chunk's slots will be (chunks > 0).
template <typename L, int NV, bool WIDE>
__global__ void __launch_bounds__(32 * kPickWarps) route_pick_kernel(const __grid_constant__ RouteParams p, int chunk, int chunks) {
    extern __shared__ int32_t counts[];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x, lane = t & 31, W = blockDim.x >> 5;
    const int begin = blockIdx.x * chunk, end = (int)blockIdx.x + 1 < (int)gridDim.x ? begin + chunk : p.M;
    if (chunks) {
        for (int i = t; i < p.E; i += blockDim.x) counts[i] = 0;
        __syncthreads();
    }
    pick_tokens<L, NV, WIDE>(p, begin + (t >> 5), end, W, lane, [&](int choice) {
        if (chunks && choice >= 0) atomicAdd(&counts[choice], 1);
    });
    if (!chunks) return;
    __syncthreads();
    for (int i = t; i < p.E; i += blockDim.x) p.slots[(int64_t)begin * p.k + i] = counts[i];
}

// The same counts from choices that other CTAs have picked.
__global__ void __launch_bounds__(256) route_count_kernel(const __grid_constant__ RouteParams p, int chunk) {
    extern __shared__ int32_t counts[];
    pdl_wait();
    pdl_trigger();
    const int begin = blockIdx.x * chunk, end = (int)blockIdx.x + 1 < (int)gridDim.x ? begin + chunk : p.M;
    for (int i = threadIdx.x; i < p.E; i += blockDim.x) counts[i] = 0;
    __syncthreads();
    for (int i = begin * p.k + threadIdx.x; i < end * p.k; i += blockDim.x) {
        const int e = p.experts[i];
        if (e >= 0) atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.E; i += blockDim.x) p.slots[(int64_t)begin * p.k + i] = counts[i];
}

// Counts of the chunks -> first row of each chunk and expert, and the offsets.
// A cluster: each CTA takes a slice of the experts, `slice` of them (a power of
// two up to 128), its threads the slice side by side and the chunks in
// stretches.
__global__ void __launch_bounds__(1024) route_scan_kernel(const __grid_constant__ RouteParams p, int chunk, int chunks, int slice) {
    __shared__ int32_t part[1024], sums[32];
    __shared__ int32_t totals[kScanCtas];
    const int rank = (int)cluster_rank(), t = threadIdx.x;
    cluster_arrive_relaxed();
    pdl_wait();
    pdl_trigger();
    const int e = rank * slice + t % slice, stretch = t / slice, stretches = min(32, 1024 / slice);
    const int per = (chunks + stretches - 1) / stretches;
    const int from = min(chunks, stretch * per), to = min(chunks, from + per);
    const int step = chunk * p.k, mine = e < p.E ? to - from : 0;
    int32_t *const table = p.slots + (int64_t)from * step + e;
    // eight reads on their way at a time
    auto read = [&](int c, int (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < mine ? table[(c + i) * step] : 0;
    };
    int sum = 0;
    for (int c = 0; c < mine; c += 8) {
        int v[8];
        read(c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[i];
    }
    part[t] = sum;
    __syncthreads();
    // first stretch: the expert's total; every stretch: what comes before it
    int total = 0, before = 0;
    for (int i = 0; i < stretches; ++i) {
        const int v = part[i * slice + t % slice];
        if (i < stretch) before += v;
        total += v;
    }
    int all;
    const int within = prefix(t < slice ? total : 0, sums, all);
    cluster_wait();  // every CTA exists
    if (t < kScanCtas) st_cluster_u32(map_to_cta((uint32_t)__cvta_generic_to_shared(&totals[rank]), t), (uint32_t)all);
    if (t < slice) part[t] = within;
    cluster_arrive_release();
    cluster_wait();
    int slices = 0, rows = 0;
    for (int i = 0; i < kScanCtas; ++i) {
        if (i < rank) slices += totals[i];
        rows += totals[i];
    }
    const int first = slices + part[t % slice];
    if (t < slice && e < p.E) p.offsets[e] = first;
    if (rank == 0 && t == 0) p.offsets[p.E] = rows;
    int row = first + before;
    for (int c = 0; c < mine; c += 8) {
        int v[8];
        read(c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i < mine) table[(c + i) * step] = row;
            row += v[i];
        }
    }
}

__global__ void __launch_bounds__(1024) route_place_kernel(const __grid_constant__ RouteParams p, int chunk) {
    extern __shared__ int32_t counts[];
    pdl_wait();
    pdl_trigger();
    const int begin = blockIdx.x * chunk, end = (int)blockIdx.x + 1 < (int)gridDim.x ? begin + chunk : p.M;
    // read before any of the chunk's slots is written (place_choices writes
    // them behind its barriers, or provisional places behind the one here)
    const int row = (int)threadIdx.x < p.E ? p.slots[(int64_t)begin * p.k + threadIdx.x] : 0;
    __syncthreads();
    place_choices(p, begin * p.k, end * p.k, counts, [&](int) { return row; });
}

template <typename L, int NV, bool WIDE> cudaError_t launch_route_form(const RouteParams &p, int sms, cudaStream_t s) {
    const int hist = (p.E + 31) / 32;  // warps that hold a thread per expert
    auto one_cta = [&](auto fn, int warps) {
        const cudaError_t e = opt_in_dynamic_smem(reinterpret_cast<const void *>(fn));
        return e != cudaSuccess ? e : launch(fn, 1, 32 * warps, (size_t)(warps + 1) * p.E * 4, 1, s, p);
    };
    if (p.M <= kSmallTokens && p.M * p.E <= kSmallLogits) return one_cta(route_small_kernel<L, NV, WIDE>, std::max(hist, std::min(p.M, 32)));
    const int n = p.M * p.k;
    cudaError_t e;
    auto pick = route_pick_kernel<L, NV, WIDE>;
    if (n <= kOneCta) {
        if ((e = launch(pick, (p.M + 7) / 8, 256, 0, 1, s, p, 8, 0)) != cudaSuccess) return e;
        return one_cta(route_place_all_kernel, 32);
    }
    // two chunks per SM; a chunk has a choice at least for every expert
    const int chunk = std::max((p.E + p.k - 1) / p.k, (p.M + 2 * sms - 1) / (2 * sms)), chunks = p.M / chunk;
    int slice = 1;
    while (slice * kScanCtas < p.E) slice *= 2;
    if (chunks >= sms) {
        const int rounds = (chunk + kPickWarps - 1) / kPickWarps, pickers = (chunk + rounds - 1) / rounds;
        if ((e = launch(pick, chunks, 32 * pickers, (size_t)p.E * 4, 1, s, p, chunk, chunks)) != cudaSuccess) return e;
    } else {  // chunks of many experts are too few to pick in (2048 tokens of 1024 experts: 45.7 us so)
        if ((e = launch(pick, (p.M + 7) / 8, 256, 0, 1, s, p, 8, 0)) != cudaSuccess) return e;
        if ((e = launch(route_count_kernel, chunks, 256, (size_t)p.E * 4, 1, s, p, chunk)) != cudaSuccess) return e;
    }
    if ((e = launch(route_scan_kernel, kScanCtas, 1024, 0, kScanCtas, s, p, chunk, chunks, slice)) != cudaSuccess) return e;
    const int warps = std::max(hist, 8);
    if ((e = opt_in_dynamic_smem(reinterpret_cast<const void *>(route_place_kernel))) != cudaSuccess) return e;
    return launch(route_place_kernel, chunks, 32 * warps, (size_t)(warps + 1) * p.E * 4, 1, s, p, chunk);
}

template <typename L, int NV> cudaError_t launch_route(const RouteParams &p, int sms, cudaStream_t s) {
    if (p.E == 32 * NV && aligned(p.logits, 16) && p.row_stride * sizeof(L) % 16 == 0)
        return launch_route_form<L, NV, true>(p, sms, s);
    return launch_route_form<L, NV, false>(p, sms, s);
}

template <typename L> cudaError_t launch_route_experts(const RouteParams &p, int sms, cudaStream_t s) {
    if (p.E <= 32) return launch_route<L, 1>(p, sms, s);
    if (p.E <= 64) return launch_route<L, 2>(p, sms, s);
    if (p.E <= 128) return launch_route<L, 4>(p, sms, s);
    if (p.E <= 256) return launch_route<L, 8>(p, sms, s);
    if (p.E <= 512) return launch_route<L, 16>(p, sms, s);
    return launch_route<L, 32>(p, sms, s);
}

}  // namespace
}  // namespace gnq

extern "C" int gnq_expert_route(const void *logits, int64_t row_stride, int logits_type, int64_t M, int64_t E, int k,
                                int renormalize, float scale, int32_t *experts, float *weights, int32_t *offsets,
                                int32_t *slots, void *stream) {
    using namespace gnq;
    if (logits_type < GNQ_BF16 || logits_type > GNQ_FP32) return GNQ_ERR_DTYPE;
    if (E < 1 || E > kMaxExperts || k < 1 || k > kMaxTopK || k > E) return GNQ_ERR_SHAPE;
    if (M < 0 || M > kMaxM || M * k > 0x7FFF0000) return GNQ_ERR_SHAPE;
    const int64_t size = logits_type == GNQ_FP32 ? 4 : 2;
    if (row_stride < E || row_stride > (int64_t)1 << 32) return GNQ_ERR_ALIGN;
    if (!offsets || (M > 0 && (!logits || !experts || !weights || !slots))) return GNQ_ERR_NULL;
    if (!aligned(logits, size) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(slots, 4))
        return GNQ_ERR_ALIGN;
    const Extent written[] = {extent(experts, 4 * M * k), extent(weights, 4 * M * k), extent(slots, 4 * M * k),
                              extent(offsets, 4 * (E + 1))};
    const Extent read[] = {{logits, M, size * row_stride, size * E}};
    if (outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
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
    if (logits_type == GNQ_BF16) return status_of(launch_route_experts<__nv_bfloat16>(p, d->sms, s));
    if (logits_type == GNQ_FP16) return status_of(launch_route_experts<__half>(p, d->sms, s));
    return status_of(launch_route_experts<float>(p, d->sms, s));
}
