// Shared by the two NVFP4 product kernels: parameters, output types and the
// tensor maps of their operands.
#pragma once

#include "gnq_host.cuh"
#include "gnq_launch.cuh"
#include "gnq_tcgen05.cuh"

namespace gnq {

constexpr int kTileN = 128;      // weight rows per CTA
constexpr int kStageK = 256;     // elements of K per stage
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;     // CTAs that share a tile's K
constexpr uint32_t kBytesW = kTileN * kStageK / 2;
constexpr uint32_t kBytesSf = 4 * 512;

struct LinearParams {
    const uint8_t *w_sf, *x_sf;
    const float *alpha;
    const uint16_t *bias;
    void *y;
    int64_t M;
    int N, K64;       // K64: K / 64
    int T;            // tokens per tile: the N of the tensor core's product
    int n_tiles;      // weight tiles
    int split;        // CTAs (a cluster) that share a tile's K
    int stages;
    uint32_t tmem_cols;
    unsigned int *err;
    long long wait_limit;
    bool early_w;       // the weight's first stages are read before the wait on the preceding grid
    uint32_t tx_extra;  // test hook: bytes announced per stage beyond the copies
    int tx_cta;         // ... by this CTA of a split alone (-1: by all)
};

template <typename O> struct OutType;
template <> struct OutType<__nv_bfloat16> {
    static __device__ __forceinline__ float bias(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};
template <> struct OutType<__half> {
    static __device__ __forceinline__ float bias(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    static __device__ __forceinline__ __half round(float v) { return __float2half_rn(v); }
};

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

// Tile store of a chunk in shared memory; clipped at the edges of y.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                 "r"(y), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most the last `N` of this thread's committed groups still read shared memory.
template <int N> __device__ __forceinline__ void tma_store_wait() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Map of a row-major (rows, K) matrix of packed codes, loaded in tiles of
// `box` rows x 128 bytes; what lies outside reads as 0.
bool encode_codes(CUtensorMap *map, const void *codes, int64_t rows, int64_t K, int box);
// Map of swizzled block scales as rows of 512 bytes (128 rows x 64 elements
// of K), `rows` of them, loaded four at a time.
bool encode_scales(CUtensorMap *map, const void *scales, int64_t rows);

// Map of the same as tiles of K64 such rows, `tiles` of them, loaded as four
// rows of `box` neighbouring tiles.
bool encode_scale_tiles(CUtensorMap *map, const void *scales, int64_t tiles, int64_t K64, int box);

// Map of a row-major (M, N) output of 2- or 4-byte values, stored in tiles of
// 32 rows x 128 bytes.
bool encode_output(CUtensorMap *map, void *y, int64_t M, int64_t N, int size);

// Map of a row-major (R, N) 16-bit output, stored in tiles of 32 rows x 64 bytes.
bool encode_output_half(CUtensorMap *map, void *y, int64_t R, int64_t N);

// The kernel of large batches (gnq_linear_pair.cu): out_type as in the ABI.
cudaError_t launch_linear_pair(const LinearParams &p, const void *q, const void *w_q, int out_type,
                               int bias_type, int sms, cudaStream_t s);

}  // namespace gnq
