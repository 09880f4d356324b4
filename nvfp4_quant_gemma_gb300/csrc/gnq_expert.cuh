// Rows in expert order, shared by the operators of a mixture of experts.
//
// Expert e owns rows offsets[e] .. offsets[e + 1] - 1; offsets (E + 1 of them,
// ascending from 0) are on the device and nobody reads them on the host.  Its
// block scales start at the 128-row tile offsets[e] / 128 + e of the 128x4
// layout: no prefix sum over the experts before it is needed to find it, and
// no two experts meet, as ceil(c / 128) <= floor((o + c) / 128) - floor(o /
// 128) + 1.  R / 128 + E tiles hold any split of R rows.
#pragma once

#include "gnq_device.cuh"

namespace gnq {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;

// Reads of what the preceding grid may have written: not to be moved ahead of
// the wait for it.
__device__ __forceinline__ int ld_i32(const int32_t *p) {
    int v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// offsets[i] kept inside the R rows that exist, whatever it holds.
__device__ __forceinline__ int row_bound(const int32_t *offsets, int i, int R) {
    return min(max(ld_i32(offsets + i), 0), R);
}

// First expert that ends behind `row` (E if none does), by a converged warp:
// two levels of 32 bounds, so two dependent reads for any E up to 1024.
__device__ __forceinline__ int find_expert(const int32_t *offsets, int E, int row, int lane) {
    const int step = (E + 31) / 32;
    uint32_t above = __ballot_sync(0xffffffffu, ld_i32(offsets + min((lane + 1) * step, E)) > row);
    if (above == 0) return E;
    const int first = (__ffs(above) - 1) * step, i = min(first + lane + 1, E);
    above = __ballot_sync(0xffffffffu, lane < step && ld_i32(offsets + i) > row);
    return above ? first + __ffs(above) - 1 : E;  // (never 0: the last of these bounds is the one found above)
}

// Byte of the scale tile row of row `r` of an expert that starts at row `o`.
__device__ __forceinline__ int64_t expert_scale_row(int e, int o, int r, int Kp4) {
    return ((int64_t)(o >> 7) + e + (r >> 7)) * Kp4 * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

}  // namespace gnq
