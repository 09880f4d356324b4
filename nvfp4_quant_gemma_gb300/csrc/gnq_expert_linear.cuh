// Shared by the two kernels of the products grouped by expert: parameters and
// the list of tiles, which every CTA builds for itself from the offsets.
#pragma once

#include "gnq_expert.cuh"
#include "gnq_linear.cuh"

namespace gnq {

struct ExpertLinearParams {
    LinearParams p;           // M: rows that exist; alpha, bias: of expert 0
    const int32_t *offsets;
    int E;
    int alpha_stride;         // 1: one alpha per expert, 0: one for all
};

// The tiles of a call: expert by expert, within an expert weight tile by
// weight tile, row tiles innermost, so that CTAs that run at a time share a
// weight tile.  In shared memory: the row tiles before each expert, and each
// expert's first row.  E + 1 entries each, then one word per warp.
struct TileList {
    const int *tiles_before, *row0;
    int E, T, n_tiles;
    int count;

    static __host__ __device__ constexpr uint32_t bytes(int E, int warps) { return (2 * (E + 1) + warps) * 4; }

    struct Tile {
        int e, n, row, rows, start;  // expert; weight tile; first row, rows that exist, expert's first row
    };

    // Tile `i` (< count), by a converged warp; `e` is the expert of an earlier tile.
    __device__ __forceinline__ Tile at(int i, int e, int lane) const {
        const int q = (int)((unsigned)i / (unsigned)n_tiles);
        uint32_t above;
        for (;; e += 32) {
            above = __ballot_sync(0xffffffffu, e + lane < E && tiles_before[e + lane + 1] > q);
            if (above) break;
        }
        return of(i, e + __ffs(above) - 1);
    }
    // Tile `i`, which is of expert `e`.
    __device__ __forceinline__ Tile of(int i, int e) const {
        const int before = tiles_before[e], tiles = tiles_before[e + 1] - before;
        const int j = i - before * n_tiles, n = (int)((unsigned)j / (unsigned)tiles), t = j - n * tiles;
        Tile x;
        x.e = e;
        x.n = n;
        x.start = row0[e];
        x.row = x.start + t * T;
        x.rows = min(T, row0[e + 1] - x.row);
        return x;
    }
};

// Builds the list with the whole CTA (warps x 32 threads), after the wait on
// the preceding grid.  Offsets that do not ascend from 0 within the R rows are reported
// and give an empty list: with others the tiles fit an int and every search ends.
__device__ __forceinline__ TileList build_tiles(const ExpertLinearParams &x, int T, int *smem, int warps) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, E = x.E, R = (int)x.p.M;
    int *const before = smem, *const row0 = smem + E + 1, *const sums = row0 + E + 1;
    const int per = (E + 32 * warps - 1) / (32 * warps), first = min(E, t * per), last = min(E, first + per);
    int mine = 0;
    bool bad = t == 0 && ld_i32(x.offsets) != 0;
    int from = row_bound(x.offsets, first, R);
    for (int e = first; e < last; ++e) {
        const int to = row_bound(x.offsets, e + 1, R);
        bad |= to < from || to != ld_i32(x.offsets + e + 1);
        row0[e] = from;
        before[e] = mine;
        mine += max(0, to - from + T - 1) / T;
        from = to;
    }
    if (first < E && last == E) row0[E] = from;
    if (bad) atomicOr(x.p.err, (unsigned)DEVERR_BAD_ROW);
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) sums[warp] = sum;
    const bool none = __syncthreads_or(bad) != 0;
    int base = sum - mine, total = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) base += sums[w];
        total += sums[w];
    }
    for (int e = first; e < last; ++e) before[e] += base;
    if (t == 0) before[E] = total;
    __syncthreads();
    return {before, row0, E, T, x.p.n_tiles, none ? 0 : total * x.p.n_tiles};
}

// The kernel of CTA pairs (gnq_expert_linear_pair.cu): out_type as in the ABI.
cudaError_t launch_expert_linear_pair(ExpertLinearParams x, const void *q, const void *w_q, int out_type, int bias_type,
                                      int sms, cudaStream_t s);

}  // namespace gnq
