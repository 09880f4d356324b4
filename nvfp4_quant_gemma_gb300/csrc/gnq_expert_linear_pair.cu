// Products grouped by expert on CTA pairs: tiles of 256 weight rows and up to
// 256 rows of one expert.
//
// As in the pair kernel of one weight, a pair of CTAs issues one product over
// both SMs and the sums of a tile leave tensor memory while the next tile's
// come in.  Here the weight takes the M side (256 rows, 128 per CTA) and the
// expert's rows the N side, as many as there are (rounded up to 32): a ragged
// last tile costs what its rows take in, not a whole tile.
//
// Tensor memory (512 columns) does not hold the sums of two tiles of 256 rows
// and the scales.  So it has a place for 256 rows (columns 0-255) and one for
// 192 (256-447), and the rows of an expert are taken 448 at a time, as 256 and
// the rest: a tile starts while the one before is on its way out of the other
// place.  A tile of at most 192 rows takes whichever place the one before it
// did not; two tiles of more in a row, and only those, wait for each other.
//
// Pairs take entries of the list in rounds, one each, and three warps of every CTA
// deal them: of the entries of a round the largest goes to the pair that has been dealt
// the least, and so on.  What runs at a time stays as near together as in the
// order of the list, and no pair ends much later than another.  (The experts'
// rows differ widely, and of some tens of entries in plain order the fullest pair had
// 15 to 60 % more than the average, now 2 to 10 %.  The two cases below took 235
// and 164 us in plain order, 225 and 143 dealt out; 257 and 159 with all entries by
// falling rows, which reads weights twice; 291 and 189 with each pair's share in
// one piece, where pairs that run at a time share nothing.)
//
// A lane holds one weight row.  16-bit sums go through shared memory, where each
// warp lays out 32 rows of y by its 32 outputs (64 bytes), and leave as a tile
// store of whole sectors, or row by row at an expert's end (8192 tokens to 8 of 64
// experts, N = 4096, K = 2048, before the deal: 233 us; 243 straight from the registers; 239
// with boxes of 128 bytes that two warps share, 277 with boxes of 16 rows).  Rows that
// a tile store cannot take, and 4-byte sums, whose rows are 128 bytes of a warp
// anyway, leave straight from registers.
//
// What bounds it: a stage is 36 to 40 KB into each SM, 590 cycles at 64 bytes a
// cycle, and as much for its products and the scale copies into tensor memory; the
// two meet with jitter at about 740.  The case above: 225 us, 4.9 PFLOP/s (the
// product of one weight on as many rows, 65536 x 4096 x 2048: 228); 2048 tokens to 8
// of 64, N = K = 4096: 143 us, where reading the weights and writing y take 114; to
// fp32 288 and 160 us, of 213 and 134.
// Copies that only prefetch into L2 take from the same 64 bytes (242 us).
//
// Warps of a CTA: 0 copies, 1 issues products (in the pair's first CTA), 2-9
// take sums out: two warps for each 32 weight rows, 64 rows in turn; 10-12
// deal.
#include <algorithm>

#include "gemma_nq.h"
#include "gnq_expert_linear.cuh"

namespace gnq {
namespace {

constexpr int kOutputs = 256;                 // weight rows of a tile
constexpr int kFirst = 256, kSecond = 192;    // rows of the two tiles that one entry of the list stands for
constexpr int kRows = kFirst + kSecond;
constexpr int kStages = 5;
constexpr int kMaxPairs = 96;                 // (of the 76 that the machine has)
constexpr int kDealWarp = 10, kPairWarps = kDealWarp + kMaxPairs / 32;
constexpr uint32_t kHalf = 128 * kStageK / 2;          // 128 rows of codes of one stage
constexpr uint32_t kStage = 2 * kHalf + 4 * kBytesSf;  // per CTA: weight, rows, weight scales, three tiles of row scales
constexpr uint32_t kBox = 32 * 64;                     // 32 rows x 64 bytes of y
constexpr uint32_t kPlaceCol = 256, kSfwCol = 448, kSfxCol = 464;  // tensor memory: second place, scales

// y of up to 32 rows (columns of `acc`) x this lane's weight row n.
template <typename O>
__device__ __forceinline__ void store_rows(O *y, int64_t stride, int n, int N, int live, const uint32_t (&acc)[32],
                                           float alpha, float bias, int lane) {
    auto result = [&](uint32_t v) { return fmaf(__uint_as_float(v), alpha, bias); };
    // Two 16-bit columns per lane: neighbouring lanes exchange, the even one
    // stores row i, the odd one i + 1.
    if constexpr (sizeof(O) == 2) {
        if (N % 2 == 0) {
            const int odd = lane & 1;
            const uint32_t halves = odd ? 0x3276 : 0x5410;
            O *o = y + n + (odd ? stride - 1 : 0);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const uint32_t own = Act<O>::pack2(result(acc[i]), result(acc[i + 1]));
                const uint32_t w = __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, 1), halves);
                if (n < N && i + odd < live) *reinterpret_cast<uint32_t *>(o) = w;
                o += 2 * stride;
            }
            return;
        }
    }
    if (n < N) {
        O *o = y + n;
#pragma unroll
        for (int i = 0; i < 32; ++i, o += stride)
            if (i < live) {
                const float v = result(acc[i]);
                if constexpr (std::is_same<O, float>::value) *o = v;
                else *o = OutType<O>::round(v);
            }
    }
}

// Arrival that a product waits for: the sums are in registers (the tensor
// memory fence before it says so) and nothing else has to be seen.  A release
// would wait for the stores of y that are under way, microseconds in which the
// warp takes no sums out (291 us against 241 in the case above).
__device__ __forceinline__ void arrive_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// What a tile takes, in the time that 32 rows of a stage take: the weight's side
// of its stages counts as eight of those.
// An entry of more than 256 rows is two tiles.
__device__ __forceinline__ int cost_of(int rows) { return (rows > kFirst ? 16 : 8) + (rows + 31) / 32; }

// What the deal hands to the other warps of its CTA: a weight tile and up to 448
// rows of an expert; rows = 0 behind the last.
struct __align__(16) Entry {
    int e, n, at, rows;  // expert, weight tile, first row in the expert, rows
};
constexpr int kRing = 4;
struct Ring {
    const Entry *slots;
    uint32_t bars;  // dealt [kRing], then taken [kRing]
    __device__ __forceinline__ uint32_t dealt(int i) const { return bars + 8u * i; }
    __device__ __forceinline__ uint32_t taken(int i) const { return bars + 8u * (kRing + i); }
};

// Where a pair is in its work: the entries dealt to it, each as one or two
// tiles, and the place in tensor memory of each tile.
struct Walk {
    int i = -1;                   // entries taken before this one
    Entry entry = {0, 0, 0, 0};
    int in = 0;                   // first row of the tile in its entry
    int at = 0, rows = 0;         // first row of the tile in its expert, rows
    int place = 1;                // 0: columns 0-255, 1: 256-447
    int use0 = 0, use1 = -1;      // tiles that have taken each place before this one

    // The next tile, by a converged warp; false behind the last.
    __device__ __forceinline__ bool next(const Ring &ring, int lane, long long limit, bool &ok) {
        (place ? use1 : use0) += 1;
        in += kFirst;
        if (in >= entry.rows) {
            ++i;
            ok = warp_wait_bounded(ring.dealt(i % kRing), i / kRing & 1, limit);
            if (!ok) return false;
            entry = ring.slots[i % kRing];
            __syncwarp();
            if (lane == 0) mbar_arrive(ring.taken(i % kRing));
            if (entry.rows == 0) return false;
            in = 0;
        }
        at = entry.at + in;
        rows = min(kFirst, entry.rows - in);
        place = rows > kSecond ? 0 : place ^ 1;
        return true;
    }
    __device__ __forceinline__ int use() const { return place ? use1 : use0; }
    // Rows of each CTA of the pair: half, rounded up to 16.
    __device__ __forceinline__ int half() const { return (rows + 31) / 32 * 16; }
    // 32-row groups of the tile's first scale tile before its first row, and
    // the scale tiles that it touches.
    __device__ __forceinline__ int shift() const { return (at & 127) >> 5; }
    __device__ __forceinline__ int scale_tiles() const { return (shift() + (rows + 31) / 32 + 3) / 4; }
};

struct Maps {
    CUtensorMap w, ws, y;  // weight codes and scales, output
    CUtensorMap x[3];      // row codes in boxes of 32, 64 and 128 rows
    CUtensorMap xs[3];     // row scales in boxes of 1, 2 and 3 tiles
};

// Load of whole scale tiles into this CTA, completing on a barrier of the
// pair's first CTA.
__device__ __forceinline__ void tma_load_tiles(uint32_t dst, const CUtensorMap *map, int k64, int tile, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(0), "r"(k64), "r"(tile), "r"(bar)
        : "memory");
}

template <typename O, typename B>
__global__ void __launch_bounds__(32 * kPairWarps, 1) expert_linear_pair_kernel(const __grid_constant__ Maps maps,
                                                                             const __grid_constant__ ExpertLinearParams x,
                                                                             bool tiled) {
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
    __shared__ __align__(16) uint4 topup[kStages];
    __shared__ Entry slots[kRing];
    __shared__ __align__(16) uint32_t sizes[kMaxPairs], loads[kMaxPairs], by_size[kMaxPairs];  // of the deal
    __shared__ int rank_of_pair, stop;
    __shared__ __align__(8) uint64_t ring_bars[2 * kRing];
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;

    const LinearParams &p = x.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t dyn0 = (uint32_t)__cvta_generic_to_shared(dyn), base = (dyn0 + 1023u) & ~1023u;
    const uint32_t bar0 = (uint32_t)__cvta_generic_to_shared(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };                          // first CTA's: both halves landed
    auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };             // each CTA's: products done with it
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * kStages + b); };      // each CTA's: a tile's sums are ready
    auto acc_free = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };  // first CTA's: they are out
    const uint32_t done = bar0 + 8u * (2 * kStages + 4);

    const Ring ring = {slots, (uint32_t)__cvta_generic_to_shared(ring_bars)};

    if (warp == 0 && lane == 0) {
        prefetch_map(&maps.w);
        prefetch_map(&maps.ws);
        prefetch_map(&maps.x[2]);
        prefetch_map(&maps.xs[1]);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_free(b), 16);
        }
        mbar_init(done, 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(ring.dealt(i), 1);
            mbar_init(ring.taken(i), rank == 0 ? 10 : 9);  // copies, sums, the first CTA's products
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        failed = 0;
        stop = 0;
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
    const TileList list = build_tiles(x, kRows, reinterpret_cast<int *>(dyn + (base - dyn0) + kStages * kStage + 8 * kBox), kPairWarps);

    const int KT = (p.K64 + 3) / 4;
    auto gave_up = [&] { return *(volatile int *)&failed != 0; };
    auto give_up = [&] {
        atomicOr(p.err, (unsigned)DEVERR_WAIT_TIMEOUT);
        *(volatile int *)&failed = 1;
    };
    auto next = [&](Walk &w) {
        bool ok = true;
        const bool more = w.next(ring, lane, 2 * p.wait_limit, ok);
        if (!ok) give_up();
        return more;
    };
    if (warp == 0) {
        // ---- copies ----
        int it = 0, s = 0;
        uint32_t parity = 1;  // of the wait on `empty`: passes at once in the first round
        const int sf_rows = (p.N + 127) / 128;
        Walk w;
        while (!__any_sync(0xffffffffu, gave_up()) && next(w)) {
            const int half = w.half(), x0 = list.row0[w.entry.e] + w.at + half * rank, sf_tiles = w.scale_tiles();
            const int box = half > 64 ? 2 : half > 32 ? 1 : 0;
            const CUtensorMap *const map_x = &maps.x[box], *const map_xs = &maps.xs[sf_tiles - 1];
            const uint32_t bytes = kHalf + (4096u << box) + (1 + sf_tiles) * kBytesSf;
            const int w0 = w.entry.e * p.N + w.entry.n * kOutputs + 128 * rank;
            const int ws = (w.entry.e * sf_rows + 2 * w.entry.n + rank) * p.K64;
            const int xs = (list.row0[w.entry.e] >> 7) + w.entry.e + (w.at >> 7);
            for (int kt = 0; kt < KT; ++kt, ++it) {
                if (!warp_wait_bounded(empty(s), parity, p.wait_limit)) {
                    give_up();
                    break;
                }
                if (elect_one()) {
                    const uint32_t at = base + kStage * s, bar = map_to_cta(full(s), 0);
                    if (rank == 0) mbar_expect_tx(full(s), 2 * bytes + p.tx_extra);
                    tma_load_pair(at, &maps.w, kt * 128, w0, bar);
                    tma_load_pair(at + kHalf, map_x, kt * 128, x0, bar);
                    tma_load_pair(at + 2 * kHalf, &maps.ws, 0, ws + 4 * kt, bar);
                    tma_load_tiles(at + 2 * kHalf + kBytesSf, map_xs, 4 * kt, xs, bar);
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
                if (p.tx_extra)
                    bulk_g2s((uint32_t)__cvta_generic_to_shared(&topup[s]), p.w_sf, p.tx_extra, full(s));
                mbar_wait_bounded(full(s), (j / kStages) & 1, p.wait_limit);
            }
    } else if (warp == 1 && rank == 0) {
        // ---- products ----
        int s = 0;
        uint32_t parity = 0;
        bool good = true;
        Walk w;
        // One tile with SF scale tiles of its rows: the loop that limits a
        // pair, so nothing in it branches or is worked out twice.
        auto tile = [&](auto sf) {
            constexpr int SF = decltype(sf)::value;
            const uint32_t idesc = __shfl_sync(0xffffffffu, idesc_nvfp4(256, 2 * w.half()), 0);
            const uint32_t acc = __shfl_sync(0xffffffffu, tmem + (w.place ? kPlaceCol : 0u), 0);
            const uint32_t sfw = __shfl_sync(0xffffffffu, tmem + kSfwCol, 0);
            const uint32_t sfx = __shfl_sync(0xffffffffu, tmem + kSfxCol, 0);
            const uint32_t shift = __shfl_sync(0xffffffffu, w.shift(), 0);
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
                        cp_scales<2>(sfw + 4 * k, desc_scales(at + (2 * kHalf + 512 * k) / 16));
#pragma unroll
                        for (int i = 0; i < SF; ++i)
                            cp_scales<2>(sfx + 12 * k + 4 * i,
                                         desc_scales(at + (2 * kHalf + (1 + i) * kBytesSf + 512 * k) / 16));
                        mma_nvfp4<2>(acc, desc_sw128(at + 2 * k), desc_sw128(at + kHalf / 16 + 2 * k), idesc, sfw + 4 * k,
                                     sfx + 12 * k + shift, kt > 0 || k > 0);
                    };
                    if (nk >= 4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) step(k);
                    } else {
                        for (int k = 0; k < nk; ++k) step(k);
                    }
                    tc_commit_pair(empty(s));
                    if (kt == KT - 1) tc_commit_pair(acc_full(w.place));
                }
                __syncwarp();
                if (++s == kStages) s = 0, parity ^= 1;
            }
        };
        while (good && next(w)) {
            if (!warp_wait_bounded(acc_free(w.place), (w.use() & 1) ^ 1, p.wait_limit)) {
                give_up();
                break;
            }
            tc_fence_after();
            const int sf_tiles = w.scale_tiles();
            if (sf_tiles == 1) tile(std::integral_constant<int, 1>{});
            else if (sf_tiles == 2) tile(std::integral_constant<int, 2>{});
            else tile(std::integral_constant<int, 3>{});
        }
        // every product is done before tensor memory goes away
        if (elect_one()) tc_commit_pair(done);
        __syncwarp();
        if (!mbar_wait_bounded(done, 0, p.wait_limit)) give_up();
    } else if (warp >= kDealWarp) {
        // ---- deal ----
        // Each CTA plays the whole deal by itself, a thread for each pair and
        // for each entry of a round.
        const int pair = blockIdx.x / 2, pairs = gridDim.x / 2, number = threadIdx.x - 32 * kDealWarp;
        auto sync = [] {
            __syncwarp();
            asm volatile("bar.sync 1, %0;" ::"n"(kMaxPairs) : "memory");
        };
        uint32_t load = number < pairs ? number : ~0u;  // of pair `number`: what it has x 128, and its number
        int e = 0;                                      // expert of the last round's entry
        int put = 0;
        for (int first = 0;; first += pairs) {
            // cost and number of the entry first + number, falling (cost 0: there is none)
            Entry entry = {0, 0, 0, 0};
            uint32_t size = number < pairs ? 127 - number : 0;
            if (number < pairs && first + number < list.count) {
                while (list.tiles_before[e + 1] * list.n_tiles <= first + number) ++e;
                const TileList::Tile tile = list.of(first + number, e);
                entry = {tile.e, tile.n, tile.row - tile.start, tile.rows};
                size += 128 * cost_of(tile.rows);
            }
            sizes[number] = size;
            loads[number] = load;
            sync();
            if (stop) break;  // the same for all: it is written behind the second sync only
            // their ranks; the first round as it comes, for an early start
            int of_size = number, of_load = number;
            if (first > 0) {
                of_size = of_load = 0;
#pragma unroll 4
                for (int j = 0; j < pairs; j += 4) {
                    const uint4 s = *reinterpret_cast<const uint4 *>(sizes + j), l = *reinterpret_cast<const uint4 *>(loads + j);
                    of_size += (s.x > size) + (s.y > size) + (s.z > size) + (s.w > size);
                    of_load += (l.x < load) + (l.y < load) + (l.z < load) + (l.w < load);
                }
            }
            // (no two pairs are further apart than an entry's cost, so this
            // leaves no load below 0, and none grows out of 32 bits)
            const uint32_t less = max((int)(loads[0] / 128) - 64, 0) * 128;
            if (number < pairs) by_size[of_size] = size & ~127u;
            if (number == pair) rank_of_pair = of_load;
            sync();
            const int mine = rank_of_pair;
            const bool more = by_size[mine] > 0;
            if (number < pairs) load += by_size[of_load] - less;
            if (more ? number < pairs && of_size == mine : number == 0) {
                if (!mbar_wait_bounded(ring.taken(put % kRing), (put / kRing & 1) ^ 1, 2 * p.wait_limit)) give_up();
                if (gave_up()) {
                    stop = 1;
                } else {
                    if (!more) entry.rows = 0;
                    slots[put % kRing] = entry;
                    mbar_arrive(ring.dealt(put % kRing));
                }
            }
            ++put;
            if (!more) break;
        }
    } else if (warp >= 2) {
        // ---- sums out ----
        // Warps 2-5 take rows 0-63 and 128-191 of a tile, warps 6-9 the
        // others, 32 at a time.
        const int quad = warp & 3, set = (warp - 2) >> 2;
        const uint32_t lanes = (uint32_t)quad << 21;  // 32 lanes per warp, lane number in bits 16-31
        const uint32_t box = base + kStages * kStage + kBox * (warp - 2);
        Walk w;
        while (next(w)) {
            const int n0 = w.entry.n * kOutputs + 128 * rank + 32 * quad, n = n0 + lane;
            const float alpha = ld_f32(p.alpha + w.entry.e * x.alpha_stride);
            const float bias = p.bias && n < p.N ? OutType<B>::bias(ld_u16(p.bias + (int64_t)w.entry.e * p.N + n)) : 0.f;
            const int row = list.row0[w.entry.e] + w.at;
            const bool ok = mbar_wait_bounded(acc_full(w.place), w.use() & 1, 2 * p.wait_limit) && !(p.tx_extra && gave_up());
            if (!__all_sync(0xffffffffu, ok)) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + lanes + (w.place ? kPlaceCol : 0u);
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
                const int c = 64 * (h & 2) + 64 * set + 32 * (h & 1), live = w.rows - c;  // rows of this chunk and behind
                uint32_t v[32];
                if (live > 0) {
                    tmem_ld32(acc + c, v);
                    tmem_wait(v);
                }
                if (h == 3) {  // all that this warp takes is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_relaxed(map_to_cta(acc_free(w.place), 0));
                }
                if (live <= 0) continue;
                O *const y = static_cast<O *>(p.y) + (int64_t)(row + c) * p.N;
                if constexpr (sizeof(O) == 2) {
                    if (tiled) {
                        if (lane == 0) tma_store_wait<0>();
                        __syncwarp();  // the box is free
                        const uint32_t at = box + 2u * lane;
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const uint32_t two = Act<O>::pack2(fmaf(__uint_as_float(v[i]), alpha, bias),
                                                               fmaf(__uint_as_float(v[i + 1]), alpha, bias));
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 64u * i), "h"((uint16_t)two) : "memory");
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 64u * (i + 1)), "h"((uint16_t)(two >> 16))
                                         : "memory");
                        }
                        if (live >= 32) fence_async_shared();
                        __syncwarp();  // all of it is written
                        if (live >= 32) {
                            if (lane == 0) {
                                if (n0 < p.N) tma_store_2d(&maps.y, n0, row + c, box);
                                tma_store_commit();
                            }
                        } else {
                            // rows of the next expert stay: two rows in one go
                            const int col = n0 + 2 * (lane & 15);
                            O *const o = y + col;
                            if (col < p.N)
                                for (int r = lane >> 4; r < live; r += 2) {
                                    uint32_t two;
                                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(two) : "r"(box + 64u * r + 4u * (lane & 15)));
                                    *reinterpret_cast<uint32_t *>(o + (int64_t)r * p.N) = two;
                                }
                        }
                        __syncwarp();
                        continue;
                    }
                }
                store_rows<O>(y, p.N, n, p.N, live, v, alpha, bias, lane);
                __syncwarp();
            }
        }
        if (lane == 0) tma_store_wait<0>();  // shared memory is read before it goes away
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
cudaError_t launch_pair(const Maps &m, const ExpertLinearParams &x, bool tiled, int64_t grid, size_t smem,
                        cudaStream_t s) {
    auto fn = expert_linear_pair_kernel<O, B>;
    const cudaError_t e = opt_in_dynamic_smem(reinterpret_cast<const void *>(fn));
    if (e != cudaSuccess) return e;
    return launch(fn, grid, 32 * kPairWarps, smem, 2, s, m, x, tiled);
}

}  // namespace

cudaError_t launch_expert_linear_pair(ExpertLinearParams x, const void *q, const void *w_q, int out_type, int bias_type,
                                      int sms, cudaStream_t s) {
    LinearParams &p = x.p;
    p.n_tiles = (p.N + kOutputs - 1) / kOutputs;
    const int64_t K = (int64_t)p.K64 * 64, E = x.E, R = p.M;
    const int64_t w_rows = E * ((p.N + 127) / 128) * p.K64;
    const int64_t tiles = (R / kRows + std::min(E, R)) * p.n_tiles;  // at most
    if (tiles > 0x3FFFFFFF || w_rows > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const bool tiled = out_type != GNQ_FP32 && p.N % 8 == 0;  // rows of y are 16-byte aligned
    Maps m = {};
    bool ok = encode_codes(&m.w, w_q, E * p.N, K, 128) && encode_scales(&m.ws, p.w_sf, w_rows) &&
              (!tiled || encode_output_half(&m.y, p.y, R, p.N));
    for (int i = 0; i < 3; ++i)
        ok = ok && encode_codes(&m.x[i], q, R, K, 32 << i) && encode_scale_tiles(&m.xs[i], p.x_sf, R / 128 + E, p.K64, i + 1);
    if (!ok) return cudaErrorInvalidValue;
    const int64_t grid = 2 * std::min<int64_t>(tiles, std::min(sms / 2, kMaxPairs));
    const size_t smem = 1024 + kStages * kStage + 8 * kBox + TileList::bytes(x.E, kPairWarps);
    if (out_type == GNQ_BF16) return launch_pair<__nv_bfloat16, __nv_bfloat16>(m, x, tiled, grid, smem, s);
    if (out_type == GNQ_FP16) return launch_pair<__half, __half>(m, x, tiled, grid, smem, s);
    if (bias_type == GNQ_FP16) return launch_pair<float, __half>(m, x, tiled, grid, smem, s);
    return launch_pair<float, __nv_bfloat16>(m, x, tiled, grid, smem, s);
}

}  // namespace gnq
