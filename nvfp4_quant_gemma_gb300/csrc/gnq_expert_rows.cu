// Quantization of rows by expert, the way back, and the weighted combination
// of a token's rows.  The contracts are in include/gemma_nq.h.
//
//   quantize   q = quant(y) with the global scale of the row's expert, y = x
//              or dtype(act(gate) * up); a token's row goes to every row that
//              its slots name, or row r to row r
//   dequantize out = type(code * (block scale / global scale))
//   combine    out[t] = type(sum_j w[t, j] y[slots[t, j]] + add[t])
//
// One pass, a few operations per byte.  A thread owns whole units (a 16-element
// block, a pair of blocks, 8 elements) of a flat index, so rows of any width keep
// every lane busy.  The arithmetic that decides a code is that of the norm
// kernels, so equal 16-bit values and scales give equal codes whatever produced
// them.
//
// A token that goes to k experts is read once and written k times, each time
// with the codes of that expert's scale.  Measured: bf16 8192 x 4096 to 8 experts
// each 50.5 us (32 at the copy rate), and 48.6 with one scale for all, which encodes a
// block once in place of eight times: not the instructions (62 and 47 % of the issue
// slots) but the stores, whose path out of the SM is the busiest part in both, at two
// thirds: a store of scales fills a sector with four bytes, 134 MB leave the SMs for
// 75 MB of 4096 tokens.  SiLU of 65536 x 2048 104 us (100), tanh-GELU 109, no
// activation 52 (51); back to bf16 51 us (51), fp32 114 (90), E4M3 32 (31);
// combination of 8192 tokens' 8 rows x 4096 102 us (99), of fp32 rows 195 (197): HBM.
#include "gemma_nq.h"
#include "gnq_elementwise.cuh"
#include "gnq_expert.cuh"
#include "gnq_host.cuh"
#include "gnq_launch.cuh"
#include "gnq_tcgen05.cuh"

namespace gnq {
namespace {

constexpr int NT = 256;

struct ExpertRows {
    const int32_t *offsets;
    int E, R;            // experts, rows that the buffers in expert order hold
    const float *scale;  // one per expert, or one
    int scale_stride;    // 1 or 0
    unsigned int *err;
};

// The expert of row `m`, one past the last where it has none; `e` is a lower
// bound of it.
__device__ __forceinline__ int expert_from(const ExpertRows &x, int e, int m, int &o) {
    while (e < x.E && ld_i32(x.offsets + e + 1) <= m) ++e;
    o = 0;
    if (e < x.E) {
        o = row_bound(x.offsets, e, x.R);
        if (o > m) e = x.E;  // (check_offsets reports such offsets)
    }
    return e;
}

// Reports offsets that do not start at 0, fall or end behind the R rows.  A row
// looks only at its own expert's bounds, so a CTA of its own, the last of the
// grid, looks at all of them: no other waits for it.
__device__ __forceinline__ void check_offsets(const ExpertRows &x) {
    bool bad = false;
#pragma unroll 1
    for (int e = threadIdx.x; e <= x.E; e += NT) {
        const int o = ld_i32(x.offsets + e);
        bad |= o > x.R || (e == 0 ? o != 0 : o < ld_i32(x.offsets + e - 1));
    }
    if (bad) atomicOr(x.err, (unsigned)DEVERR_BAD_ROW);
}

// ---------------------------------------------------------------------------
// 16-bit rows -> NVFP4
// ---------------------------------------------------------------------------
struct ExpertQuantParams {
    ExpertRows x;
    const uint16_t *in;
    int64_t row_stride;
    const int32_t *slots, *experts;  // (M, k), or nullptr: row m goes to row m
    int k;
    uint8_t *q, *block_scale;
    int64_t units;  // 16-element blocks in all rows of `in`
    int H, upr;     // elements and units of a row
    int M;          // rows of `in`
    int wave;       // CTAs of the first wave, which prefetch before the wait
    int rows_ahead; // rows from a unit to the one prefetched in its place
};

// RN(g / v) for the value v of a block scale, from v and RN(1 / v) of a table in
// shared memory (0 for v = 0: then 1 / v counts as 0): the correction step of
// div_fma, exact for these g; other g divide.
__device__ __forceinline__ bool quotient_table_serves(float g) { return g >= 0x1p-100f && g <= 0x1p100f; }
__device__ __forceinline__ void fill_reciprocals(float2 (&tab)[128], int t) {
    if (t < 128) {
        const float v = e4m3_value(t);
        tab[t] = make_float2(v, t ? __frcp_rn(v) : 0.f);
    }
    __syncthreads();
}

// The codes and scale byte of a block `v` with amax / 6 = sixth for global
// scale g: the steps of epilogue_unit.  TABLE: for g that it serves, and worth its
// filling where a thread takes several quotients (SiLU of 16384 x 2048 in expert order, one each: 31.4
// us without, 34.0 with it).
template <bool TABLE>
__device__ __forceinline__ void nvfp4_block(const float (&v)[16], float sixth, float g, const float2 *tab, uint32_t &lo,
                                            uint32_t &hi, uint32_t &sf) {
    sf = e4m3x2(__fmul_rn(g, sixth), 0.f) & 0xFF;
    [[maybe_unused]] float es, q0;
    if constexpr (TABLE) {
        const float2 r = tab[sf];  // (g and amax are not below 0: no sign)
        es = div_fma(g, r.x, r.y, q0);
    } else {
        es = element_scale(g, sf);
    }
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = v[i];
    mul_arr_s<16>(x, es);
    lo = e2m1x8(&x[0]);
    hi = e2m1x8(&x[8]);
}

// B blocks of 16 a thread, side by side in a row.  Two in expert order without an
// activation, where a thread's search and addresses cost as much as its codes (65536 x
// 2048: 51 us, with one block 70, with four 59); one elsewhere: a token to its rows
// takes 50 us, with two 51, and with an activation a block is work enough (SiLU 104
// us, HBM).
template <typename T, int ACT, bool FAN, bool V8, int B>
__global__ void __launch_bounds__(NT) expert_quant_kernel(const __grid_constant__ ExpertQuantParams p) {
    __shared__ float2 tab[128];
    if (blockIdx.x + 1 == gridDim.x) {
        pdl_wait();
        pdl_trigger();
        check_offsets(p.x);
        return;
    }
    const int lane = threadIdx.x & 31, upr = p.upr / B;
    const int64_t at = (int64_t)blockIdx.x * NT + threadIdx.x;
    const bool ok = at < p.units / B;
    const int m = ok ? (int)(at / upr) : 0, col = ok ? (int)(at - (int64_t)m * upr) * 16 * B : 0;
    if (FAN) fill_reciprocals(tab, threadIdx.x);
    const uint16_t *src = p.in + m * p.row_stride + col;
    auto prefetch = [&](const uint16_t *at, bool last) {
        prefetch_l2_line(at, last);
        if (ACT != ACT_NONE) prefetch_l2_line(at + p.H, last);
    };
    // The first wave's units into L2 while the preceding grid drains, and later
    // the units that take this place three quarters of a round from now: hints.
    if ((int)blockIdx.x < p.wave && ok) prefetch(src, false);
    pdl_wait();
    pdl_trigger();
    uint4 y[B][2], u[B][2];
#pragma unroll
    for (int i = 0; i < B; ++i) {
        load_unit<T, V8>(src + 16 * i, y[i]);
        if constexpr (ACT != ACT_NONE) load_unit<T, V8>(src + p.H + 16 * i, u[i]);
    }
    if (p.rows_ahead && ok && m + p.rows_ahead < p.M) prefetch(src + p.rows_ahead * p.row_stride, true);
    // in expert order: the row's expert while its values are on their way, by
    // one search for the warp and from there each lane by itself
    [[maybe_unused]] int o = 0, e = 0;
    [[maybe_unused]] float own_scale = 0.f;
    if constexpr (!FAN) {
        e = find_expert(p.x.offsets, p.x.E, __shfl_sync(0xffffffffu, m, 0), lane);
        e = ok ? expert_from(p.x, e, m, o) : p.x.E;
        if (e < p.x.E) own_scale = ld_f32(p.x.scale + e * p.x.scale_stride);
    }
    float v[B][16], sixth[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
        if constexpr (ACT != ACT_NONE) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float g[8], f[8];
                Act<T>::unpack(y[i][c], g);
                Act<T>::unpack(u[i][c], f);
                auto activate = [&](auto far) {
#pragma unroll
                    for (int j = 0; j < 8; j += 2)
                        upk2(act_mul2<T, ACT, decltype(far)::value>(pk2(g[j], g[j + 1]), pk2(f[j], f[j + 1])), g[j], g[j + 1]);
                };
                if (__any_sync(0xffffffffu, gates_far<T, ACT>(y[i][c]))) activate(std::true_type{});
                else activate(std::false_type{});
                y[i][c] = pack8<T>(g);
            }
        }
        sixth[i] = div6(absmax16<T>(y[i][0], y[i][1]));
        Act<T>::unpack(y[i][0], &v[i][0]);
        Act<T>::unpack(y[i][1], &v[i][8]);
    }
    const int Kp4 = p.upr >> 2;
    uint8_t *const codes = p.q + (col >> 1), *const scales = p.block_scale + sf_col_offset(col);
    uint32_t code[2 * B], sf[B];
    auto encode = [&](auto table, float g) {
#pragma unroll
        for (int i = 0; i < B; ++i)
            nvfp4_block<decltype(table)::value>(v[i], sixth[i], g, tab, code[2 * i], code[2 * i + 1], sf[i]);
    };
    auto store = [&](int row, int64_t sf_row) {
        uint8_t *const q = codes + (int64_t)row * (p.H >> 1);
        if constexpr (B == 2) {
            st_v4(q, make_uint4(code[0], code[1], code[2], code[3]));
            st_u16(scales + sf_row, sf[0] | sf[1] << 8);
        } else {
            st_v2(q, code[0], code[1]);
            st_u8(scales + sf_row, sf[0]);
        }
    };
    if constexpr (FAN) {
        // The choices of a token by the lanes of the warp, one each, so that
        // their reads run side by side; then all units of the token in this
        // warp take them in turn.  A warp holds one token, or parts of a few.
        const bool shared = p.x.scale_stride == 0;
        if (shared) encode(std::false_type{}, ld_f32(p.x.scale));
        uint32_t left = __ballot_sync(0xffffffffu, ok);
        while (left) {
            const int token = __shfl_sync(0xffffffffu, m, __ffs(left) - 1);
            int row = -1;
            float g = 0.f;
            int64_t sf_row = 0;
            if (lane < p.k) {
                const int64_t tj = (int64_t)token * p.k + lane;
                const int e = ld_i32(p.experts + tj);
                row = ld_i32(p.slots + tj);
                const bool known = (unsigned)e < (unsigned)p.x.E;
                const int at = known ? e : 0;
                const int o = row_bound(p.x.offsets, at, p.x.R), to = row_bound(p.x.offsets, at + 1, p.x.R);
                if (!shared) g = ld_f32(p.x.scale + at);
                if (row >= 0 && (!known || row < o || row >= to)) {
                    atomicOr(p.x.err, (unsigned)DEVERR_BAD_ROW);
                    row = -1;
                }
                sf_row = expert_scale_row(at, o, row - o, Kp4);
            }
            const bool mine = ok && m == token;
            auto take = [&](auto whole, auto table) {
                for (uint32_t live = __ballot_sync(0xffffffffu, row >= 0); live; live &= live - 1) {
                    const int j = __ffs(live) - 1;
                    const int rj = __shfl_sync(0xffffffffu, row, j);
                    const int64_t sj = __shfl_sync(0xffffffffu, sf_row, j);
                    const float gj = __shfl_sync(0xffffffffu, g, j);
                    if (!decltype(whole)::value && !mine) continue;
                    if (!shared) encode(table, gj);
                    store(rj, sj);
                }
            };
            // (the common case apart: a warp of one token, scales that the table serves)
            const bool served = __all_sync(0xffffffffu, row < 0 || shared || quotient_table_serves(g));
            if (served && __all_sync(0xffffffffu, mine)) take(std::true_type{}, std::true_type{});
            else if (served) take(std::false_type{}, std::true_type{});
            else take(std::false_type{}, std::false_type{});
            left &= ~__ballot_sync(0xffffffffu, mine);
        }
    } else {
        if (e == p.x.E) return;
        encode(std::false_type{}, own_scale);
        store(m, expert_scale_row(e, o, m - o, Kp4));
    }
}

template <typename T, int ACT> cudaError_t launch_expert_quant(ExpertQuantParams &p, bool v8, cudaStream_t s) {
    auto start = [&](auto fn, int blocks, bool ahead) {
        const int64_t grid = (p.units / blocks + NT - 1) / NT + 1;  // (the last for check_offsets)
        if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
        p.wave = one_wave_ctas(reinterpret_cast<const void *>(fn), NT);
        const int upr = p.upr / blocks;
        p.rows_ahead = ahead ? (int)(((int64_t)p.wave * 3 / 4 * NT + upr - 1) / upr) : 0;
        return launch(fn, grid, NT, 0, 1, s, p);
    };
    constexpr int own = ACT == ACT_NONE ? 2 : 1;
    if (p.slots)
        return v8 ? start(expert_quant_kernel<T, ACT, true, true, 1>, 1, true)
                  : start(expert_quant_kernel<T, ACT, true, false, 1>, 1, true);
    return v8 ? start(expert_quant_kernel<T, ACT, false, true, own>, own, own == 1)
              : start(expert_quant_kernel<T, ACT, false, false, own>, own, own == 1);
}

template <typename T> cudaError_t launch_expert_quant_act(ExpertQuantParams &p, int act, bool v8, cudaStream_t s) {
    if (act == ACT_SILU) return launch_expert_quant<T, ACT_SILU>(p, v8, s);
    if (act == ACT_GELU_TANH) return launch_expert_quant<T, ACT_GELU_TANH>(p, v8, s);
    return launch_expert_quant<T, ACT_NONE>(p, v8, s);
}

// ---------------------------------------------------------------------------
// NVFP4 -> values
// ---------------------------------------------------------------------------
struct ExpertDequantParams {
    ExpertRows x;
    const uint8_t *q, *block_scale;
    void *out;
    int64_t pairs;  // pairs of 16-element blocks in all rows
    int ppr, Kp4;   // of a row; scale tiles per 128 rows
};

// P pairs a thread: two where the output is small (65536 x 2048 to E4M3: 32 us, with
// one 40, which is the instructions of the search and the addresses), else one.
// Both of a pair's quotients come first (EARLY): 32 registers then hold it, where
// values that wait for the second one take 37, and 44 to E4M3 (65536 x 2048: bf16 51.1
// us, with six CTAs on an SM in place of eight 54.4; E4M3 32.4 and 36.6).
template <int OUT, bool V8, int P>
__global__ void __launch_bounds__(NT) expert_dequant_kernel(const __grid_constant__ ExpertDequantParams p) {
    if (blockIdx.x + 1 == gridDim.x) {
        pdl_wait();
        pdl_trigger();
        check_offsets(p.x);
        return;
    }
    const int lane = threadIdx.x & 31, ppr = p.ppr / P;
    const int64_t at = (int64_t)blockIdx.x * NT + threadIdx.x;
    const bool ok = at < p.pairs / P;
    const int m = ok ? (int)(at / ppr) : 0, b = ok ? 2 * P * (int)(at - (int64_t)m * ppr) : 0;
    pdl_wait();
    pdl_trigger();
    uint4 code[P];
#pragma unroll
    for (int i = 0; i < P; ++i) code[i] = ok ? ld_stream(p.q + 16 * (P * at + i)) : make_uint4(0, 0, 0, 0);
    int o, e = find_expert(p.x.offsets, p.x.E, __shfl_sync(0xffffffffu, m, 0), lane);
    if (!ok) return;
    e = expert_from(p.x, e, m, o);
    if (e == p.x.E) return;
    const uint8_t *const scales = p.block_scale + expert_scale_row(e, o, m - o, p.Kp4) + (b >> 2) * 512 + (b & 3);
    const uint32_t sf = P == 2 ? (uint32_t)ld_i32(reinterpret_cast<const int32_t *>(scales)) : ld_u16(scales);
    const float g = p.x.scale ? ld_f32(p.x.scale + e * p.x.scale_stride) : 1.f;
#pragma unroll
    for (int i = 0; i < P; ++i) nvfp4_pair_out<OUT, V8, true>(p.out, (P * at + i) * 32, code[i], sf >> 16 * i, g);
}

template <int OUT> cudaError_t launch_expert_dequant(const ExpertDequantParams &p, cudaStream_t s) {
    constexpr int P = OUT == OUT_E4M3 ? 2 : 1;
    const int64_t grid = (p.pairs / P + NT - 1) / NT + 1;  // (the last for check_offsets)
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if (aligned(p.out, 32)) return launch(expert_dequant_kernel<OUT, true, P>, grid, NT, 0, 1, s, p);
    return launch(expert_dequant_kernel<OUT, false, P>, grid, NT, 0, 1, s, p);
}

// ---------------------------------------------------------------------------
// weighted combination
// ---------------------------------------------------------------------------
struct CombineParams {
    const void *y, *add;
    const int32_t *slots;
    const float *weights;
    void *out;
    int64_t units;  // of 8 elements, in all tokens
    int upr, k, R, H;
    unsigned int *err;
};

template <typename T> struct Row8 {  // 8 values of a row, 16 bytes
    using Raw = uint4;
    static __device__ __forceinline__ Raw load(const void *p, int64_t i) { return ld_inout(static_cast<const uint16_t *>(p) + i); }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) { Act<T>::unpack(r, f); }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float (&f)[8]) {
        st_v4(static_cast<uint16_t *>(p) + i, pack8<T>(f));
    }
};
template <> struct Row8<float> {
    struct Raw {
        uint4 a, b;
    };
    static __device__ __forceinline__ Raw load(const void *p, int64_t i) {
        const float *f = static_cast<const float *>(p) + i;
        return {ld_inout(f), ld_inout(f + 4)};
    }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float (&f)[8]) {
        float *o = static_cast<float *>(p) + i;
        st_v4(o, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
        st_v4(o + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
    }
};

// Y: type of the rows, O: of `add` and the result.  Sums in fp32, `add` last,
// one rounding.
// G: rows on their way at a time.
template <typename Y, typename O, int G>
__global__ void __launch_bounds__(NT) expert_combine_kernel(const __grid_constant__ CombineParams p) {
    const int64_t at = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (at >= p.units) return;
    const int64_t t = at / p.upr;
    const int col = (int)(at - t * p.upr) * 8;
    pdl_wait();
    pdl_trigger();
    float acc[8] = {};
    const int32_t *const slots = p.slots + t * p.k;
    const float *const weights = p.weights + t * p.k;
    for (int j0 = 0; j0 < p.k; j0 += G) {
        // G rows on their way at a time, added pair by pair in the order of j
        // whatever G is: a token's sum does not depend on the batch it is in.
        int row[G];
        float w[G];
        typename Row8<Y>::Raw raw[G];
#pragma unroll
        for (int j = 0; j < G; ++j) {
            row[j] = j0 + j < p.k ? ld_i32(slots + j0 + j) : -1;
            w[j] = j0 + j < p.k ? ld_f32(weights + j0 + j) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < G; ++j) {
            if (row[j] >= p.R) {
                atomicOr(p.err, (unsigned)DEVERR_BAD_ROW);
                row[j] = -1;
            }
            raw[j] = typename Row8<Y>::Raw{};
            if (row[j] >= 0) raw[j] = Row8<Y>::load(p.y, (int64_t)row[j] * p.H + col);
        }
#pragma unroll
        for (int j = 0; j < G; j += 2) {
            float a[8], b[8];
            Row8<Y>::unpack(raw[j], a);
            Row8<Y>::unpack(raw[j + 1], b);
            const float wa = row[j] < 0 ? 0.f : w[j], wb = row[j + 1] < 0 ? 0.f : w[j + 1];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += fmaf(wb, b[i], wa * a[i]);
        }
    }
    if (p.add) {
        float f[8];
        Row8<O>::unpack(Row8<O>::load(p.add, t * p.H + col), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += f[i];
    }
    Row8<O>::store(p.out, t * p.H + col, acc);
}

template <typename Y, typename O> cudaError_t launch_combine(const CombineParams &p, int sms, cudaStream_t s) {
    const int64_t grid = (p.units + NT - 1) / NT;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    // Eight where the batch is a part of one wave, for latency (one token of 8
    // rows x 2048: 2.4, 2.2, 1.8 us with 2, 4, 8); two in larger ones, whose
    // occupancy keeps more on their way (8192 tokens of 8 x 4096: 102.5, 110.5,
    // 117.7 us).
    if (p.units <= (int64_t)sms * 1024) return launch(expert_combine_kernel<Y, O, 8>, grid, NT, 0, 1, s, p);
    return launch(expert_combine_kernel<Y, O, 2>, grid, NT, 0, 1, s, p);
}

}  // namespace
}  // namespace gnq

extern "C" {

int gnq_expert_quantize(const void *x, int64_t row_stride, int act, const int32_t *offsets, int64_t E,
                        const int32_t *slots, const int32_t *experts, int k, const float *scale, int scale_stride,
                        void *q, void *block_scale, int64_t R, int64_t M, int64_t H, int dtype, void *stream) {
    using namespace gnq;
    if (dtype != GNQ_BF16 && dtype != GNQ_FP16) return GNQ_ERR_DTYPE;
    if (act != ACT_NONE && act != GNQ_SILU && act != GNQ_GELU_TANH) return GNQ_ERR_MODE;
    if (scale_stride != 0 && scale_stride != 1) return GNQ_ERR_MODE;
    if (E < 1 || E > kMaxExperts || R < 0 || R > kMaxM || M < 0 || M > kMaxM) return GNQ_ERR_SHAPE;
    if (H <= 0 || H > kMaxH || H % 64 != 0) return GNQ_ERR_SHAPE;
    if (slots ? k < 1 || k > kMaxTopK : M != R) return GNQ_ERR_SHAPE;
    const int64_t width = act == ACT_NONE ? H : 2 * H;
    if (row_stride < width || row_stride % 8 != 0 || row_stride > (int64_t)1 << 32) return GNQ_ERR_ALIGN;
    if (M == 0 || R == 0) return GNQ_OK;
    if (!x || !offsets || !scale || !q || !block_scale || !slots != !experts) return GNQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(block_scale, 4) || !aligned(offsets, 4) || !aligned(scale, 4) ||
        !aligned(slots, 4) || !aligned(experts, 4))
        return GNQ_ERR_ALIGN;
    const Extent written[] = {extent(q, code_bytes(GNQ_NVFP4, R, H)), extent(block_scale, (R / 128 + E) * 8 * H)};
    const Extent read[] = {{x, M, 2 * row_stride, 2 * width}, extent(offsets, 4 * (E + 1)),
                           extent(scale, 4 * (scale_stride ? E : 1)), extent(slots, 4 * M * k), extent(experts, 4 * M * k)};
    if (outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
    ExpertQuantParams p = {};
    p.x = {offsets, (int)E, (int)R, scale, scale_stride, d->err};
    p.in = static_cast<const uint16_t *>(x);
    p.row_stride = row_stride;
    p.slots = slots;
    p.experts = experts;
    p.k = k;
    p.q = static_cast<uint8_t *>(q);
    p.block_scale = static_cast<uint8_t *>(block_scale);
    p.H = (int)H;
    p.upr = (int)(H / 16);
    p.units = M * p.upr;
    p.M = (int)M;
    const bool v8 = aligned(x, 32) && row_stride % 16 == 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return status_of(dtype == GNQ_BF16 ? launch_expert_quant_act<__nv_bfloat16>(p, act, v8, s)
                                       : launch_expert_quant_act<__half>(p, act, v8, s));
}

int gnq_expert_dequantize(const void *q, const void *block_scale, const int32_t *offsets, int64_t E,
                          const float *scale, int scale_stride, void *out, int64_t R, int64_t K, int out_type,
                          void *stream) {
    using namespace gnq;
    if (out_type < GNQ_BF16 || out_type > GNQ_E4M3) return GNQ_ERR_DTYPE;
    if (scale_stride != 0 && scale_stride != 1) return GNQ_ERR_MODE;
    if (E < 1 || E > kMaxExperts || R < 0 || R > kMaxM || K <= 0 || K > kMaxH || K % 64 != 0) return GNQ_ERR_SHAPE;
    if (R == 0) return GNQ_OK;
    if (!q || !block_scale || !offsets || !out) return GNQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_scale, 4) || !aligned(offsets, 4) || !aligned(scale, 4))
        return GNQ_ERR_ALIGN;
    const int size = out_type == GNQ_E4M3 ? 1 : out_type == GNQ_FP32 ? 4 : 2;
    const Extent written[] = {extent(out, R * K * size)};
    const Extent read[] = {extent(q, code_bytes(GNQ_NVFP4, R, K)), extent(block_scale, (R / 128 + E) * 8 * K),
                           extent(offsets, 4 * (E + 1)), extent(scale, 4 * (scale_stride ? E : 1))};
    if (outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
    ExpertDequantParams p = {};
    p.x = {offsets, (int)E, (int)R, scale, scale_stride, d->err};
    p.q = static_cast<const uint8_t *>(q);
    p.block_scale = static_cast<const uint8_t *>(block_scale);
    p.out = out;
    p.ppr = (int)(K / 32);
    p.Kp4 = (int)(K / 64);
    p.pairs = R * p.ppr;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (out_type) {
        case GNQ_BF16: return status_of(launch_expert_dequant<OUT_BF16>(p, s));
        case GNQ_FP16: return status_of(launch_expert_dequant<OUT_FP16>(p, s));
        case GNQ_FP32: return status_of(launch_expert_dequant<OUT_FP32>(p, s));
        default: return status_of(launch_expert_dequant<OUT_E4M3>(p, s));
    }
}

int gnq_expert_combine(const void *y, const int32_t *slots, const float *weights, const void *add, void *out,
                       int64_t R, int64_t M, int64_t H, int k, int y_type, int out_type, void *stream) {
    using namespace gnq;
    if (y_type < GNQ_BF16 || y_type > GNQ_FP32 || out_type < GNQ_BF16 || out_type > GNQ_FP32) return GNQ_ERR_DTYPE;
    if (y_type != GNQ_FP32 && y_type != out_type) return GNQ_ERR_DTYPE;
    if (R < 0 || R > kMaxM || M < 0 || M > kMaxM || k < 1 || k > kMaxTopK) return GNQ_ERR_SHAPE;
    if (H <= 0 || H > kMaxH || H % 8 != 0) return GNQ_ERR_SHAPE;
    if (M == 0) return GNQ_OK;
    if ((!y && R > 0) || !slots || !weights || !out) return GNQ_ERR_NULL;
    if (!aligned(y, 16) || !aligned(out, 16) || !aligned(add, 16) || !aligned(slots, 4) || !aligned(weights, 4))
        return GNQ_ERR_ALIGN;
    const int64_t size = out_type == GNQ_FP32 ? 4 : 2;
    const Extent written[] = {extent(out, M * H * size)};
    const Extent read[] = {extent(y, R * H * (y_type == GNQ_FP32 ? 4 : 2)), extent(slots, 4 * M * k),
                           extent(weights, 4 * M * k), extent(add == out ? nullptr : add, M * H * size)};
    if (outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
    CombineParams p = {};
    p.y = y;
    p.add = add;
    p.slots = slots;
    p.weights = weights;
    p.out = out;
    p.upr = (int)(H / 8);
    p.units = M * p.upr;
    p.k = k;
    p.R = (int)R;
    p.H = (int)H;
    p.err = d->err;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (y_type == GNQ_BF16) return status_of(launch_combine<__nv_bfloat16, __nv_bfloat16>(p, d->sms, s));
    if (y_type == GNQ_FP16) return status_of(launch_combine<__half, __half>(p, d->sms, s));
    if (out_type == GNQ_BF16) return status_of(launch_combine<float, __nv_bfloat16>(p, d->sms, s));
    if (out_type == GNQ_FP16) return status_of(launch_combine<float, __half>(p, d->sms, s));
    return status_of(launch_combine<float, float>(p, d->sms, s));
}

}  // extern "C"
