// Sandwich norm: the norm after a block, its gate and residual scale, the
// residual add, the norm before the next block and the quantization for that
// block's first linear, in one pass.  The contract is in include/gemma_nq.h.
//
//   u = x * rsqrt(mean(x^2) + eps) * (1 + w_post)     (u = x without w_post)
//   h = dtype(residual + residual_scale * gate * u)   one rounding
//   y = dtype(h * rsqrt(mean(h^2) + eps) * (1 + w))   from the rounded h
//   q = quant(y)
//
// Per element it reads x, the residual and a gate of its own, writes h and the
// codes, and computes about 14 operations: bound by HBM, like the single norm,
// and by latency below about one row per SM.  One CTA (a cluster for rows
// wider than 1024 units) holds a row in registers from the first load to the
// codes.  The second mean needs every h, and h needs the first mean, so a row
// meets twice; both meetings are a warp shuffle tree and one barrier.
#include "gemma_nq.h"
#include "gnq_host.cuh"
#include "gnq_launch.cuh"

namespace gnq {
namespace {

struct SandwichParams {
    Params p;               // x, residual (read), w, outputs, sizes, quantization
    uint16_t *res_out;      // (M, H), may be p.residual
    const uint16_t *w_post; // (H,) or nullptr: no norm after the block
    const uint16_t *gate;   // nullptr, (H,) or (M, H)
    int64_t gate_stride;    // elements from one row's gate to the next, 0: one for all
    float res_scale;
};

// The chunks of one unit, in one 256-bit access where V8.
enum { LD_STREAM, LD_INOUT, LD_WEIGHT };
template <int KIND, bool V8, int U>
__device__ __forceinline__ void load_unit(const uint16_t *src, uint4 (&d)[U]) {
    if constexpr (V8 && U == 2) {
        if (KIND == LD_STREAM) ld_stream_v8(src, d[0], d[1]);
        else if (KIND == LD_INOUT) ld_inout_v8(src, d[0], d[1]);
        else ld_weight_v8(src, d[0], d[1]);
    } else {
#pragma unroll
        for (int c = 0; c < U; ++c)
            d[c] = KIND == LD_STREAM ? ld_stream(src + 8 * c)
                   : KIND == LD_INOUT ? ld_inout(src + 8 * c) : ld_weight(src + 8 * c);
    }
}

// 1 / sqrt(v) with one Newton step on the fast value, which brings its error
// from two units in the last place to about half a unit: it scales a whole row
// of h, so its error is kept below that of the other steps.  (Values near the
// ends of the range stay as they are: the step would turn 0 and inf into NaN.)
__device__ __forceinline__ float rsqrt_refined(float v) {
    const float y = rsqrtf(v);
    const float e = fmaf(-v * y, y, 1.f);
    return v > 0x1p-100f && v < 0x1p100f ? fmaf(0.5f * y, e, y) : y;
}

// Register budget of an instance.  At four 16-byte chunks per thread and
// operand (256 threads a row for H = 8192), 64 registers keep four rows per
// SM: fp16 16384 x 8192 into NVFP4 123.2 us with 64 (7.2 TB/s), 131 with 72 and
// 80, 158 with 96; into FP8 134.9 (7.0 TB/s), 133.8, 133.5, 170; bf16 into MXFP8
// 134.3, 145.6, 144.7; bf16 8192 x 16384 into FP8, two CTAs a row, 198, 230, 233.
// With a gate bf16 2048 x 5120 into NVFP4 takes 14.4 us with 72, 14.8 with 64.
template <int MODE, int VPT, bool GATED> struct SandwichForm {
    static constexpr int chunks = VPT * Unit<MODE>::U;  // of 16 bytes, per thread and operand
    static constexpr int cap = 65536 / (1024 / VPT) < 255 ? 65536 / (1024 / VPT) : 255;
    static constexpr int maxnreg = chunks == 4 ? (GATED ? 72 : 64) : chunks == 8 ? 128 : cap;
};

// GATED: a gate, per row or per channel, read with x and the residual (where
// it is used, after the first row sum, it cost bf16 16384 x 8192 302 us
// against 179).  V8: 256-bit accesses.
template <typename T, int MODE, int VPT, bool GATED, bool V8>
__global__ void __launch_bounds__(1024 / VPT) __maxnreg__((SandwichForm<MODE, VPT, GATED>::maxnreg))
    sandwich_kernel(const __grid_constant__ SandwichParams sp) {
    constexpr int U = Unit<MODE>::U, E = Unit<MODE>::E;
    constexpr bool ESDIV = MODE == MODE_NVFP4;
    __shared__ __align__(16) float warp_ss[2][32];
    __shared__ float cta_ss[2][8];
    const Params &p = sp.p;
    const uint32_t C = cluster_size();
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int64_t m = C > 1 ? (int64_t)cluster_id_x() : (int64_t)blockIdx.x;
    const int NT = blockDim.x, t = threadIdx.x, nw = NT >> 5;
    const int nunits = p.seg / E;
    const int64_t row = m * (int64_t)p.H;

    int col[VPT], lc[VPT];  // lc: the column a unit loads (clamped in range)
    bool ok[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int u = v * NT + t;
        ok[v] = u < nunits;
        col[v] = (int)rank * p.seg + u * E;
        lc[v] = ok[v] ? col[v] : (int)rank * p.seg;
    }
    if (C > 1) cluster_arrive_relaxed();
    // The first wave's rows into L2 while the preceding grid drains: a hint
    // (the values are read after the wait), as in the single norm.
    if ((int)blockIdx.x < p.pf_ctas) {
        const int64_t seg0 = row + (int64_t)rank * p.seg;
        for (int l = t; l < (p.seg * 2 + 127) >> 7; l += NT) {
            prefetch_l2_line(reinterpret_cast<const char *>(p.x + seg0) + 128 * l, false);
            prefetch_l2_line(reinterpret_cast<const char *>(p.residual + seg0) + 128 * l, false);
        }
    }
    pdl_wait();  // inputs may come from the preceding grid
    pdl_trigger();

    uint4 xv[VPT][U], rv[VPT][U], gv[GATED ? VPT : 1][U];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        load_unit<LD_STREAM, V8>(p.x + row + lc[v], xv[v]);
        load_unit<LD_INOUT, V8>(p.residual + row + lc[v], rv[v]);
        if constexpr (GATED) {
            if (sp.gate_stride) load_unit<LD_STREAM, V8>(sp.gate + m * sp.gate_stride + lc[v], gv[v]);
            else load_unit<LD_WEIGHT, V8>(sp.gate + lc[v], gv[v]);
        }
    }
    // Many rows: the one that takes a place three quarters of a round from
    // now, into L2 with the evict-last priority, so that DRAM stays busy while
    // the resident rows are at their sums (bf16 2048 x 5120 into FP8 15.5 ->
    // 13.8 us, fp16 16384 x 8192 into NVFP4 130.4 -> 123.2; a quarter or a
    // whole round ahead gains less on the large ones, a few per cent more or
    // less on the small).
    if constexpr (VPT > 1) {
        const int64_t ahead = m + p.pf_ctas * 3 / 4;
        if (C == 1 && ahead < p.M) {
            const char *x = reinterpret_cast<const char *>(p.x + ahead * p.H);
            const char *r = reinterpret_cast<const char *>(p.residual + ahead * p.H);
            const char *g = reinterpret_cast<const char *>(sp.gate + ahead * sp.gate_stride);
            for (int l = 128 * t; l < 2 * p.H; l += 128 * NT) {
                prefetch_l2_line(x + l, true);
                prefetch_l2_line(r + l, true);
                if (GATED && sp.gate_stride) prefetch_l2_line(g + l, true);
            }
        }
    }
    // One unit per thread (few rows, bound by latency): the weights come in
    // with the activations.
    constexpr bool W_FIRST = VPT == 1;
    uint4 pv[U], wv[U];
    if constexpr (W_FIRST) {
        if (sp.w_post) load_unit<LD_WEIGHT, V8>(sp.w_post + lc[0], pv);
        load_unit<LD_WEIGHT, V8>(p.w + lc[0], wv);
    }
    const QuantCtx qc = make_quant_ctx<T, !ESDIV>(p, MODE, nullptr, t, NT);

    // The mean of squares of `ss` over the row, as inv = rsqrt(mean + eps).
    auto row_inv = [&](float ss, int k) {
        ss = warp_sum(ss);
        if ((t & 31) == 0) warp_ss[k][t >> 5] = ss;
        __syncthreads();
        float tot = block_total(warp_ss[k], nw, t & 31);
        if (C > 1) {
            if (k == 0 || !sp.w_post) cluster_wait();  // the peers have started
            tot = cluster_total(cta_ss[k], tot, rank, C, t);
        }
        return rsqrt_refined(fmaf(tot, p.inv_h, p.eps));
    };

    // ---- the norm after the block ----
    float a = sp.res_scale;  // times inv with a post-norm
    if (sp.w_post) {
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float sv = 0.f;
#pragma unroll
            for (int c = 0; c < U; ++c) sv = sumsq16x8<T>(xv[v][c], sv);
            ss += ok[v] ? sv : 0.f;
        }
        a *= row_inv(ss, 0);
    }

    // ---- h = dtype(residual + a * gate * (1 + w_post) * x) ----
    uint4 hb[VPT][U];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if constexpr (!W_FIRST) {
            if (sp.w_post) load_unit<LD_WEIGHT, V8>(sp.w_post + lc[v], pv);
        }
        float sv = 0.f;
#pragma unroll
        for (int c = 0; c < U; ++c) {
            float x[8], f[8];
            Act<T>::unpack(xv[v][c], x);
            if (sp.w_post) {
                Act<T>::unpack(pv[c], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], f[i], x[i]);  // x (1 + w_post)
            }
            if constexpr (GATED) {
                Act<T>::unpack(gv[v][c], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= f[i];
            }
            Act<T>::unpack(rv[v][c], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], a, f[i]);
            hb[v][c] = pack8<T>(x);
            sv = sumsq16x8<T>(hb[v][c], sv);
        }
        ss += ok[v] ? sv : 0.f;
        uint16_t *o = sp.res_out + row + col[v];
        if constexpr (V8) {
            st_v8_if(o, hb[v][0], hb[v][1], ok[v]);
        } else {
#pragma unroll
            for (int c = 0; c < U; ++c) st_v4_if(o + 8 * c, hb[v][c], ok[v]);
        }
    }
    const float inv = row_inv(ss, 1);

    // ---- the norm before the next block, then the quantization ----
    const RowOut o = row_out<MODE>(p, m);
    auto finish = [&](auto path) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if constexpr (!W_FIRST) load_unit<LD_WEIGHT, V8>(p.w + lc[v], wv);
            float y[E];
#pragma unroll
            for (int c = 0; c < U; ++c) {
                float w[8];
                Act<T>::unpack(hb[v][c], &y[8 * c]);
                Act<T>::unpack(wv[c], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[8 * c + i] = fmaf(y[8 * c + i], w[i], y[8 * c + i]) * inv;
            }
            epilogue_unit<T, MODE, decltype(path)::value, true, V8, ESDIV>(
                p, qc, y, o, col[v], sf_col_offset(col[v]), ok[v], t);
        }
    };
    if (MODE == MODE_FP8 && !qc.fd.fast) finish(std::integral_constant<int, FP8_IEEE>{});
    else finish(std::integral_constant<int, FP8_PAIR>{});
}

template <typename T, int MODE, int VPT, bool GATED, bool V8>
cudaError_t launch_instance(SandwichParams &sp, int cluster, cudaStream_t s) {
    auto fn = sandwich_kernel<T, MODE, VPT, GATED, V8>;
    const int units = sp.p.seg / Unit<MODE>::E;
    const int threads = ((units + VPT - 1) / VPT + 31) / 32 * 32;
    sp.p.pf_ctas = one_wave_ctas(reinterpret_cast<const void *>(fn), threads);
    return launch(fn, sp.p.M * cluster, threads, 0, cluster, s, sp);
}

template <typename T, int MODE, int VPT>
cudaError_t launch_vpt(SandwichParams &sp, bool v8, int cluster, cudaStream_t s) {
    const bool gated = sp.gate != nullptr;
    if constexpr (MODE == MODE_NVFP4) {
        if (v8)
            return gated ? launch_instance<T, MODE, VPT, true, true>(sp, cluster, s)
                        : launch_instance<T, MODE, VPT, false, true>(sp, cluster, s);
    }
    return gated ? launch_instance<T, MODE, VPT, true, false>(sp, cluster, s)
                : launch_instance<T, MODE, VPT, false, false>(sp, cluster, s);
}

// CTAs per row: a CTA holds at most 1024 units.  0 if the row does not split.
int row_cluster(int64_t H, int mode) {
    const int64_t units = H / (mode == MODE_NVFP4 ? 16 : 8);
    const int gran = mode == MODE_NVFP4 ? 64 : mode == MODE_MXFP8 ? 32 : 8;
    int c = 1;
    while (c < 8 && units / c > 1024 && H % (2 * gran * c) == 0) c *= 2;
    return units <= 1024 * c ? c : 0;
}

// One unit per thread while all rows run at a time so (1024 threads of that
// form per SM; M = 256, H = 4096 without quantization: 2.9 us against 3.7 at
// two units), else about 256 threads per row (512 or more: 16384 x 8192 into
// FP8 309 us); rows wider than 1024 units are split over a cluster, as for the
// single norm.
template <typename T, int MODE>
cudaError_t launch_sandwich(SandwichParams &sp, bool v8, int sms, cudaStream_t s) {
    constexpr int E = Unit<MODE>::E;
    const int cluster = row_cluster(sp.p.H, MODE);
    sp.p.seg = sp.p.H / cluster;
    const int units = sp.p.seg / E;
    int vpt = 1;
    const int per_sm = 1024 / ((units + 31) / 32 * 32);  // rows at one unit per thread
    while (vpt < 4 && sp.p.M * cluster > (int64_t)sms * per_sm && units > 256 * vpt) vpt *= 2;
    switch (vpt) {
        case 1: return launch_vpt<T, MODE, 1>(sp, v8, cluster, s);
        case 2: return launch_vpt<T, MODE, 2>(sp, v8, cluster, s);
        default: return launch_vpt<T, MODE, 4>(sp, v8, cluster, s);
    }
}

template <typename T>
cudaError_t launch_sandwich_mode(SandwichParams &sp, int mode, bool v8, int sms, cudaStream_t s) {
    switch (mode) {
        case MODE_NONE: return launch_sandwich<T, MODE_NONE>(sp, v8, sms, s);
        case MODE_FP8: return launch_sandwich<T, MODE_FP8>(sp, v8, sms, s);
        case MODE_NVFP4: return launch_sandwich<T, MODE_NVFP4>(sp, v8, sms, s);
        default: return launch_sandwich<T, MODE_MXFP8>(sp, v8, sms, s);
    }
}

}  // namespace
}  // namespace gnq

extern "C" int gemma_sandwich_norm_quant(const void *x, void *residual, void *residual_out,
                                         const void *w_post, const void *w, const void *gate,
                                         int64_t gate_stride, float residual_scale, float eps,
                                         const float *scale, int mode, int write_y, void *q,
                                         void *block_scale, void *y, int64_t M, int64_t H, int dtype,
                                         void *stream) {
    using namespace gnq;
    if (dtype != GNQ_BF16 && dtype != GNQ_FP16) return GNQ_ERR_DTYPE;
    if (mode < MODE_NONE || mode > MODE_MXFP8) return GNQ_ERR_MODE;
    if (M < 0 || M > kMaxM || H <= 0 || H > kMaxH || H % 8 != 0) return GNQ_ERR_SHAPE;
    if (mode == MODE_NVFP4 && H % 64 != 0) return GNQ_ERR_SHAPE;
    if (mode == MODE_MXFP8 && H % 32 != 0) return GNQ_ERR_SHAPE;
    if (!row_cluster(H, mode)) return GNQ_ERR_SHAPE;
    if (gate && gate_stride != 0 && (gate_stride < H || gate_stride % 8 != 0)) return GNQ_ERR_ALIGN;
    if (mode == MODE_NONE) write_y = 1;
    if (M == 0) return GNQ_OK;
    if (!residual_out) residual_out = residual;
    if (!x || !residual || !w || (write_y && !y) || (mode != MODE_NONE && !q)) return GNQ_ERR_NULL;
    if ((mode == MODE_FP8 || mode == MODE_NVFP4) && !scale) return GNQ_ERR_NULL;
    if ((mode == MODE_NVFP4 || mode == MODE_MXFP8) && !block_scale) return GNQ_ERR_NULL;
    if (x == residual) return GNQ_ERR_ALIAS;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(w, 16) ||
        (w_post && !aligned(w_post, 16)) || (gate && !aligned(gate, 16)) || (write_y && !aligned(y, 16)) ||
        (mode != MODE_NONE && !aligned(q, 16)) || (scale && !aligned(scale, 4)) ||
        (block_scale && mode >= MODE_NVFP4 && !aligned(block_scale, 4)))
        return GNQ_ERR_ALIGN;
    const int64_t n = 2 * M * H;
    const Extent written[] = {extent(residual_out, n), extent(q, code_bytes(mode, M, H)),
                              extent(block_scale, scale_bytes(mode, M, H)), extent(y, write_y ? n : 0)};
    const Extent read[] = {extent(x, n), extent(w_post, 2 * H), extent(w, 2 * H),
                           gate_stride ? Extent{gate, gate ? M : 0, 2 * gate_stride, 2 * H} : extent(gate, 2 * H),
                           extent(scale, mode == MODE_FP8 || mode == MODE_NVFP4 ? 4 : 0)};
    if (outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    if (residual_out != residual)  // in place is the same element read and written by one thread
        for (const Extent &o : written)
            if (meets(o, extent(residual, n))) return GNQ_ERR_ALIAS;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
    SandwichParams sp = {};
    sp.p.x = static_cast<const uint16_t *>(x);
    sp.p.residual = static_cast<uint16_t *>(residual);
    sp.p.w = static_cast<const uint16_t *>(w);
    sp.p.eps = eps;
    sp.p.inv_h = 1.0f / (float)H;
    sp.p.scale = scale;
    sp.p.q = static_cast<uint8_t *>(q);
    sp.p.block_scale = static_cast<uint8_t *>(block_scale);
    sp.p.y = write_y ? static_cast<uint16_t *>(y) : nullptr;
    sp.p.M = M;
    sp.p.H = (int)H;
    sp.p.Kp4 = (int)(H / 64);
    sp.p.write_y = write_y ? 1 : 0;
    sp.res_out = static_cast<uint16_t *>(residual_out);
    sp.w_post = static_cast<const uint16_t *>(w_post);
    sp.gate = static_cast<const uint16_t *>(gate);
    sp.gate_stride = gate ? gate_stride : 0;
    sp.res_scale = residual_scale;
    const bool v8 = mode == MODE_NVFP4 && aligned(x, 32) && aligned(residual, 32) &&
                    aligned(residual_out, 32) && aligned(w, 32) && (!w_post || aligned(w_post, 32)) &&
                    (!gate || (aligned(gate, 32) && gate_stride % 16 == 0)) &&
                    (!write_y || aligned(y, 32));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == GNQ_BF16
                              ? launch_sandwich_mode<__nv_bfloat16>(sp, mode, v8, d->sms, s)
                              : launch_sandwich_mode<__half>(sp, mode, v8, d->sms, s);
    if (e == cudaSuccess) return GNQ_OK;
    cudaGetLastError();
    return GNQ_ERR_CUDA;
}
