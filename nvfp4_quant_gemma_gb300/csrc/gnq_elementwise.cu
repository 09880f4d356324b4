// Quantization of a 16-bit matrix, the gated activation of an MLP with the
// quantization of its output, and the way back from NVFP4 to plain values.
// The contracts are in include/gemma_nq.h.
//
//   quantize         q = quant(x)
//   gated activation y = dtype(act(gate) * up), q = quant(y), x = [gate | up]
//   dequantize       out = type(code * (block scale / global scale))
//
// One pass over the data, no reduction beyond a block of 16 or 32 elements,
// at most a few operations per byte: bound by HBM.  A thread owns whole units
// (8 elements, a 16-element block for NVFP4) of a flat index over the matrix,
// neighbouring threads neighbouring units, so rows of any width keep every
// lane busy.  The arithmetic that decides a code is that of the norm kernels
// (epilogue_unit), so equal 16-bit values give equal codes whatever produced
// them.
#include "gemma_nq.h"
#include "gnq_host.cuh"
#include "gnq_kernels.cuh"

namespace gnq {
namespace {

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU_TANH = 2 };

struct QuantParams {
    Params p;            // scale, outputs, M, H, Kp4, write_y (the rest unused)
    int64_t row_stride;  // elements from one row of x to the next
    int64_t units;       // units in the whole matrix
    int upr;             // units per row
};

// act(g) * u in fp32.  silu(g) = g / (1 + e^-g); gelu_tanh(g) =
// g / 2 * (1 + tanh t) = g / (1 + e^-2t), t = sqrt(2/pi) (g + 0.044715 g^3).
// The fast exponential and quotient are good to about 1e-6, far inside the
// one rounding to 16 bits that follows; both forms go to -0 and g as g goes
// to -inf and +inf.
template <int ACT> __device__ __forceinline__ float act_mul(float g, float u) {
    float t;
    if (ACT == ACT_SILU) t = -g;
    else t = g * fmaf(g * g, -0.0713548162726009f, -1.5957691216057308f);
    return __fdividef(g, 1.f + __expf(t)) * u;
}

template <typename T, bool V8, int U>
__device__ __forceinline__ void load_unit(const uint16_t *p, uint4 (&v)[U]) {
    if constexpr (V8 && U == 2) {
        ld_stream_v8(p, v[0], v[1]);
    } else {
#pragma unroll
        for (int c = 0; c < U; ++c) v[c] = ld_stream(p + 8 * c);
    }
}

// V8: 32-byte aligned 16-bit tensors move a unit's block in one access.
template <typename T, int MODE, int ACT, int VPT, bool V8>
__global__ void __launch_bounds__(256) quant_kernel(const __grid_constant__ QuantParams qp) {
    constexpr int U = Unit<MODE>::U, E = Unit<MODE>::E;
    const Params &p = qp.p;
    const int t = threadIdx.x, NT = blockDim.x;
    const int64_t base = (int64_t)blockIdx.x * (NT * VPT);
    const int64_t m0 = base / qp.upr;
    const uint32_t u0 = (uint32_t)(base - m0 * qp.upr);

    int64_t m[VPT];
    int col[VPT];
    bool ok[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const uint32_t i = u0 + v * NT + t;
        const uint32_t r = i / (uint32_t)qp.upr;
        ok[v] = base + v * NT + t < qp.units;
        m[v] = m0 + r;
        col[v] = (int)(i - r * qp.upr) * E;
    }
    pdl_wait();
    pdl_trigger();

    uint4 g[VPT][U], u[VPT][U];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const uint16_t *src = p.x + (ok[v] ? m[v] * qp.row_stride + col[v] : 0);  // out of range: unit 0
        load_unit<T, V8>(src, g[v]);
        if constexpr (ACT != ACT_NONE) load_unit<T, V8>(src + p.H, u[v]);
    }
    const QuantCtx qc = make_quant_ctx<false>(p, MODE, nullptr, t, NT);
    auto finish = [&](auto path) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float y[E];
#pragma unroll
            for (int c = 0; c < U; ++c) {
                Act<T>::unpack(g[v][c], &y[8 * c]);
                if constexpr (ACT != ACT_NONE) {
                    float f[8];
                    Act<T>::unpack(u[v][c], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[8 * c + i] = act_mul<ACT>(y[8 * c + i], f[i]);
                }
            }
            const RowOut o = row_out<MODE>(p, m[v]);
            epilogue_unit<T, MODE, decltype(path)::value, true, V8, true>(
                p, qc, y, o, col[v], sf_col_offset(col[v]), ok[v], t);
        }
    };
    if (MODE == MODE_FP8 && !qc.fd.fast) finish(std::integral_constant<int, FP8_IEEE>{});
    else finish(std::integral_constant<int, FP8_PAIR>{});
}

template <typename T, int MODE, int ACT>
cudaError_t launch_quant(QuantParams &qp, bool v8, cudaStream_t s) {
    constexpr int E = Unit<MODE>::E, VPT = 1, NT = 256;
    qp.upr = qp.p.H / E;
    qp.units = qp.p.M * qp.upr;
    const int64_t grid = (qp.units + NT * VPT - 1) / (NT * VPT);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if constexpr (MODE == MODE_NVFP4) {
        if (v8) return launch(quant_kernel<T, MODE, ACT, VPT, true>, grid, NT, 0, 1, s, qp);
    }
    return launch(quant_kernel<T, MODE, ACT, VPT, false>, grid, NT, 0, 1, s, qp);
}

template <typename T, int ACT>
cudaError_t launch_quant_mode(QuantParams &qp, int mode, bool v8, cudaStream_t s) {
    switch (mode) {
        case MODE_NONE:
            if constexpr (ACT != ACT_NONE) return launch_quant<T, MODE_NONE, ACT>(qp, v8, s);
            return cudaErrorInvalidConfiguration;
        case MODE_FP8: return launch_quant<T, MODE_FP8, ACT>(qp, v8, s);
        case MODE_NVFP4: return launch_quant<T, MODE_NVFP4, ACT>(qp, v8, s);
        default: return launch_quant<T, MODE_MXFP8, ACT>(qp, v8, s);
    }
}

template <typename T>
cudaError_t launch_quant_act(QuantParams &qp, int mode, int act, bool v8, cudaStream_t s) {
    if (act == ACT_SILU) return launch_quant_mode<T, ACT_SILU>(qp, mode, v8, s);
    if (act == ACT_GELU_TANH) return launch_quant_mode<T, ACT_GELU_TANH>(qp, mode, v8, s);
    return launch_quant_mode<T, ACT_NONE>(qp, mode, v8, s);
}

int status_of(cudaError_t e) {
    if (e == cudaSuccess) return GNQ_OK;
    cudaGetLastError();  // reported here; do not leave it for the caller's next check
    return GNQ_ERR_CUDA;
}

int run_quant(const void *x, int64_t row_stride, int act, const float *scale, int mode, int write_y,
              void *q, void *block_scale, void *y, int64_t M, int64_t H, int dtype, void *stream) {
    if (dtype != GNQ_BF16 && dtype != GNQ_FP16) return GNQ_ERR_DTYPE;
    if (M < 0 || M > kMaxM || H <= 0 || H > kMaxH || H % 8 != 0) return GNQ_ERR_SHAPE;
    if (mode == MODE_NVFP4 && H % 64 != 0) return GNQ_ERR_SHAPE;
    if (mode == MODE_MXFP8 && H % 32 != 0) return GNQ_ERR_SHAPE;
    const int64_t width = act == ACT_NONE ? H : 2 * H;
    if (row_stride < width || row_stride % 8 != 0 || row_stride > (int64_t)1 << 32) return GNQ_ERR_ALIGN;
    if (mode == MODE_NONE) write_y = 1;
    if (M == 0) return GNQ_OK;
    if (!x || (write_y && !y) || (mode != MODE_NONE && !q)) return GNQ_ERR_NULL;
    if ((mode == MODE_FP8 || mode == MODE_NVFP4) && !scale) return GNQ_ERR_NULL;
    if ((mode == MODE_NVFP4 || mode == MODE_MXFP8) && !block_scale) return GNQ_ERR_NULL;
    if (write_y && y == x) return GNQ_ERR_ALIAS;
    if (!aligned(x, 16) || (write_y && !aligned(y, 16)) || (mode != MODE_NONE && !aligned(q, 16)) ||
        (scale && !aligned(scale, 4)) || (block_scale && mode >= MODE_NVFP4 && !aligned(block_scale, 4)))
        return GNQ_ERR_ALIGN;
    QuantParams qp = {};
    qp.p.x = static_cast<const uint16_t *>(x);
    qp.p.scale = scale;
    qp.p.q = static_cast<uint8_t *>(q);
    qp.p.block_scale = static_cast<uint8_t *>(block_scale);
    qp.p.y = write_y ? static_cast<uint16_t *>(y) : nullptr;
    qp.p.M = M;
    qp.p.H = (int)H;
    qp.p.Kp4 = (int)(H / 64);
    qp.p.write_y = write_y ? 1 : 0;
    qp.row_stride = row_stride;
    const bool v8 = aligned(x, 32) && row_stride % 16 == 0 && (!write_y || aligned(y, 32));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return status_of(dtype == GNQ_BF16 ? launch_quant_act<__nv_bfloat16>(qp, mode, act, v8, s)
                                       : launch_quant_act<__half>(qp, mode, act, v8, s));
}

// ---------------------------------------------------------------------------
// NVFP4 -> values
// ---------------------------------------------------------------------------
enum { OUT_BF16 = 0, OUT_FP16 = 1, OUT_FP32 = 2, OUT_E4M3 = 3 };

struct DequantParams {
    const uint8_t *q;
    const uint8_t *block_scale;
    const float *scale;  // global scale, or nullptr for 1
    void *out;
    int64_t blocks;      // 16-element blocks in the whole matrix
    int bpr;             // blocks per row
    int Kp4;
};

// The 8 values of a 32-bit word of E2M1 codes (exact in fp16), as fp32.
__device__ __forceinline__ void e2m1_values8(uint32_t w, float *f) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) Act<__half>::unpack2(h[i], f[2 * i], f[2 * i + 1]);
}

// A thread per 16-element block.  The block's factor is one IEEE quotient of
// its scale and the global one; value = RN(code * factor), then one rounding
// to the output type.
template <int OUT, int VPT>
__global__ void __launch_bounds__(256) dequant_kernel(const __grid_constant__ DequantParams p) {
    const int t = threadIdx.x, NT = blockDim.x;
    const int64_t base = (int64_t)blockIdx.x * (NT * VPT);
    const int64_t m0 = base / p.bpr;
    const uint32_t b0 = (uint32_t)(base - m0 * p.bpr);
    pdl_wait();
    pdl_trigger();
    uint2 code[VPT];
    uint32_t sf[VPT];
    bool ok[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const uint32_t i = b0 + v * NT + t;
        const uint32_t r = i / (uint32_t)p.bpr;
        const int b = (int)(i - r * p.bpr);
        const int64_t m = m0 + r, at = base + v * NT + t;
        ok[v] = at < p.blocks;
        code[v] = ok[v] ? __ldg(reinterpret_cast<const uint2 *>(p.q) + at) : make_uint2(0, 0);
        sf[v] = ok[v] ? __ldg(p.block_scale + swizzled_group(m, b & ~3, p.Kp4) + (b & 3)) : 0;
    }
    const float g = p.scale ? __ldg(p.scale) : 1.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        float f[16];
        e2m1_values8(code[v].x, &f[0]);
        e2m1_values8(code[v].y, &f[8]);
        mul_arr_s<16>(f, __fdiv_rn(e4m3_value(sf[v]), g));
        if (!ok[v]) continue;
        const int64_t at = (base + v * NT + t) * 16;
        if constexpr (OUT == OUT_FP32) {
            float *o = static_cast<float *>(p.out) + at;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                st_v4(o + 4 * c, make_uint4(__float_as_uint(f[4 * c]), __float_as_uint(f[4 * c + 1]),
                                            __float_as_uint(f[4 * c + 2]), __float_as_uint(f[4 * c + 3])));
        } else if constexpr (OUT == OUT_E4M3) {
            uint8_t *o = static_cast<uint8_t *>(p.out) + at;
            st_v4(o, make_uint4(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]),
                                e4m3x4(f[8], f[9], f[10], f[11]), e4m3x4(f[12], f[13], f[14], f[15])));
        } else {
            using T = typename std::conditional<OUT == OUT_BF16, __nv_bfloat16, __half>::type;
            uint16_t *o = static_cast<uint16_t *>(p.out) + at;
            st_v4(o, pack8<T>(&f[0]));
            st_v4(o + 8, pack8<T>(&f[8]));
        }
    }
}

template <int OUT> cudaError_t launch_dequant(const DequantParams &p, cudaStream_t s) {
    constexpr int VPT = 1, NT = 256;
    const int64_t grid = (p.blocks + NT * VPT - 1) / (NT * VPT);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch(dequant_kernel<OUT, VPT>, grid, NT, 0, 1, s, p);
}

}  // namespace
}  // namespace gnq

extern "C" {

int gnq_quantize(const void *x, int64_t row_stride, const float *scale, int mode, void *q,
                 void *block_scale, int64_t M, int64_t H, int dtype, void *stream) {
    if (mode < GNQ_FP8 || mode > GNQ_MXFP8) return GNQ_ERR_MODE;
    return gnq::run_quant(x, row_stride, gnq::ACT_NONE, scale, mode, 0, q, block_scale, nullptr, M, H,
                          dtype, stream);
}

int gated_act_quant(const void *x, int64_t row_stride, int act, const float *scale, int mode,
                    int write_y, void *q, void *block_scale, void *y, int64_t M, int64_t H,
                    int dtype, void *stream) {
    if (mode < gnq::MODE_NONE || mode > GNQ_MXFP8) return GNQ_ERR_MODE;
    if (act != GNQ_SILU && act != GNQ_GELU_TANH) return GNQ_ERR_MODE;
    return gnq::run_quant(x, row_stride, act, scale, mode, write_y, q, block_scale, y, M, H, dtype,
                          stream);
}

int gnq_nvfp4_dequantize(const void *q, const void *block_scale, const float *scale, void *out,
                         int64_t M, int64_t K, int out_type, void *stream) {
    if (out_type < GNQ_BF16 || out_type > GNQ_E4M3) return GNQ_ERR_DTYPE;
    if (M < 0 || M > gnq::kMaxM || K <= 0 || K > gnq::kMaxH || K % 64 != 0) return GNQ_ERR_SHAPE;
    if (M == 0) return GNQ_OK;
    if (!q || !block_scale || !out) return GNQ_ERR_NULL;
    if (out == q || out == block_scale) return GNQ_ERR_ALIAS;
    if (!gnq::aligned(q, 16) || !gnq::aligned(out, 16) || !gnq::aligned(block_scale, 4) ||
        (scale && !gnq::aligned(scale, 4)))
        return GNQ_ERR_ALIGN;
    gnq::DequantParams p;
    p.q = static_cast<const uint8_t *>(q);
    p.block_scale = static_cast<const uint8_t *>(block_scale);
    p.scale = scale;
    p.out = out;
    p.blocks = M * (K / 16);
    p.bpr = (int)(K / 16);
    p.Kp4 = (int)(K / 64);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (out_type) {
        case GNQ_BF16: return gnq::status_of(gnq::launch_dequant<gnq::OUT_BF16>(p, s));
        case GNQ_FP16: return gnq::status_of(gnq::launch_dequant<gnq::OUT_FP16>(p, s));
        case GNQ_FP32: return gnq::status_of(gnq::launch_dequant<gnq::OUT_FP32>(p, s));
        default: return gnq::status_of(gnq::launch_dequant<gnq::OUT_E4M3>(p, s));
    }
}

}  // extern "C"
