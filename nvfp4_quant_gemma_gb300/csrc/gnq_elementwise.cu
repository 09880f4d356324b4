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
// them.  Measured on 16384 rows: fp16 8192 wide to NVFP4 54.8 us (6.3 TB/s),
// bf16 to FP8 63.9 us (6.3), to MXFP8 67.0 (6.1), NVFP4 to bf16 50.0 us (6.9), to
// fp32 113.6 (5.4), to E4M3 34.2 (6.1), SiLU of 7168 columns to NVFP4 78.5 us
// (6.8), tanh-GELU to FP8 96.6 (6.1), to MXFP8 96.3 (6.1), not quantized 99.5 (7.1).
#include "gemma_nq.h"
#include "gnq_elementwise.cuh"
#include "gnq_host.cuh"
#include "gnq_launch.cuh"
#include "gnq_tcgen05.cuh"

namespace gnq {
namespace {

struct QuantParams {
    Params p;            // scale, outputs, M, H, Kp4, write_y (the rest unused)
    int64_t row_stride;  // elements from one row of x to the next
    int64_t units;       // units in the whole matrix
    int upr;             // units per row
    int rows_ahead;      // rows from a unit to the one prefetched in its place
};

// V8: 32-byte aligned 16-bit tensors move a unit's block in one access.  Six
// CTAs per SM for four 8-element units a thread (bf16 16384 x 8192 to FP8:
// 68.8, 67.9, 65.7, 64.1 us with the compiler's choice, 4, 5 and 6; NVFP4's
// 16-element units spill there: 57.2 us with its choice, 69 and 77 with 5 and
// 6).
template <typename T, int MODE, int ACT, int VPT, bool V8>
__global__ void __launch_bounds__(256, VPT == 4 && MODE != MODE_NVFP4 ? 6 : 0) quant_kernel(const __grid_constant__ QuantParams qp) {
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
    // The first wave's units into L2 while the preceding grid drains: a hint
    // (the values are read after the wait).
    if ((int)blockIdx.x < p.pf_ctas) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (ok[v]) {
                const uint16_t *src = p.x + m[v] * qp.row_stride + col[v];
                prefetch_l2_line(src, false);
                if (ACT != ACT_NONE) prefetch_l2_line(src + p.H, false);
            }
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
    // The units that take this place three quarters of a round from now, into
    // L2 with the evict-last priority: bytes in flight that need no register
    // (SiLU of 16384 x 7168 to NVFP4 86.1 -> 78.5 us, tanh-GELU to FP8 102.4 ->
    // 96.6, without quantization 105.1 -> 99.5, fp16 16384 x 8192 to NVFP4
    // 57.3 -> 54.9; the plain FP8 and MXFP8 instances spill with it and lose).
    if constexpr (ACT != ACT_NONE || MODE == MODE_NVFP4) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (m[v] + qp.rows_ahead < p.M) {
                const uint16_t *src = p.x + (m[v] + qp.rows_ahead) * qp.row_stride + col[v];
                prefetch_l2_line(src, true);
                if (ACT != ACT_NONE) prefetch_l2_line(src + p.H, true);
            }
    }
    const QuantCtx qc = make_quant_ctx<T, false>(p, MODE, nullptr, t, NT);
    auto finish = [&](auto path) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float y[E];
#pragma unroll
            for (int c = 0; c < U; ++c) Act<T>::unpack(g[v][c], &y[8 * c]);
            if constexpr (ACT != ACT_NONE) {
#pragma unroll
                for (int c = 0; c < U; ++c) {
                    auto activate = [&](auto far) {
                        float f[8];
                        Act<T>::unpack(u[v][c], f);
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            float *o = &y[8 * c + i];
                            upk2(act_mul2<T, ACT, decltype(far)::value>(pk2(o[0], o[1]), pk2(f[i], f[i + 1])), o[0], o[1]);
                        }
                    };
                    if (__any_sync(0xffffffffu, gates_far<T, ACT>(g[v][c]))) activate(std::true_type{});
                    else activate(std::false_type{});
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

// Units per thread.  Several keep enough bytes in flight per SM in a large
// batch (fp16 16384 x 8192 to NVFP4: 66.6, 61.6, 57.6 us with 1, 2, 4); the
// gated form reads twice as much per unit (NVFP4 16384 x 7168: 87, 89, 109 us;
// no quantization 107, 103, 107).  Small batches take one, for latency.
template <int MODE, int ACT>
constexpr int kUnitsPerThread = ACT == ACT_NONE ? 4 : MODE == MODE_NVFP4 ? 1 : 2;

template <typename T, int MODE, int ACT, int VPT>
cudaError_t launch_quant_vpt(QuantParams &qp, bool v8, cudaStream_t s) {
    constexpr int NT = 256;
    const int64_t grid = (qp.units + NT * VPT - 1) / (NT * VPT);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    auto start = [&](auto fn) {
        qp.p.pf_ctas = one_wave_ctas(reinterpret_cast<const void *>(fn), NT);
        qp.rows_ahead = (int)(((int64_t)qp.p.pf_ctas * 3 / 4 * NT * VPT + qp.upr - 1) / qp.upr);
        return launch(fn, grid, NT, 0, 1, s, qp);
    };
    if constexpr (MODE == MODE_NVFP4) {
        if (v8) return start(quant_kernel<T, MODE, ACT, VPT, true>);
    }
    return start(quant_kernel<T, MODE, ACT, VPT, false>);
}

template <typename T, int MODE, int ACT>
cudaError_t launch_quant(QuantParams &qp, bool v8, int sms, cudaStream_t s) {
    constexpr int VPT = kUnitsPerThread<MODE, ACT>;
    qp.upr = qp.p.H / Unit<MODE>::E;
    qp.units = qp.p.M * qp.upr;
    if (qp.units >= (int64_t)sms * 2048 * VPT) return launch_quant_vpt<T, MODE, ACT, VPT>(qp, v8, s);
    return launch_quant_vpt<T, MODE, ACT, 1>(qp, v8, s);
}

template <typename T, int ACT>
cudaError_t launch_quant_mode(QuantParams &qp, int mode, bool v8, int sms, cudaStream_t s) {
    switch (mode) {
        case MODE_NONE:
            if constexpr (ACT != ACT_NONE) return launch_quant<T, MODE_NONE, ACT>(qp, v8, sms, s);
            return cudaErrorInvalidConfiguration;
        case MODE_FP8: return launch_quant<T, MODE_FP8, ACT>(qp, v8, sms, s);
        case MODE_NVFP4: return launch_quant<T, MODE_NVFP4, ACT>(qp, v8, sms, s);
        default: return launch_quant<T, MODE_MXFP8, ACT>(qp, v8, sms, s);
    }
}

template <typename T>
cudaError_t launch_quant_act(QuantParams &qp, int mode, int act, bool v8, int sms, cudaStream_t s) {
    if (act == ACT_SILU) return launch_quant_mode<T, ACT_SILU>(qp, mode, v8, sms, s);
    if (act == ACT_GELU_TANH) return launch_quant_mode<T, ACT_GELU_TANH>(qp, mode, v8, sms, s);
    return launch_quant_mode<T, ACT_NONE>(qp, mode, v8, sms, s);
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
    if (!aligned(x, 16) || (write_y && !aligned(y, 16)) || (mode != MODE_NONE && !aligned(q, 16)) ||
        (scale && !aligned(scale, 4)) || (block_scale && mode >= MODE_NVFP4 && !aligned(block_scale, 4)))
        return GNQ_ERR_ALIGN;
    const Extent written[] = {extent(q, code_bytes(mode, M, H)), extent(block_scale, scale_bytes(mode, M, H)),
                              extent(y, write_y ? 2 * M * H : 0)};
    const Extent read[] = {{x, M, 2 * row_stride, 2 * width},
                           extent(scale, mode == MODE_FP8 || mode == MODE_NVFP4 ? 4 : 0)};
    if (outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    const DevInfo *d = dev_info();
    if (!d) return GNQ_ERR_CUDA;
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
    return status_of(dtype == GNQ_BF16 ? launch_quant_act<__nv_bfloat16>(qp, mode, act, v8, d->sms, s)
                                       : launch_quant_act<__half>(qp, mode, act, v8, d->sms, s));
}

// ---------------------------------------------------------------------------
// NVFP4 -> values
// ---------------------------------------------------------------------------
struct DequantParams {
    const uint8_t *q;
    const uint8_t *block_scale;
    const float *scale;  // global scale, or nullptr for 1
    void *out;
    int64_t pairs;       // pairs of 16-element blocks in the whole matrix
    int ppr;             // pairs per row
    int Kp4;
};

// A thread takes pairs of neighbouring blocks: 16 bytes of codes, two of
// scales, 32 values out (nvfp4_pair_out).
template <int OUT, int VPT, bool V8>
__global__ void __launch_bounds__(256) dequant_kernel(const __grid_constant__ DequantParams p) {
    const int t = threadIdx.x, NT = blockDim.x;
    const int64_t base = (int64_t)blockIdx.x * (NT * VPT);
    const int64_t m0 = base / p.ppr;
    const uint32_t b0 = (uint32_t)(base - m0 * p.ppr);
    pdl_wait();
    pdl_trigger();
    uint4 code[VPT];
    uint32_t sf[VPT];
    bool ok[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const uint32_t i = b0 + v * NT + t;
        const uint32_t r = i / (uint32_t)p.ppr;
        const int b = 2 * (int)(i - r * p.ppr);
        const int64_t m = m0 + r, at = base + v * NT + t;
        ok[v] = at < p.pairs;
        code[v] = make_uint4(0, 0, 0, 0);
        sf[v] = 0;
        if (ok[v]) {
            code[v] = ld_stream(p.q + 16 * at);
            sf[v] = ld_u16(p.block_scale + swizzled_group(m, b & ~3, p.Kp4) + (b & 3));
        }
    }
    const float g = p.scale ? ld_f32(p.scale) : 1.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if (!ok[v]) continue;
        nvfp4_pair_out<OUT, V8>(p.out, (base + v * NT + t) * 32, code[v], sf[v], g);
    }
}

template <int OUT, int VPT> cudaError_t launch_dequant_vpt(const DequantParams &p, cudaStream_t s) {
    constexpr int NT = 256;
    const int64_t grid = (p.pairs + NT * VPT - 1) / (NT * VPT);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if (aligned(p.out, 32)) return launch(dequant_kernel<OUT, VPT, true>, grid, NT, 0, 1, s, p);
    return launch(dequant_kernel<OUT, VPT, false>, grid, NT, 0, 1, s, p);
}

template <int OUT> cudaError_t launch_dequant(const DequantParams &p, int sms, cudaStream_t s) {
    constexpr int VPT = 2;
    if (p.pairs >= (int64_t)sms * 2048 * VPT) return launch_dequant_vpt<OUT, VPT>(p, s);
    return launch_dequant_vpt<OUT, 1>(p, s);
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
    if (!gnq::aligned(q, 16) || !gnq::aligned(out, 16) || !gnq::aligned(block_scale, 4) ||
        (scale && !gnq::aligned(scale, 4)))
        return GNQ_ERR_ALIGN;
    const int size = out_type == GNQ_E4M3 ? 1 : out_type == GNQ_FP32 ? 4 : 2;
    const gnq::Extent written[] = {gnq::extent(out, M * K * size)};
    const gnq::Extent read[] = {gnq::extent(q, gnq::code_bytes(GNQ_NVFP4, M, K)),
                                gnq::extent(block_scale, gnq::scale_bytes(GNQ_NVFP4, M, K)), gnq::extent(scale, 4)};
    if (gnq::outputs_meet(written, read)) return GNQ_ERR_ALIAS;
    const gnq::DevInfo *d = gnq::dev_info();
    if (!d) return GNQ_ERR_CUDA;
    gnq::DequantParams p;
    p.q = static_cast<const uint8_t *>(q);
    p.block_scale = static_cast<const uint8_t *>(block_scale);
    p.scale = scale;
    p.out = out;
    p.pairs = M * (K / 32);
    p.ppr = (int)(K / 32);
    p.Kp4 = (int)(K / 64);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (out_type) {
        case GNQ_BF16: return gnq::status_of(gnq::launch_dequant<gnq::OUT_BF16>(p, d->sms, s));
        case GNQ_FP16: return gnq::status_of(gnq::launch_dequant<gnq::OUT_FP16>(p, d->sms, s));
        case GNQ_FP32: return gnq::status_of(gnq::launch_dequant<gnq::OUT_FP32>(p, d->sms, s));
        default: return gnq::status_of(gnq::launch_dequant<gnq::OUT_E4M3>(p, d->sms, s));
    }
}

}  // extern "C"
