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
#include "gnq_host.cuh"
#include "gnq_launch.cuh"
#include "gnq_tcgen05.cuh"

namespace gnq {
namespace {

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU_TANH = 2 };

struct QuantParams {
    Params p;            // scale, outputs, M, H, Kp4, write_y (the rest unused)
    int64_t row_stride;  // elements from one row of x to the next
    int64_t units;       // units in the whole matrix
    int upr;             // units per row
    int rows_ahead;      // rows from a unit to the one prefetched in its place
};

// act(g) * u of two elements in fp32.  silu(g) = g / (1 + e^-g); gelu_tanh(g)
// = g / 2 * (1 + tanh z) = g / (1 + e^-2z), z = sqrt(2/pi) (g + 0.044715 g^3):
// both g / (1 + 2^t).  The power of two and the reciprocal are the fast ones:
// relative errors of 2^-22 and 2^-23, and the roundings of t count |t| ln 2
// times 1.25 (SiLU) or at most 6 (tanh-GELU) units of 2^-24: 5e-7 for g near 0,
// 1.2e-6 and 4e-6 where act(g) is 1e-4 of g, 6e-5 at the end of the range.  The
// one rounding to 16 bits that follows is 2^-8 (bf16) or 2^-11 (fp16).  Two fp16
// values have an exact product in fp32, so there it is formed first: one rounding
// less, and nearly as many results rounded rightly as with an exact exponential
// and quotient (wrong ones of a SiLU of standard normal gates 6.0e-5, 5.3e-5
// with those, 6.8e-5 with the product last; a Newton step on the reciprocal and
// a two-part exponent give 5.8e-5 and cost a quarter of the time).  In bf16 that
// product could overflow, and rounding hides the difference.  The rest is paired
// fp32 arithmetic: with one operation per instruction a 16384 x 7168 batch into
// FP8 was bound by instruction issue.
// FAR: beyond t = 100 everything is taken 2^100 times smaller until the last
// product, so that 1 + 2^t does not pass 2^126, whose reciprocal is subnormal
// and would be 0 (silu(-88) is -5.3e-37, a normal bf16 value).  Exact scaling:
// for t <= 100 the bits are those of the plain path.  Past t = 226, where act(g)
// is below 2^-218, the result is 0; both forms go to -0 and to g as g goes to
// -inf and +inf.  A warp takes this form for eight gates a lane where one of
// them is that far out (tanh-GELU of 16384 x 7168 into FP8: 96.8 us without such
// a gate, 108.1 where every warp has one; taken always 106.6).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <typename T, int ACT, bool FAR> __device__ __forceinline__ uint64_t act_mul2(uint64_t g, uint64_t u) {
    constexpr float kLog2e = 1.4426950408889634f;
    uint64_t t;  // the exponent of two
    if (ACT == ACT_SILU) {
        t = mul2(g, pk2(-kLog2e, -kLog2e));
    } else {
        constexpr float c1 = -1.5957691216057308f * kLog2e, c3 = -0.0713548162726009f * kLog2e;
        t = mul2(g, fma2(mul2(g, g), pk2(c3, c3), pk2(c1, c1)));
    }
    float t0, t1, d0, d1;
    upk2(t, t0, t1);
    uint64_t one = pk2(1.f, 1.f);
    if constexpr (FAR) {
        const bool f0 = t0 > 100.f, f1 = t1 > 100.f;
        one = pk2(f0 ? 0x1p-100f : 1.f, f1 ? 0x1p-100f : 1.f);
        t0 = f0 ? t0 - 100.f : t0;
        t1 = f1 ? t1 - 100.f : t1;
    }
    upk2(add2(pk2(exp2_fast(t0), exp2_fast(t1)), one), d0, d1);
    const uint64_t r = pk2(rcp_fast(d0), rcp_fast(d1));
    uint64_t y;
    if constexpr (std::is_same<T, __half>::value) y = mul2(mul2(g, u), r);
    else y = mul2(mul2(g, r), u);
    return FAR ? mul2(y, one) : y;
}

// Whether any of 8 packed gates may have t > 100.
template <typename T, int ACT> __device__ __forceinline__ bool gates_far(const uint4 &g) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 *v = reinterpret_cast<const T2 *>(&g);
    const T2 m = __hmin2(__hmin2(v[0], v[1]), __hmin2(v[2], v[3]));
    float lo, hi;
    Act<T>::unpack2(*reinterpret_cast<const uint32_t *>(&m), lo, hi);
    return fminf(lo, hi) < (ACT == ACT_SILU ? -69.f : -9.f);  // t = 99.5, 95.8
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
enum { OUT_BF16 = 0, OUT_FP16 = 1, OUT_FP32 = 2, OUT_E4M3 = 3 };

struct DequantParams {
    const uint8_t *q;
    const uint8_t *block_scale;
    const float *scale;  // global scale, or nullptr for 1
    void *out;
    int64_t pairs;       // pairs of 16-element blocks in the whole matrix
    int ppr;             // pairs per row
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

// A thread takes pairs of neighbouring blocks: 16 bytes of codes, two of
// scales, 32 values out in whole 32-byte sectors (V8) or 16-byte stores.  A
// block's factor is one IEEE quotient of its scale and the global one; value
// = RN(code * factor), then one rounding to the output type.
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
        const int64_t at = (base + v * NT + t) * 32;
        uint4 e4m3[2];  // E4M3: both blocks leave together
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[16];
            e2m1_values8(h ? code[v].z : code[v].x, &f[0]);
            e2m1_values8(h ? code[v].w : code[v].y, &f[8]);
            mul_arr_s<16>(f, __fdiv_rn(e4m3_value(sf[v] >> (8 * h) & 0xFF), g));
            uint4 w[4];
            constexpr int N = OUT == OUT_FP32 ? 4 : OUT == OUT_E4M3 ? 1 : 2;  // 16-byte words of a block
            if constexpr (OUT == OUT_FP32) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    w[c] = make_uint4(__float_as_uint(f[4 * c]), __float_as_uint(f[4 * c + 1]),
                                      __float_as_uint(f[4 * c + 2]), __float_as_uint(f[4 * c + 3]));
            } else if constexpr (OUT == OUT_E4M3) {
                e4m3[h] = make_uint4(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]),
                                     e4m3x4(f[8], f[9], f[10], f[11]), e4m3x4(f[12], f[13], f[14], f[15]));
                continue;
            } else {
                using T = typename std::conditional<OUT == OUT_BF16, __nv_bfloat16, __half>::type;
                w[0] = pack8<T>(&f[0]);
                w[1] = pack8<T>(&f[8]);
            }
            uint8_t *o = static_cast<uint8_t *>(p.out) + (at + 16 * h) * N;
            if constexpr (V8 && N > 1) {
#pragma unroll
                for (int c = 0; c < N; c += 2) st_v8(o + 16 * c, w[c], w[c + 1]);
            } else {
#pragma unroll
                for (int c = 0; c < N; ++c) st_v4(o + 16 * c, w[c]);
            }
        }
        if constexpr (OUT == OUT_E4M3) {
            uint8_t *o = static_cast<uint8_t *>(p.out) + at;
            if constexpr (V8) {
                st_v8(o, e4m3[0], e4m3[1]);
            } else {
                st_v4(o, e4m3[0]);
                st_v4(o + 16, e4m3[1]);
            }
        }
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
