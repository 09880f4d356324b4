// Element arithmetic shared by the translation units that quantize rows and
// take them back: the gated activation, the values of NVFP4 blocks.
#pragma once

#include <type_traits>

#include "gnq_device.cuh"

namespace gnq {

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU_TANH = 2 };

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

enum { OUT_BF16 = 0, OUT_FP16 = 1, OUT_FP32 = 2, OUT_E4M3 = 3 };

// Two neighbouring blocks (16 bytes of codes, two scale bytes) to values from
// element `at` of `out`, in whole 32-byte sectors (V8) or 16-byte stores.  A
// block's factor is one IEEE quotient of its scale and the global one; value =
// RN(code * factor), then one rounding to the output type.  EARLY: both quotients
// before a code is unpacked, so that no values wait in registers meanwhile.
template <int OUT, bool V8, bool EARLY = false>
__device__ __forceinline__ void nvfp4_pair_out(void *out, int64_t at, const uint4 &code, uint32_t sf, float g) {
    uint4 e4m3[2];  // E4M3: both blocks leave together
    auto quotient = [&](int h) { return __fdiv_rn(e4m3_value(sf >> (8 * h) & 0xFF), g); };
    [[maybe_unused]] float factor[2];
    if constexpr (EARLY) factor[0] = quotient(0), factor[1] = quotient(1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float f[16];
        e2m1_values8(h ? code.z : code.x, &f[0]);
        e2m1_values8(h ? code.w : code.y, &f[8]);
        mul_arr_s<16>(f, EARLY ? factor[h] : quotient(h));
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
        uint8_t *o = static_cast<uint8_t *>(out) + (at + 16 * h) * N;
        if constexpr (V8 && N > 1) {
#pragma unroll
            for (int c = 0; c < N; c += 2) st_v8(o + 16 * c, w[c], w[c + 1]);
        } else {
#pragma unroll
            for (int c = 0; c < N; ++c) st_v4(o + 16 * c, w[c]);
        }
    }
    if constexpr (OUT == OUT_E4M3) {
        uint8_t *o = static_cast<uint8_t *>(out) + at;
        if constexpr (V8) {
            st_v8(o, e4m3[0], e4m3[1]);
        } else {
            st_v4(o, e4m3[0]);
            st_v4(o + 16, e4m3[1]);
        }
    }
}

}  // namespace gnq
