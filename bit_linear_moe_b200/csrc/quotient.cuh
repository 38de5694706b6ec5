// Quantizer pieces shared by the kernels that write NVFP4 (quantize.cu) and
// the key-value cache (kv_cache.cu): vector loads to fp32, magnitudes, and
// E4M3 / E2M1 codes of IEEE round-to-nearest quotients.
#pragma once

#include "common.cuh"

namespace nvfp4 {

// Eight consecutive elements (16 bytes of bf16, 32 of fp32) -> fp32.
template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
    static NVFP4_DEV void load(const __nv_bfloat16* p, float (&v)[8]) {
        const uint4 a = ldg_v4(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16lo_to_f32(w[i]);
            v[2 * i + 1] = bf16hi_to_f32(w[i]);
        }
    }
};

template <>
struct Vec8<float> {
    static NVFP4_DEV void load(const float* p, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 a = ldg_v4(p + 4 * i);
            v[4 * i] = __uint_as_float(a.x);
            v[4 * i + 1] = __uint_as_float(a.y);
            v[4 * i + 2] = __uint_as_float(a.z);
            v[4 * i + 3] = __uint_as_float(a.w);
        }
    }
};

// Sixteen consecutive elements -> fp32 (two Vec8 loads).
template <typename T>
NVFP4_DEV void load16(const T* p, float (&v)[16]) {
    float a[8], b[8];
    Vec8<T>::load(p, a);
    Vec8<T>::load(p + 8, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = a[j];
        v[8 + j] = b[j];
    }
}

// Largest magnitude (0 where all are NaN).
NVFP4_DEV float amax8(const float (&v)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
    return m;
}

// Approximate reciprocal (relative error below 2^-22 for normal inputs).
NVFP4_DEV float rcp_approx(float a) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}

constexpr float kBracketLo = 0.99999618530273437500f;  // 1 - 2^-18
constexpr float kBracketHi = 1.00000381469726562500f;  // 1 + 2^-18

// E4M3 byte of RN(a / d), a >= 0 (the block scale).  inv ~ 1/d within 2^-22
// (0 when d is 0, subnormal or not finite).  t = RN(a * inv) lies within
// 2^-21 of RN(a / d); E4M3 rounding is monotone, so when t (1 - 2^-18) and
// t (1 + 2^-18) give the same byte (one cvt converts both) it is the byte of
// RN(a / d); otherwise the division decides.
NVFP4_DEV uint32_t e4m3_of_quotient(float a, float d, float inv) {
    if (inv != 0.0f) {
        const float t = __fmul_rn(a, inv);
        uint16_t pr;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
            : "=h"(pr)
            : "f"(__fmul_rn(t, kBracketHi)), "f"(__fmul_rn(t, kBracketLo)));
        if ((pr & 0xFF) == (pr >> 8)) return pr & 0xFF;
    }
    return f32_to_e4m3(__fdiv_rn(a, d));
}

// E2M1 code (low nibble) of RN(v / r).
NVFP4_DEV uint32_t e2m1_of_division(float v, float r) {
    uint16_t pr;
    asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tcvt.u16.u8 %0, c;\n\t}"
        : "=h"(pr)
        : "f"(0.0f), "f"(__fdiv_rn(v, r)));
    return pr & 0xF;
}

// E2M1 codes of v[j] / r (j < 16, two words), each quotient the IEEE-rounded
// division.  inv ~ 1/r within 2^-22 (0: always divide) and p = RN(v * inv)
// put p within 2^-21 |v / r| of RN(v / r).  E2M1 rounding is monotone over
// finite inputs (a NaN gives the same code either way), so where p (1 - 2^-18)
// and p (1 + 2^-18) round to the same code, that is the code of RN(v / r); an
// element whose bracket straddles a rounding boundary is divided.  (With bf16
// inputs that is not rare: an element with the mantissa of the tensor's amax
// makes v / r a boundary value in exact arithmetic, 0.75, 1.75 or 3.5, up to
// the roundings of gs and r.)  A block whose amax / r is not below 15 (an
// infinity, or near overflow) divides every element.
NVFP4_DEV uint2 e2m1x16_of_quotients(const float (&v)[16], float amax, float r, float inv) {
    uint32_t code[2], diff[2];
    if (inv != 0.0f && __fmul_rn(amax, inv) < 15.0f) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float lo[8], hi[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = __fmul_rn(v[8 * w + j], inv);
                lo[j] = __fmul_rn(p, kBracketLo);
                hi[j] = __fmul_rn(p, kBracketHi);
            }
            code[w] = f32x8_to_e2m1(hi);
            diff[w] = f32x8_to_e2m1(lo) ^ code[w];
        }
    } else {
        code[0] = code[1] = 0u;
        diff[0] = diff[1] = 0xFFFFFFFFu;
    }
    if (diff[0] | diff[1]) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (diff[w] & (0xFu << (4 * j)))
                    code[w] = (code[w] & ~(0xFu << (4 * j))) | (e2m1_of_division(v[8 * w + j], r) << (4 * j));
    }
    return make_uint2(code[0], code[1]);
}

// r is a normal float with a normal, finite reciprocal.
NVFP4_DEV bool rcp_safe(float r) { return r >= 1.17549435e-38f && r <= 1.0e37f; }

}  // namespace nvfp4
