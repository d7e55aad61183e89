// activation.cuh -- the activation functions of the dense products and their
// slopes, in fp32.  One definition for the forward epilogues and the backward
// kernels.
#pragma once

#include "device.cuh"

namespace moe {

// moe_fn of include/moe.h
enum { FN_NONE = 0, FN_RELU = 1, FN_SILU = 2, FN_GELU = 3, FN_GELU_TANH = 4 };

// The tanh form of GELU is z * sigmoid(2 q), q = sqrt(2/pi) (z + 0.044715 z^3):
// (1 + tanh q) / 2 is the sigmoid of 2 q, so no difference of near-equal
// numbers is formed for negative z.  kGeluTanh2 = 2 sqrt(2/pi).
constexpr float kGeluTanh2 = 1.5957691216057308f;
constexpr float kGeluCubic = 0.044715f;

// Two fp32 operations in one instruction, each rounded as alone.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The normal distribution function Phi(z); `e` gets exp(-z^2 / 2) (its density
// times sqrt(2 pi)).  For x = |z| / sqrt 2, erfc(x) = exp(-x^2) erfcx(x), and
// erfcx(x) is t P(t) with t = 1 / (1 + 0.4 x): P is the polynomial of degree 8
// with the least relative error over 0 <= x <= 14 (reweighted least squares on
// 4000 Chebyshev points): 9e-8, 4e-7 evaluated in fp32.  The relative error
// holds far into the negative tail, where 1 + erf would cancel, and one
// exponential serves the value and the slope.  erfcf took 2.5 times the
// instructions, and a gelu epilogue or gradient was bound by them.
// Two at a time.
__device__ __forceinline__ float2 normal_cdf2(float2 z, float2& e) {
    auto pair = [](float v) { return make_float2(v, v); };
    const float2 d = fma2(pair(0.28284271247461903f), make_float2(fabsf(z.x), fabsf(z.y)), pair(1.0f));
    const float2 t = make_float2(__fdividef(1.0f, d.x), __fdividef(1.0f, d.y));
    float2 p = pair(0.0459682680666447f);
    p = fma2(p, t, pair(-0.1630595624446869f));
    p = fma2(p, t, pair(0.1304987967014313f));
    p = fma2(p, t, pair(0.0354329086840153f));
    p = fma2(p, t, pair(0.1154701560735703f));
    p = fma2(p, t, pair(0.1784794181585312f));
    p = fma2(p, t, pair(0.2056105583906174f));
    p = fma2(p, t, pair(0.2259367406368256f));
    p = fma2(p, t, pair(0.2256629019975662f));
    const float2 h = mul2(mul2(z, z), pair(-0.5f));
    e = make_float2(__expf(h.x), __expf(h.y));
    const float2 tail = mul2(mul2(e, pair(0.5f)), mul2(p, t));
    return make_float2(z.x >= 0.0f ? 1.0f - tail.x : tail.x, z.y >= 0.0f ? 1.0f - tail.y : tail.y);
}

__device__ __forceinline__ float act_relu(float z) { return z <= 0.0f ? 0.0f : z; }  // a NaN stays one
__device__ __forceinline__ float act_gelu_tanh(float z) {
    return __fdividef(z, 1.0f + __expf(-kGeluTanh2 * (z + kGeluCubic * z * z * z)));
}

// fn(z) for an array.  fn is the same for every thread of a launch; the choice
// stands outside the unrolled loop, so that a launch fetches the instructions of
// its own activation only (inside it, the five of them 32 times over cost a small
// gated product 2.5 us of instruction misses).
template <int N>
__device__ __forceinline__ void act_values(int fn, float (&z)[N]) {
    if (fn == FN_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = silu_f32(z[j]);
    } else if (fn == FN_GELU) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            float2 e;
            const float2 v = make_float2(z[j], z[(j + 1) % N]);
            const float2 r = mul2(v, normal_cdf2(v, e));
            z[j] = r.x;
            if (j + 1 < N) z[(j + 1) % N] = r.y;
        }
    } else if (fn == FN_GELU_TANH) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = act_gelu_tanh(z[j]);
    } else if (fn == FN_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = act_relu(z[j]);
    }
}

// Value and slope together (the gated backward needs both).  The exponential
// is taken of -|q|, so neither e^-|q| nor the sum 1 + e^-|q| can overflow.
__device__ __forceinline__ float sigmoid_f32(float q, float& one_minus) {
    const float e = __expf(-fabsf(q));
    const float r = __fdividef(1.0f, 1.0f + e);
    const float small = e * r;  // the sigmoid of -|q|
    one_minus = q >= 0.0f ? small : r;
    return q >= 0.0f ? r : small;
}

// slope[j] = fn'(z[j]) and z[j] = fn(z[j]), N even.
template <int N>
__device__ __forceinline__ void act_slopes(int fn, float (&z)[N], float (&slope)[N]) {
    static_assert(N % 2 == 0, "pairs");
    if (fn == FN_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float m;
            const float p = sigmoid_f32(z[j], m);
            slope[j] = p * (1.0f + z[j] * m);
            z[j] *= p;
        }
    } else if (fn == FN_GELU) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            float2 e;
            const float2 v = make_float2(z[j], z[j + 1]);
            const float2 c = normal_cdf2(v, e);
            const float2 s = fma2(mul2(v, make_float2(0.3989422804014327f, 0.3989422804014327f)), e, c);  // 1/sqrt(2 pi)
            const float2 r = mul2(v, c);
            slope[j] = s.x;
            slope[j + 1] = s.y;
            z[j] = r.x;
            z[j + 1] = r.y;
        }
    } else if (fn == FN_GELU_TANH) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float m;
            const float x = z[j], p = sigmoid_f32(kGeluTanh2 * (x + kGeluCubic * x * x * x), m);
            // m is 0 long before |x| = 64; beyond 1e19 its product with x^2 = infinity would be a NaN
            const float y = fminf(fmaxf(x, -64.0f), 64.0f);
            slope[j] = p * (1.0f + y * m * kGeluTanh2 * (1.0f + 3.0f * kGeluCubic * y * y));
            z[j] = x * p;
        }
    } else if (fn == FN_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            slope[j] = z[j] <= 0.0f ? 0.0f : (z[j] > 0.0f ? 1.0f : z[j]);
            z[j] = act_relu(z[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) slope[j] = 1.0f;
    }
}

// Eight bf16 values in 16 bytes, to and from fp32.
__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

}  // namespace moe
