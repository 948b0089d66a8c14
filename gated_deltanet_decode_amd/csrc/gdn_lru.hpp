// gdn_lru.hpp -- the arithmetic of the gated linear recurrent layer, shared by
// its kernels: the gates of one token, and the composition of the affine maps
// that tokens are over lanes and waves.
#pragma once

#include "gdn_core.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace lru {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kChannels = 64;          // of a tile: 16 lanes of 4
constexpr int kGroups = 4 * kWaves;    // groups of consecutive tokens
constexpr int kSaveStep = 128;         // tokens between the states that a forward pass saves

// Four fp32 values in the activation type; bf16 rounds to nearest even, the
// outputs' only rounding below fp32.
__device__ __forceinline__ uint2 pack(const float (&v)[4], uint16_t) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 lo = {static_cast<__bf16>(v[0]), static_cast<__bf16>(v[1])};
    const bf2 hi = {static_cast<__bf16>(v[2]), static_cast<__bf16>(v[3])};
    return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}
__device__ __forceinline__ float4 pack(const float (&v)[4], float) { return make_float4(v[0], v[1], v[2], v[3]); }

// A is taken as min(A, 0), so that a decay never exceeds 1 (a NaN stays one); in
// units of log2 for the hardware's exp2.
__device__ __forceinline__ float rate_of(float A) { return A > 0.0f ? 0.0f : A; }
__device__ __forceinline__ float rate2(float A) { return rate_of(A) * kLog2e; }

// 1 / (1 + e^-v) with the hardware exp2 and reciprocal (about one ulp each).
// e^-v overflowing gives 0 and underflowing 1, the limits.
__device__ __forceinline__ float sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2e));
}
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }

// sigmoid and its derivative s (1 - s).  The exponential is taken of -|v|, so
// that neither s nor 1 - s is a difference of near values.
__device__ __forceinline__ void sigmoid_slope(float v, float& s, float& slope) {
    const float e = __builtin_amdgcn_exp2f(fabsf(v) * -kLog2e);
    const float inv = __builtin_amdgcn_rcpf(1.0f + e);
    const float less = e * inv;
    s = v >= 0.0f ? inv : less;
    slope = less * inv;
}
// SiLU and its derivative s (1 + v (1 - s)).
__device__ __forceinline__ void silu_slope(float v, float& out, float& slope) {
    float s, d;
    sigmoid_slope(v, s, d);
    out = v * s;
    slope = __builtin_fmaf(v, d, s);
}

// 1 - a^2 from log2 a: 1 - a is a difference of near values for most tokens, so
// below 1/2 of -ln a it comes from a polynomial of degree 4 in log2 a, the
// Chebyshev interpolant of (1 - 2^s)/s over that range (8.4e-8 relative, 2e-7
// evaluated in fp32; m = sqrt(1 - a^2) keeps half of it).
__device__ __forceinline__ float one_minus_square(float l2, float a) {
    float p = __builtin_fmaf(l2, -0.0010852762497961521f, -0.009467288851737976f);
    p = __builtin_fmaf(l2, p, -0.05546589940786362f);
    p = __builtin_fmaf(l2, p, -0.24022309482097626f);
    p = __builtin_fmaf(l2, p, -0.6931471228599548f);
    const float d = l2 > -0.72134752f ? l2 * p : 1.0f - a;   // 1 - a
    return d * (2.0f - d);
}

// One token's map h -> a h + v.
__device__ __forceinline__ void step(float x, float r, float i, float rate2, float& a, float& v) {
    const float l2 = rate2 * sigmoid(r);
    a = __builtin_amdgcn_exp2f(l2);
    v = __builtin_amdgcn_sqrtf(one_minus_square(l2, a)) * (sigmoid(i) * x);
}

// a, m and 1/m, for the gradient.  Where m^2 is below the normal numbers (a gate
// that is shut to the last bit, or a rate of 0) both are taken as 0: what 1/m is
// multiplied with goes to 0 faster than m does.
__device__ __forceinline__ void decay(float l2, float& a, float& m, float& inv) {
    a = __builtin_amdgcn_exp2f(l2);
    const float m2 = one_minus_square(l2, a);
    inv = m2 < 1.17549435e-38f ? 0.0f : __builtin_amdgcn_rsqf(m2);
    m = m2 * inv;
}

__device__ __forceinline__ void compose(float (&h)[4], float4 a, float4 v) {
    h[0] = __builtin_fmaf(a.x, h[0], v.x);
    h[1] = __builtin_fmaf(a.y, h[1], v.y);
    h[2] = __builtin_fmaf(a.z, h[2], v.z);
    h[3] = __builtin_fmaf(a.w, h[3], v.w);
}

// Inclusive scan of maps over a wave's 4 groups of 16 lanes, first group first;
// then each group takes the maps of the groups before it.
__device__ __forceinline__ void scan_forward(int lane, float (&a)[4], float (&v)[4]) {
#pragma unroll
    for (int d = 16; d < 64; d *= 2)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float pa = __shfl_up(a[k], d), pv = __shfl_up(v[k], d);
            if (lane >= d) {
                v[k] = __builtin_fmaf(a[k], pv, v[k]);
                a[k] *= pa;
            }
        }
}
__device__ __forceinline__ void shift_forward(int lane, float (&a)[4], float (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float pa = __shfl_up(a[k], 16), pv = __shfl_up(v[k], 16);
        a[k] = lane >= 16 ? pa : 1.0f;
        v[k] = lane >= 16 ? pv : 0.0f;
    }
}
// The same from the last group back.
__device__ __forceinline__ void scan_reverse(int lane, float (&a)[4], float (&v)[4]) {
#pragma unroll
    for (int d = 16; d < 64; d *= 2)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float pa = __shfl_down(a[k], d), pv = __shfl_down(v[k], d);
            if (lane < 64 - d) {
                v[k] = __builtin_fmaf(a[k], pv, v[k]);
                a[k] *= pa;
            }
        }
}
__device__ __forceinline__ void shift_reverse(int lane, float (&a)[4], float (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float pa = __shfl_down(a[k], 16), pv = __shfl_down(v[k], 16);
        a[k] = lane < 48 ? pa : 1.0f;
        v[k] = lane < 48 ? pv : 0.0f;
    }
}

}  // namespace lru
}  // namespace gdn
