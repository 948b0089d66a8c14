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

// Rows of an array from one of them on, for one lane's four channels: a uniform
// base and 32-bit byte offsets (a tile's rows lie within 2^31 bytes).
template <typename Act>
struct Rows {
    const char* base;
    uint32_t pitch, lane;
    __device__ Rows(const Act* p, int64_t row, int64_t elements, int c)
        : base(reinterpret_cast<const char*>(p + row * elements)),
          pitch(static_cast<uint32_t>(elements * sizeof(Act))), lane(static_cast<uint32_t>(c * sizeof(Act))) {}
    __device__ typename Quad<Act>::raw load(int t) const {
        return Quad<Act>::load(reinterpret_cast<const Act*>(base + (static_cast<uint32_t>(t) * pitch + lane)));
    }
    __device__ void store(int t, typename Quad<Act>::raw v) const {
        Quad<Act>::store(reinterpret_cast<Act*>(const_cast<char*>(base) + (static_cast<uint32_t>(t) * pitch + lane)), v);
    }
};

// ------------------------------------------------------------ chains of tiles

constexpr uint32_t kNan = 0x7FC00000u;

// Announcements of a chained kernel's tiles, tile * 64 + channel, and the counter
// that hands the tiles out.
struct Chain {
    unsigned* next;
    uint64_t* maps;
    uint32_t* states;
    __device__ void announce_map(int tile, int lane, float a, float v) const {
        const uint32_t ua = a != a ? kNan : __float_as_uint(a);
        __hip_atomic_store(maps + static_cast<int64_t>(tile) * kChannels + lane,
                           static_cast<uint64_t>(ua) << 32 | __float_as_uint(v), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ void announce_state(int tile, int lane, float h) const {
        __hip_atomic_store(states + static_cast<int64_t>(tile) * kChannels + lane, h != h ? kNan : __float_as_uint(h),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
};

// What the waves of a workgroup tell each other: the maps of their groups, the
// tiles that each of them has looked up, and the tile that was taken.
struct Exchange {
    float4 maps[kWaves][2][16];
    float4 look[kWaves][2][16];
    int known[kWaves];   // 2: a state, 1: a map, 0: neither (ahead of the chain's start)
    int tile;
    __device__ const float* map(int w, int k) const { return reinterpret_cast<const float*>(maps[w][k]); }
};

__device__ __forceinline__ int take_tile(const Chain& ch, Exchange& ex) {
    if (threadIdx.x == 0)
        ex.tile = static_cast<int>(__hip_atomic_fetch_add(ch.next, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    __syncthreads();
    return ex.tile;
}

// The state that enters a tile: h for this lane's four channels, and as the
// result, in the first wave, the one of channel `lane`.  `first` is where the
// state lies that enters the chain.  Only the first wave of the chain's first tile
// reads it, before it announces what it leaves, so that the last tile may replace
// it.  A chain's tiles are `chains` apart.
//
// The wait is bounded all the same: where a word does not come (a second call on
// the same workspace has cleared it, against the rules), the tile goes on with NaN.
constexpr int kPolls = 1 << 22;   // some seconds
template <bool CHAIN>
__device__ __forceinline__ float gather(const Chain& ch, Exchange& ex, int tile, int chains, int seg, const float* first,
                                        float (&h)[4]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane & 15;
    float ga[4] = {1, 1, 1, 1}, gv[4] = {0, 0, 0, 0};   // the maps between the window and the tile
    float la = 1.0f, lv = 0.0f;                           // the same of channel `lane`
    for (int near = seg - 1;; near -= kWaves) {
        const int s = near - wave;
        int known = 0;
        float a = 0.0f, v = 0.0f;
        if (!CHAIN || seg == 0) {
            known = 2;
            if (wave == 0)
                v = *first;
        } else if (s >= 0) {
            const int64_t at = (static_cast<int64_t>(tile) - static_cast<int64_t>(seg - s) * chains) * kChannels + lane;
            for (int poll = 0;; ++poll) {
                const uint32_t st = __hip_atomic_load(ch.states + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                const uint64_t mp = __hip_atomic_load(ch.maps + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                if (__all(st != ~0u)) {
                    known = 2;
                    v = __uint_as_float(st);
                    break;
                }
                if (__all(static_cast<uint32_t>(mp >> 32) != ~0u)) {
                    known = 1;
                    a = __uint_as_float(static_cast<uint32_t>(mp >> 32));
                    v = __uint_as_float(static_cast<uint32_t>(mp));
                    break;
                }
                if (poll == kPolls) {
                    known = 2;
                    v = __uint_as_float(kNan);
                    break;
                }
                __builtin_amdgcn_s_sleep(1);
            }
        }
        reinterpret_cast<float*>(ex.look[wave][0])[lane] = a;
        reinterpret_cast<float*>(ex.look[wave][1])[lane] = v;
        if (lane == 0)
            ex.known[wave] = known;
        __syncthreads();
        int w = 0;
        for (; w < kWaves; ++w) {
            const float4 va = ex.look[w][0][q], vv = ex.look[w][1][q];
            const float ma = reinterpret_cast<const float*>(ex.look[w][0])[lane],
                        mv = reinterpret_cast<const float*>(ex.look[w][1])[lane];
            const bool end = __builtin_amdgcn_readfirstlane(ex.known[w]) == 2;
            const float fa[4] = {va.x, va.y, va.z, va.w}, fv[4] = {vv.x, vv.y, vv.z, vv.w};
            lv = __builtin_fmaf(la, mv, lv);
            la *= ma;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                gv[k] = __builtin_fmaf(ga[k], fv[k], gv[k]);
                ga[k] *= fa[k];
            }
            if (end)
                break;
        }
        if (w < kWaves)
            break;
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        h[k] = gv[k];
    return lv;
}

}  // namespace lru
}  // namespace gdn
