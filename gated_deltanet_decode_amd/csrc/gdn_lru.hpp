// gdn_lru.hpp -- the arithmetic of the gated linear recurrent layer, shared by
// its kernels: the gates of one token, and the composition of the affine maps
// that tokens are over lanes and waves.
#pragma once

#include "gdn_core.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace lru {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSaveStep = 32;         // tokens between the states that a forward pass saves

// A tile of a kernel over prompts: LPC lanes of 4 channels each, 64 / LPC groups of
// N consecutive tokens to a wave, WAVES waves.
template <int LPC, int WAVES, int N>
struct Tile {
    static constexpr int kChannels = 4 * LPC;
    static constexpr int kPerWave = kWave / LPC;
    static constexpr int kTokens = N * kPerWave * WAVES;
    static constexpr int kThreads = WAVES * kWave;
    static constexpr int kWords = kChannels / kWave;   // waves that hold a tile's channels, one to a lane
};

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
// sigmoid and 1 - sigmoid, neither a difference of near values.
__device__ __forceinline__ void sigmoid_both(float v, float& s, float& rest) {
    const float e = __builtin_amdgcn_exp2f(fabsf(v) * -kLog2e);
    const float inv = __builtin_amdgcn_rcpf(1.0f + e);
    const float less = e * inv;
    s = v >= 0.0f ? inv : less;
    rest = v >= 0.0f ? less : inv;
}
// SiLU and its derivative s (1 + v (1 - s)).
__device__ __forceinline__ void silu_slope(float v, float& out, float& slope) {
    float s, d;
    sigmoid_slope(v, s, d);
    out = v * s;
    slope = __builtin_fmaf(v, d, s);
}

// Has a value computed here and not, piece by piece, where it is used: a product that
// is moved behind a barrier keeps both of its factors in registers until then.
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }

// 1 - a^2 from log2 a: 1 - a is a difference of near values for most tokens, so
// below 1/2 of -ln a it comes from a polynomial of degree 4 in log2 a, the
// Chebyshev interpolant of (1 - 2^s)/s over that range (8.4e-8 relative, 2e-7
// evaluated in fp32; m = sqrt(1 - a^2) keeps half of it).
__device__ __forceinline__ float one_minus_square(float l2, float a) {
    float p = __builtin_fmaf(l2, -0.0010852762497961521f, -0.009467288851737976f);
    p = __builtin_fmaf(l2, p, -0.05546589940786362f);
    p = __builtin_fmaf(l2, p, -0.24022309482097626f);
    p = __builtin_fmaf(l2, p, -0.6931471228599548f);
    float near = l2 * p, far = 1.0f - a;
    settle(near);   // a select of two values, not a branch to either's instructions
    settle(far);
    const float d = l2 > -0.72134752f ? near : far;          // 1 - a
    return __builtin_fmaf(d, a, d);                          // (1 - a) (1 + a)
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

// Scan of maps over a wave's groups of LPC lanes.  On return `a, v` is the map of the
// groups before this one (first group first), and lanes of the last group hold the
// wave's in `wa, wv`.
template <int LPC>
__device__ __forceinline__ void scan_forward(int lane, float (&a)[4], float (&v)[4], float (&wa)[4], float (&wv)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int d = LPC; d < kWave; d *= 2) {
            const float pa = __shfl_up(a[k], d), pv = __shfl_up(v[k], d);
            v[k] = lane >= d ? __builtin_fmaf(a[k], pv, v[k]) : v[k];
            a[k] = lane >= d ? a[k] * pa : a[k];
        }
        wa[k] = a[k];
        wv[k] = v[k];
        if constexpr (LPC < kWave) {
            const float pa = __shfl_up(a[k], LPC), pv = __shfl_up(v[k], LPC);
            a[k] = lane >= LPC ? pa : 1.0f;
            v[k] = lane >= LPC ? pv : 0.0f;
        } else {
            a[k] = 1.0f;
            v[k] = 0.0f;
        }
    }
}
// The same from the last group back; the first group's lanes hold the wave's.
template <int LPC>
__device__ __forceinline__ void scan_reverse(int lane, float (&a)[4], float (&v)[4], float (&wv)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int d = LPC; d < kWave; d *= 2) {
            const float pa = __shfl_down(a[k], d), pv = __shfl_down(v[k], d);
            v[k] = lane < kWave - d ? __builtin_fmaf(a[k], pv, v[k]) : v[k];
            a[k] = lane < kWave - d ? a[k] * pa : a[k];
        }
        wv[k] = v[k];
        if constexpr (LPC < kWave) {
            const float pa = __shfl_down(a[k], LPC), pv = __shfl_down(v[k], LPC);
            a[k] = lane < kWave - LPC ? pa : 1.0f;
            v[k] = lane < kWave - LPC ? pv : 0.0f;
        } else {
            a[k] = 1.0f;
            v[k] = 0.0f;
        }
    }
}

// Four values of one row, read or written once per call: past what the caches hold for reuse.
typedef uint32_t nt2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint2 load_row(const uint16_t* p) {
    const nt2 v = __builtin_nontemporal_load(reinterpret_cast<const nt2*>(p));
    return make_uint2(v.x, v.y);
}
__device__ __forceinline__ float4 load_row(const float* p) { return load_stream(p); }
__device__ __forceinline__ void store_row(uint16_t* p, uint2 v) {
    __builtin_nontemporal_store(nt2{v.x, v.y}, reinterpret_cast<nt2*>(p));
}
__device__ __forceinline__ void store_row(float* p, float4 v) { store_stream(p, v); }

// Rows of an array from one of them on, for one lane's four channels: a uniform
// base and 32-bit byte offsets (a tile's rows lie within 2^31 bytes).
template <typename Act>
struct Rows {
    char* base;
    uint32_t pitch, lane;
    __device__ Rows(const Act* p, int64_t row, int64_t elements, int c)
        : base(reinterpret_cast<char*>(const_cast<Act*>(p + row * elements))),
          pitch(static_cast<uint32_t>(elements * sizeof(Act))), lane(static_cast<uint32_t>(c * sizeof(Act))) {}
    // Row t + j; j is the same for the whole wave and costs no vector instruction.
    __device__ Act* at(int t, int j = 0) const {
        return reinterpret_cast<Act*>(base + static_cast<int64_t>(j) * pitch + (static_cast<uint32_t>(t) * pitch + lane));
    }
    __device__ typename Quad<Act>::raw load(int t, int j = 0) const { return load_row(at(t, j)); }
    __device__ void store(int t, int j, typename Quad<Act>::raw v) const { store_row(at(t, j), v); }
};

// ------------------------------------------------------------ chains of tiles

constexpr uint32_t kNan = 0x7FC00000u;
constexpr uint32_t kNone = 0xFFFFFFFFu, kState = 0xFFFFFFFEu;

// Announcements of a chained kernel's tiles, one word per channel at tile *
// channels + channel, and the counter that hands the tiles out.  A word's high half
// is kNone (nothing yet), kState (the low half is the value that leaves the tile) or
// the a of the tile's map (the low half is its v); no a is one of the two, since a
// NaN is made kNan.
struct Chain {
    unsigned* next;
    uint64_t* words;
    __device__ void put(int64_t at, uint32_t high, float low) const {
        __hip_atomic_store(words + at, static_cast<uint64_t>(high) << 32 | __float_as_uint(low), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ void announce_map(int64_t at, float a, float v) const { put(at, a != a ? kNan : __float_as_uint(a), v); }
    __device__ void announce_state(int64_t at, float h) const { put(at, kState, h); }
};

// What the waves of a workgroup tell each other: the MAPS parts of their own maps,
// the tiles that each of them has looked up, and the tile that was taken.
template <typename TL, int WAVES, int MAPS>
struct Exchange {
    float4 maps[WAVES][MAPS][TL::kChannels / 4];
    float4 look[WAVES][2][TL::kChannels / 4];
    int known[WAVES];   // 2: a state, 1: a map, 0: neither (ahead of the chain's start)
    int tile;
    __device__ float map(int w, int part, int c) const { return reinterpret_cast<const float*>(maps[w][part])[c]; }
};

template <typename EX>
__device__ __forceinline__ int take_tile(const Chain& ch, EX& ex) {
    if (threadIdx.x == 0)
        ex.tile = static_cast<int>(__hip_atomic_fetch_add(ch.next, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(ex.tile);
}

// Looks at a word before a tile goes on with NaN: no wait is without an end, also where
// a second call on the same workspace has cleared the word, against the rules.
constexpr int kPolls = 1 << 22;   // some seconds

// The value that enters a tile: `h` for this lane's four channels, and as the result,
// in the first kWords waves, the one of channel 64 * wave + lane.  The tile is the
// dist-th of its chain, whose tiles are `chains` apart.  `first` is what enters the
// first of them, for the same channels: only that tile has read it, before it
// announces what it leaves, so that the last tile may replace it in memory.
//
// Each wave looks at one of the tiles before, the nearest to the first wave, until
// one of them shows a state; from there the maps are applied one after the other, as
// those tiles apply theirs themselves.  So the bits do not depend on which tile had
// come how far.
template <typename TL, int WAVES, bool CHAIN, typename EX>
__device__ __forceinline__ float gather(const Chain& ch, EX& ex, int wave, int tile, int chains, int dist, float first,
                                        float (&h)[4]) {
    constexpr int E = TL::kWords;
    static_assert(E <= WAVES, "a wave to each 64 channels");
    const int lane = threadIdx.x & 63, q = lane % (TL::kChannels / 4);
    if (!CHAIN || dist == 0) {
        if (wave < E)
            reinterpret_cast<float*>(ex.look[0][1])[wave * kWave + lane] = first;
        __syncthreads();
        const float4 v = ex.look[0][1][q];
        h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
        return first;
    }
    const int s = dist - 1 - wave;
    const uint64_t* at = ch.words + (static_cast<int64_t>(tile) - static_cast<int64_t>(wave + 1) * chains) * TL::kChannels + lane;
    int known = 0, w;
    for (int poll = 0;;) {
        if (s >= 0 && known < 2) {
            const int before = known;
            float a[E], v[E];
            do {
                uint64_t word[E];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    word[e] = __hip_atomic_load(at + e * kWave, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                bool none = false, all_state = true, any_state = false;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t high = static_cast<uint32_t>(word[e] >> 32);
                    none |= high == kNone;
                    all_state &= high == kState;
                    any_state |= high == kState;
                    a[e] = high == kState ? 0.0f : __uint_as_float(high);
                    v[e] = __uint_as_float(static_cast<uint32_t>(word[e]));
                }
                // where only some channels show the state yet, the others' is on its way
                if (!__any(none) && (__all(all_state) || !__any(any_state)))
                    known = __any(any_state) ? 2 : 1;
                else
                    __builtin_amdgcn_s_sleep(1);
                if (++poll >= kPolls) {
                    known = 2;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        v[e] = __uint_as_float(kNan);
                }
            } while (known == 0);
            if (known != before)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    reinterpret_cast<float*>(ex.look[wave][0])[e * kWave + lane] = a[e];
                    reinterpret_cast<float*>(ex.look[wave][1])[e * kWave + lane] = v[e];
                }
        }
        if (lane == 0)
            ex.known[wave] = known;
        __syncthreads();
        for (w = 0; w < WAVES && __builtin_amdgcn_readfirstlane(ex.known[w]) != 2; ++w) {
        }
        if (w < WAVES)
            break;
        __syncthreads();
    }
    float mine = wave < E ? reinterpret_cast<const float*>(ex.look[w][1])[wave * kWave + lane] : 0.0f;
    const float4 from = ex.look[w][1][q];
    h[0] = from.x, h[1] = from.y, h[2] = from.z, h[3] = from.w;
    while (--w >= 0) {
        compose(h, ex.look[w][0][q], ex.look[w][1][q]);
        if (wave < E)
            mine = __builtin_fmaf(reinterpret_cast<const float*>(ex.look[w][0])[wave * kWave + lane], mine,
                                  reinterpret_cast<const float*>(ex.look[w][1])[wave * kWave + lane]);
    }
    return mine;
}

}  // namespace lru
}  // namespace gdn
