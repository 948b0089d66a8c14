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

// 1 / (1 + e^-v) with the hardware exp2 and reciprocal (about one ulp each).  v log2 e is
// rounded before exp2 and its constant before that, so e^-v is off by 1.25 |v| half steps
// more: some 25 at v = -20, where the gate is 2e-9.  e^-v overflowing gives 0 and
// underflowing 1, the limits.
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

// A value of the wave's lower and of its upper 32 lanes, in all lanes.
__device__ __forceinline__ void both_halves(float x, float& lower, float& upper) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lower = __uint_as_float(r[0]);
    upper = __uint_as_float(r[1]);
}

// Maps of a wave's groups of LPC lanes, of one channel: `a, v` becomes the map of the
// groups before this one (first group first); `wa, wv` is the wave's, in the last
// group's lanes.
template <int LPC>
__device__ __forceinline__ void scan_forward(int lane, float& a, float& v, float& wa, float& wv) {
    if constexpr (LPC == 32) {
        float a0, a1, v0, v1;
        both_halves(a, a0, a1);
        both_halves(v, v0, v1);
        wa = a0 * a1;
        wv = __builtin_fmaf(a1, v0, v1);
        a = lane >= 32 ? a0 : 1.0f;
        v = lane >= 32 ? v0 : 0.0f;
    } else {
#pragma unroll
        for (int d = LPC; d < kWave; d *= 2) {
            const float pa = __shfl_up(a, d), pv = __shfl_up(v, d);
            v = lane >= d ? __builtin_fmaf(a, pv, v) : v;
            a = lane >= d ? a * pa : a;
        }
        wa = a;
        wv = v;
        const float pa = __shfl_up(a, LPC), pv = __shfl_up(v, LPC);
        a = lane >= LPC ? pa : 1.0f;
        v = lane >= LPC ? pv : 0.0f;
    }
}
// The same from the last group back; the wave's is in the first group's lanes.
template <int LPC>
__device__ __forceinline__ void scan_reverse(int lane, float& a, float& v, float& wv) {
    if constexpr (LPC == 32) {
        float a0, a1, v0, v1;
        both_halves(a, a0, a1);
        both_halves(v, v0, v1);
        wv = __builtin_fmaf(a0, v1, v0);
        a = lane >= 32 ? 1.0f : a1;
        v = lane >= 32 ? 0.0f : v1;
    } else {
#pragma unroll
        for (int d = LPC; d < kWave; d *= 2) {
            const float pa = __shfl_down(a, d), pv = __shfl_down(v, d);
            v = lane < kWave - d ? __builtin_fmaf(a, pv, v) : v;
            a = lane < kWave - d ? a * pa : a;
        }
        wv = v;
        const float pa = __shfl_down(a, LPC), pv = __shfl_down(v, LPC);
        a = lane < kWave - LPC ? pa : 1.0f;
        v = lane < kWave - LPC ? pv : 0.0f;
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

// What the waves of a workgroup tell each other, per channel: the MAPS parts of their
// maps, the tiles that each of them has looked up, and what enters each wave's tokens
// (the state and, in a gradient, what is passed back).  The first kWords waves hold a
// channel to a lane where one value is carried over all waves.
template <typename TL, int WAVES, int MAPS>
struct Exchange {
    using Row = float[TL::kChannels];
    alignas(16) Row maps[WAVES][MAPS];
    alignas(16) Row look[WAVES][2];
    alignas(16) Row into[MAPS - 1][WAVES];
    int known[WAVES];   // 2: a state, 1: a map, 0: neither (ahead of the chain's start)
    int tile;
};

__device__ __forceinline__ void put4(float* row, int q, const float (&v)[4]) {
    reinterpret_cast<float4*>(row)[q] = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void get4(const float* row, int q, float (&v)[4]) {
    const float4 f = reinterpret_cast<const float4*>(row)[q];
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}

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

// The value that enters a tile, in the first kWords waves, for the channel
// 64 * wave + lane.  The tile is the dist-th of its chain, whose tiles are `chains`
// apart.  `first` is what enters the first of them, for the same channels: only that
// tile has read it, before it announces what it leaves, so that the last tile may
// replace it in memory.  All waves pass a barrier here.
//
// Each wave looks at one of the tiles before, the nearest to the first wave, until
// one of them shows a state; from there the maps are applied one after the other, as
// those tiles apply theirs themselves.  So the bits do not depend on which tile had
// come how far.
template <typename TL, int WAVES, bool CHAIN, typename EX>
__device__ __forceinline__ float gather(const Chain& ch, EX& ex, int wave, int tile, int chains, int dist, float first) {
    constexpr int E = TL::kWords;
    static_assert(E <= WAVES, "a wave to each 64 channels");
    const int lane = threadIdx.x & 63;
    if (!CHAIN || dist == 0) {
        __syncthreads();
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
                    ex.look[wave][0][e * kWave + lane] = a[e];
                    ex.look[wave][1][e * kWave + lane] = v[e];
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
    float in = 0.0f;
    if (wave < E) {
        const int c = wave * kWave + lane;
        in = ex.look[w][1][c];
        while (--w >= 0)
            in = __builtin_fmaf(ex.look[w][0][c], in, ex.look[w][1][c]);
    }
    return in;
}

}  // namespace lru
}  // namespace gdn
