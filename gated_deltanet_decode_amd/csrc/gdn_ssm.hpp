// gdn_ssm.hpp -- pieces shared by the selective state space kernels: the
// argument block, the activation type's loads and stores, and the per-token
// arithmetic.
//
// Per sequence and token, with C = H*P + 2*G*N channels (x | B | C):
//   u[c] = SiLU(bias[c] + sum_{j<4} w[c][j] * win[c][j])
//   dt_h = softplus(dt[h] + dt_bias[h]);  a_h = exp(dt_h * min(A_h, 0))
//   S_h <- a_h S_h + (dt_h x_h) B_g^T;    y_h = S_h C_g + D_h x_h
//   y   <- y * SiLU(z)                    (with z)
#pragma once

#include "gdn_core.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace ssm {

constexpr float kLog2e = 1.4426950408889634f;

// fp32 -> activation type.  bf16 rounds to nearest even (one conversion
// instruction on gfx950); this is the output's only rounding below fp32.
__device__ __forceinline__ void narrow(float v, uint16_t& out) {
    out = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
__device__ __forceinline__ void narrow(float v, float& out) { out = v; }

// z * sigmoid(z) with the hardware exp2 and reciprocal (about one ulp each, as
// in conv_silu).
__device__ __forceinline__ float silu(float z) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -kLog2e));
}

// u = SiLU(bias + taps, oldest first).
__device__ __forceinline__ float conv_bias_silu(const float w[4], const float win[4], float bias) {
    float acc = bias;
    acc = __builtin_fmaf(w[0], win[0], acc);
    acc = __builtin_fmaf(w[1], win[1], acc);
    acc = __builtin_fmaf(w[2], win[2], acc);
    acc = __builtin_fmaf(w[3], win[3], acc);
    return silu(acc);
}

// dt = softplus(raw + bias), without overflow on either side.
__device__ __forceinline__ float step_size(float raw) { return fmaxf(raw, 0.0f) + log1pf(expf(-fabsf(raw))); }

// log2 of the decay per unit step: A is taken as min(A, 0), so a decay never exceeds 1 (a NaN stays one).
__device__ __forceinline__ float rate2(float A) { return (A > 0.0f ? 0.0f : A) * kLog2e; }

// A state row of N entries over LPR consecutive lanes, NV float4 per lane.
template <int N>
struct Rows {
    static constexpr int LPR = N == 32 ? 8 : 16;
    static constexpr int NV = N / (4 * LPR);
    static constexpr int RPW = kWave / LPR;
    static constexpr int PASS = 4 * RPW;   // rows of a 256-thread workgroup's pass
    __device__ static int key(int j, int r) { return j * 4 * LPR + 4 * r; }
};

// Prompts up to this length take the token walk, which costs about 0.5 us a token
// (2 us where its workgroups no longer fit the chip at once) against 15 to 28 us
// for a chunk of any length.  16 heads of 64 rows: 13.4 against 15.0 us at 16
// tokens, 17.7 against 14.8 at 24; 8 x 64 heads: 26 against 26 us at 8 tokens, 43
// against 26 at 16.
inline int walk_tokens(const SsmGeo& g) { return static_cast<int64_t>(g.B) * g.H * g.P <= 16384 ? 16 : 8; }
size_t chunked_ws_bytes(const SsmGeo& g, int T);
hipError_t launch_ssm_chunked(const SsmGeo& g, const SsmArgs& a, int T, const int32_t* lengths, int32_t* status,
                              void* ws, hipStream_t s);

}  // namespace ssm
}  // namespace gdn
