// gdn_ssm_prefill.hip -- prompts of a selective state space layer in chunks of
// 64 tokens on the matrix cores.
//
// Per head and chunk, with c_t the inclusive sum of d_s min(A, 0) log2 e inside
// the chunk, X' = d x and S0 the state that enters,
//   Y  = (M . G) X' + 2^c (C S0^T),   G = C B^T,  M_ij = 2^(c_i - c_j) for j <= i, else 0
//   S1 = 2^c_last S0 + X''^T B,       X'' = 2^(c_last - c) X'
// Only c_i - c_j with i >= j is exponentiated, so nothing overflows however
// strong the decay.
//
//   prep   one workgroup per (sequence, chunk, group): conv and SiLU of the
//          group's B and C channels, and G, once for all heads of the group.
//   steps  one wave per (sequence, chunk, head): d and c.
//   chunk  one wave per (sequence, head, 32 rows of the state, segment of
//          chunks): the state stays transposed in accumulators (entries down,
//          rows across) from chunk to chunk, and since a lane's accumulators
//          of one product are its operand of the next (the fragment order
//          below), no value passes between lanes.
//   A prompt is cut into segments where there are too few (sequence, head)
//   pairs to fill the chip: one pass forms each segment's own state from zero,
//   `join` adds them up (the decay of a head is one number, so states combine
//   by a scaled sum), and a second pass forms the outputs from the states that
//   enter the segments.  The price is reading x twice.
//
// Precision.  fp16 matrix products with fp32 accumulation.  Every operand is
// scaled by a power of two that keeps its largest value in range: B and C per
// token, X' and X'' per state row and chunk, the state per row; scaling is
// exact and undone on the accumulators.  Products that reach the state or fp32
// outputs take each operand as the sum of two fp16 numbers (22 bits) and three
// matrix products, so that the state is as exact as one kept in fp32.  Outputs
// that are rounded to bf16 take one fp16 number (11 bits against bf16's 8).
#include <algorithm>

#include "gdn.h"
#include "gdn_ssm.hpp"

namespace gdn {
namespace ssm {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int Q = 64;   // tokens per chunk

// 32x32x16 fp16 MFMA.  Lane (hi, c) = (lane / 32, lane % 32).  A fragment: row
// c, eight k; B fragment: column c, the same eight k; accumulator v: row
// 8 (v / 4) + 4 hi + v % 4, column c.  Slot e of lane half hi holds
// k = 16 ks + kperm(hi, e), which makes accumulators 8 s .. 8 s + 7 of a tile
// the B fragment of k-step s over its rows.
__device__ __forceinline__ f16v mma(h8 a, h8 b, f16v c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
__host__ __device__ constexpr int kperm(int hi, int e) { return ((e >> 2) << 3) + 4 * hi + (e & 3); }
__device__ __forceinline__ f16v zero16() {
    f16v z;
#pragma unroll
    for (int v = 0; v < 16; ++v)
        z[v] = 0.0f;
    return z;
}
__device__ __forceinline__ h8 ld_frag(const _Float16* m, int frag, int lane) {
    return *reinterpret_cast<const h8*>(m + frag * 512 + lane * 8);
}
__device__ __forceinline__ void st_frag(_Float16* m, int frag, int lane, h8 v) {
    *reinterpret_cast<h8*>(m + frag * 512 + lane * 8) = v;
}
// v = hi + lo in fp16 (22 bits where v is well inside fp16's range).  The value
// is pinned first: a product's rounding to fp16 may be fused into the multiply
// (one rounding), which now and then is not the fp16 that lo is the rest of.
__device__ __forceinline__ void split8(const float (&v)[8], h8& hi, h8& lo) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float x = v[e];
        asm("" : "+v"(x));
        hi[e] = static_cast<_Float16>(x);
        lo[e] = static_cast<_Float16>(x - static_cast<float>(hi[e]));
    }
}
// One fp16 number per value.
__device__ __forceinline__ h8 half8(const float (&v)[8]) {
    h8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = static_cast<_Float16>(v[e]);
    return h;
}
// hi alone, or both parts.
template <bool TWO>
__device__ __forceinline__ void parts8(const float (&v)[8], h8& hi, h8& lo) {
    if constexpr (TWO)
        split8(v, hi, lo);
    else
        lo = hi = half8(v);
}

// The power of two that brings m into [2^TO, 2^(TO + 1)), at most 2^MOST; and the
// exact inverse of such a power.
template <int TO, int MOST>
__device__ __forceinline__ float pow2_to(float m) {
    const int e = static_cast<int>(__float_as_uint(m) >> 23) & 255;
    const int f = 254 + TO - e;
    return __uint_as_float(static_cast<uint32_t>(f < 127 + MOST ? f : 127 + MOST) << 23);
}
// Caps of the scales.  Values below 2^-38 (B, C of a token) or 2^-32 (X' of a
// row) lose relative precision to the absolute 2^-64 of fp16 at that scale; in
// return no product of scales leaves fp32's range.
constexpr int kMostBC = 40, kMostX = 40, kMostS = 100;
__device__ __forceinline__ float inverse_pow2(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// What prep leaves for one (sequence, group, chunk), in fragments of 64 lanes x
// 8 fp16 (1 KB): C (rows: tokens, k: entries), B transposed (rows: entries, k:
// tokens) and G (rows: tokens, k: tokens; the six k-steps at or below the
// diagonal), each as hi and, where wanted, lo; then 2^-s per token of B and C.
template <int N, bool FINE>
struct Shared {
    static constexpr int CF = 2 * (N / 16), BF = 4 * (N / 32), GF = 6;   // fragments of one part
    static constexpr int kC = 0, kCl = CF, kG = FINE ? 2 * CF : CF, kGl = kG + GF, kB = kG + (FINE ? 2 : 1) * GF,
                         kBl = kB + BF, kFrags = kBl + BF;
    static constexpr size_t kHalfs = static_cast<size_t>(kFrags) * 512 + 256;   // scales: 128 floats
    static __device__ int g_frag(int it, int ks) { return it == 0 ? ks : 2 + ks; }
};

template <int N, typename Act, bool FINE>
__global__ __launch_bounds__(512) void ssm_prep_kernel(const Act* __restrict__ x, const Act* __restrict__ tail,
                                                       const Act* __restrict__ w, const Act* __restrict__ bias,
                                                       const int32_t* __restrict__ lengths, int T, int H, int G, int P,
                                                       int C, int nc, _Float16* __restrict__ out) {
    using Sh = Shared<N, FINE>;
    using Qd = Quad<Act>;
    constexpr int PITCH = 2 * N + 1;
    constexpr int SPLIT = 512 / (2 * N) > 0 ? 512 / (2 * N) : 1;   // threads per channel
    constexpr int PER = Q / SPLIT;                                 // tokens per thread
    extern __shared__ __align__(16) float lds[];                   // [Q][PITCH], then [2][Q] scales
    float* sc = lds + Q * PITCH;

    const int chunk = blockIdx.x % nc;
    const int g = (blockIdx.x / nc) % G;
    const int seq = blockIdx.x / nc / G;
    const int len = lengths ? lengths[seq] : T;
    const int t0 = chunk * Q;
    if (len > T || t0 >= len)
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

    {
        const int j = tid % (2 * N);
        const int tb = tid / (2 * N) * PER;
        const int ch = H * P + (j < N ? g * N + j : G * N + g * N + j - N);
        const Act* xs = x + static_cast<size_t>(seq) * T * C + ch;
        float wf[4], tw[4], win[4];
        Qd::to_float(Qd::load(w + static_cast<size_t>(ch) * 4), wf);
        Qd::to_float(Qd::load(tail + (static_cast<size_t>(seq) * C + ch) * 4), tw);
        const float bf = bias ? widen(bias[ch]) : 0.0f;
        win[0] = 0.0f;
#pragma unroll
        for (int k = 1; k < 4; ++k) {   // the three inputs before this thread's first
            const int t = t0 + tb - 4 + k;
            win[k] = t < 0 ? tw[k] : t < len ? widen(xs[static_cast<size_t>(t) * C]) : 0.0f;
        }
#pragma unroll 16
        for (int i = 0; i < PER; ++i) {
            const int t = t0 + tb + i;
            win[0] = win[1];
            win[1] = win[2];
            win[2] = win[3];
            win[3] = t < len ? widen(xs[static_cast<size_t>(t) * C]) : 0.0f;
            lds[(tb + i) * PITCH + j] = t < len ? conv_bias_silu(wf, win, bf) : 0.0f;
        }
    }
    __syncthreads();
    _Float16* o = out + ((static_cast<size_t>(seq) * G + g) * nc + chunk) * Sh::kHalfs;
    float* osc = reinterpret_cast<float*>(o + Sh::kFrags * 512);
    // each token's row of B and of C is brought to [4, 8): |G| <= 64 N stays in range
    for (int r = wave; r < 2 * Q; r += 8) {
        const float* row = lds + (r % Q) * PITCH + (r < Q ? 0 : N);
        float m = 0.0f;
        for (int n = lane; n < N; n += 64)
            m = fmaxf(m, fabsf(row[n]));
#pragma unroll
        for (int k = 32; k >= 1; k >>= 1)
            m = fmaxf(m, __shfl_xor(m, k));
        if (lane == 0) {
            const float s = pow2_to<2, kMostBC>(m);
            sc[r] = s;
            osc[r] = inverse_pow2(s);
        }
    }
    __syncthreads();
    const int hi = lane >> 5, c = lane & 31;
    // row fragment: token row, entries in k order
    auto row_frag = [&](int tok, int off, int ks, float s, h8& fh, h8& fl) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = lds[tok * PITCH + off + 16 * ks + kperm(hi, e)] * s;
        split8(v, fh, fl);
    };
    for (int f = wave; f < Sh::CF; f += 8) {
        const int it = f / (N / 16), ks = f % (N / 16);
        h8 fh, fl;
        row_frag(32 * it + c, N, ks, sc[Q + 32 * it + c], fh, fl);
        st_frag(o, Sh::kC + f, lane, fh);
        if (FINE)
            st_frag(o, Sh::kCl + f, lane, fl);
    }
    for (int f = wave; f < Sh::BF; f += 8) {
        const int nt = f / 4, ks = f % 4;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = 16 * ks + kperm(hi, e);
            v[e] = lds[t * PITCH + 32 * nt + c] * sc[t];
        }
        h8 fh, fl;
        split8(v, fh, fl);
        st_frag(o, Sh::kB + f, lane, fh);
        st_frag(o, Sh::kBl + f, lane, fl);
    }
    // G transposed (rows j, columns i): its accumulators are the rows-i fragments
    if (wave < 3) {
        const int it = wave == 0 ? 0 : 1, jt = wave == 2 ? 1 : 0;
        f16v acc = zero16();
        for (int ks = 0; ks < N / 16; ++ks) {
            h8 bh, bl, ch, cl;
            row_frag(32 * jt + c, 0, ks, sc[32 * jt + c], bh, bl);
            row_frag(32 * it + c, N, ks, sc[Q + 32 * it + c], ch, cl);
            acc = mma(bh, ch, acc);
            if (FINE) {
                acc = mma(bh, cl, acc);
                acc = mma(bl, ch, acc);
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = acc[8 * s + e];
            h8 fh, fl;
            split8(v, fh, fl);
            const int f = Sh::g_frag(it, 2 * jt + s);
            st_frag(o, Sh::kG + f, lane, fh);
            if (FINE)
                st_frag(o, Sh::kGl + f, lane, fl);
        }
    }
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ double wave_scan(double v, int lane) {
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const double u = __shfl_up(v, k);
        v += lane >= k ? u : 0.0;
    }
    return v;
}

// Step sizes and summed decays of a chunk's tokens, one wave per (sequence,
// chunk, head): d, then c as a high and a low fp32 part, 64 each.  c is summed
// in fp64: what matters are differences of it, also where it is large.
__global__ __launch_bounds__(256) void ssm_steps_kernel(const float* __restrict__ dt,
                                                        const float* __restrict__ dt_bias,
                                                        const float* __restrict__ A,
                                                        const int32_t* __restrict__ lengths, int T, int H, int nc,
                                                        int64_t waves, float* __restrict__ steps) {
    const int lane = threadIdx.x & 63;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64;
    if (id >= waves)
        return;
    const int h = static_cast<int>(id % H);
    const int chunk = static_cast<int>(id / H % nc);
    const int seq = static_cast<int>(id / H / nc);
    const int len = lengths ? lengths[seq] : T;
    if (len > T || chunk * Q >= len)
        return;
    const int t = chunk * Q + lane;
    const float d = t < len ? step_size(dt[(static_cast<size_t>(seq) * T + t) * H + h] + (dt_bias ? dt_bias[h] : 0.0f))
                            : 0.0f;
    const double cum = wave_scan(static_cast<double>(d) * static_cast<double>(rate2(A[h])), lane);
    const float high = static_cast<float>(cum);
    float* o = steps + ((static_cast<size_t>(seq) * H + h) * nc + chunk) * (3 * Q);
    o[lane] = d;
    o[Q + lane] = high;
    o[2 * Q + lane] = static_cast<float>(cum - static_cast<double>(high));
}

struct ChunkArgs {
    SsmArgs p;
    const int32_t* lengths;
    const _Float16* shared;   // prep's output
    const float* steps;       // steps' output [B][H][nc][3][64]
    float* seg_state;         // [B][H][segments][P][N]
    float* seg_decay;         // [B][H][segments] log2 of the segment's decay
    int T, B, H, G, P, C, nc, segs, chunks_per_seg, by_xcd;
};

// A wave's tile of 64 tokens x 32 channels of x in LDS, and later of y in fp32,
// 32 tokens at a time.  The pitch (40 elements) puts the two lane halves' rows,
// four apart, into different banks.
template <typename Act>
struct Tile {
    static constexpr int kUnit = 16 / sizeof(Act);     // channels per 16 bytes
    static constexpr int kPerRow = 32 / kUnit;         // 16-byte units per row; also units per lane of 64 rows
    static constexpr int kRowStep = 64 / kPerRow;      // rows between a lane's units
    static constexpr int kPitch = 40;
    static constexpr int kBytes = Q * kPitch * sizeof(Act);
    static_assert(kBytes >= 32 * kPitch * 4, "half a tile of fp32 outputs fits");
};
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// Nothing moves across, and values loaded before are loaded again after: the
// compiler would otherwise hoist whole phases' loads, or keep their values, and
// run out of registers.
__device__ __forceinline__ void phase() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The value is computed by here (the compiler may otherwise sink what computes
// it past a phase and keep all its operands instead).
__device__ __forceinline__ void pin(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void pin(h8& v) { asm volatile("" : "+v"(v)); }

// Orders a wave's LDS accesses: what one lane wrote is there for the others.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// One workgroup per (sequence, head, segment), one wave per 32 rows of the
// state.  With every row's operands in one scale, a chunk's outputs are a single
// product over 64 + N terms, Y = [M . G | 2^c C] [X'; S0^T]; its left factor is
// the head's, so each wave builds a part of it and leaves it in LDS for all (the
// one thing that the waves share; all else is a wave's own).  x comes a chunk
// ahead, in 16-byte loads through a tile in LDS, and y leaves the same way.
// OUT: form the outputs.  EXACT: the state's products in two fp16 parts.  With
// segments, OUT without EXACT serves bf16 outputs (the state comes from join).
template <int N, typename Act, bool FINE, bool OUT, bool EXACT>
__global__ __launch_bounds__(256, N > 128 || FINE ? 1 : 2) void ssm_chunk_kernel(ChunkArgs a) {
    using Sh = Shared<N, FINE>;
    using Qd = Quad<Act>;
    using Tl = Tile<Act>;
    constexpr int NT = N / 32, KS = N / 16;
    constexpr int AF = Sh::GF + Sh::CF;   // fragments of the left factor (of one part)
    constexpr int NF = OUT ? 6 : 2;
    extern __shared__ __align__(16) char pool[];   // [waves][tile, factors], then the left factor

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hi = lane >> 5, c = lane & 31;
    const int waves = a.P / 32;
    // workgroup -> (sequence, segment, group), head of the group: all heads that
    // read the same fragments on one XCD (workgroups go to the eight in turn)
    const int rep = a.H / a.G;
    int set, member;
    if (a.by_xcd) {
        set = blockIdx.x / 8 / rep * 8 + blockIdx.x % 8;
        member = blockIdx.x / 8 % rep;
    } else {
        set = blockIdx.x / rep;
        member = blockIdx.x % rep;
    }
    if (set >= a.B * a.segs * a.G)
        return;
    const int g = set % a.G;
    const int h = g * rep + member;
    const int seg = set / a.G % a.segs;
    const int seq = set / a.G / a.segs;
    const int len = a.lengths ? a.lengths[seq] : a.T;
    if (len < 1 || len > a.T)
        return;
    const int last = (len + Q - 1) / Q;
    const int ch0 = seg * a.chunks_per_seg;
    const int ch1 = ch0 + a.chunks_per_seg < last ? ch0 + a.chunks_per_seg : last;
    if (ch0 >= ch1)
        return;
    const bool split = a.segs > 1;

    constexpr int kWaveBytes = Tl::kBytes + NF * Q * 4;
    Act* xt = reinterpret_cast<Act*>(pool + wave * kWaveBytes);
    float* yt = reinterpret_cast<float*>(pool + wave * kWaveBytes);
    float* fF = reinterpret_cast<float*>(pool + wave * kWaveBytes + Tl::kBytes);   // d * 2^-s_B
    float* fW = fF + Q;       // 2^(c_last - c)
    float* fS = fF + 2 * Q;   // 2^-s_C
    float* fK = fF + 3 * Q;   // D * 2^s_C
    float* fH = fF + 4 * Q;   // c, high and low part
    float* fL = fF + 5 * Q;
    _Float16* L = reinterpret_cast<_Float16*>(pool + waves * kWaveBytes);

    const int col0 = h * a.P + wave * 32;
    const int chan = col0 + c;   // this lane's state row, as an x channel
    const Act* xs = static_cast<const Act*>(a.p.x) + static_cast<size_t>(seq) * a.T * a.C;
    float wf[4];
    Qd::to_float(Qd::load(static_cast<const Act*>(a.p.w) + static_cast<size_t>(chan) * 4), wf);
    const float bf = a.p.bias ? widen(static_cast<const Act*>(a.p.bias)[chan]) : 0.0f;
    const float skip = a.p.D ? a.p.D[h] : 0.0f;
    const size_t head = static_cast<size_t>(seq) * a.H + h;
    const float* steps = a.steps + head * a.nc * (3 * Q);
    const _Float16* shared0 = a.shared + (static_cast<size_t>(seq) * a.G + g) * a.nc * Sh::kHalfs;

    // unit k of this lane: row urow + k * kRowStep, channels ucol ..
    const int urow = lane / Tl::kPerRow, ucol = lane % Tl::kPerRow * Tl::kUnit;
    u4 xu[Tl::kPerRow];
    float st_d, st_h, st_l, st_b, st_c = 1.0f;   // the chunk's step, c, scales (one token per lane)
    auto load_chunk = [&](int ch) {
        // rows behind the sequence's end are the last row again; their step size is 0
#pragma unroll
        for (int k = 0; k < Tl::kPerRow; ++k) {
            const int t = min(ch * Q + urow + k * Tl::kRowStep, len - 1);
            xu[k] = *reinterpret_cast<const u4*>(xs + static_cast<size_t>(t) * a.C + col0 + ucol);
        }
        const float* st = steps + static_cast<size_t>(ch) * (3 * Q);
        const float* sc = reinterpret_cast<const float*>(shared0 + ch * Sh::kHalfs + Sh::kFrags * 512);
        st_d = st[lane];
        st_h = st[Q + lane];
        st_l = st[2 * Q + lane];
        st_b = sc[lane];
        if (OUT)
            st_c = sc[Q + lane];
    };

    // the three inputs before the segment
    Act before[3];
    {
        const typename Qd::raw tr = Qd::load(static_cast<const Act*>(a.p.tail_in) +
                                             (static_cast<size_t>(seq) * a.C + chan) * 4);
#pragma unroll
        for (int k = 0; k < 3; ++k)
            before[k] = ch0 == 0 ? Qd::elem(tr, k + 1) : xs[static_cast<size_t>(ch0 * Q - 3 + k) * a.C + chan];
    }

    // the state, transposed: S[nt][v] is entry 32 nt + 8 (v / 4) + 4 hi + v % 4 of this lane's row, times `unit`
    f16v S[NT];
    float unit = 1.0f;
    const size_t row_off = static_cast<size_t>(wave * 32 + c) * N + 4 * hi;
    float* seg_row = a.seg_state + (head * a.segs + seg) * a.P * N + row_off;
    float* state_row = a.p.state + head * a.P * N + row_off;
    if (OUT) {
        const float* from = split ? seg_row : state_row;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 v = *reinterpret_cast<const float4*>(from + 32 * nt + 8 * q);
                S[nt][4 * q] = v.x;
                S[nt][4 * q + 1] = v.y;
                S[nt][4 * q + 2] = v.z;
                S[nt][4 * q + 3] = v.w;
            }
    } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            S[nt] = zero16();
    }
    // One dword of each 128-byte line of the chunk's fragments, so that they are in
    // this XCD's L2 when their chunk comes: all heads of a group ask for them at
    // about the same time, and all would wait for the memory behind it.
    constexpr int kFrom = OUT ? 0 : Sh::kB, kTo = EXACT ? Sh::kFrags : Sh::kBl;
    constexpr int kLines = (kTo - kFrom) * 8;
    constexpr int kTouch = (kLines + 63) / 64;
    uint32_t touched[kTouch];
    auto touch = [&](int ch) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(shared0 + ch * Sh::kHalfs + kFrom * 512);
#pragma unroll
        for (int k = 0; k < kTouch; ++k)
            if ((k * waves + wave) * 64 < kLines)   // kLines is a multiple of 32
                touched[k] = p[min((k * waves + wave) * 64 + lane, kLines - 1) * 32];
    };
#pragma unroll
    for (int k = 0; k < kTouch; ++k)
        touched[k] = 0;
    load_chunk(ch0);

    // B's fragments of a k-step, loaded ahead of their products
    constexpr int kAhead = OUT ? 1 : 2, kRing = kAhead + 1;
    h8 bh_[kRing][NT], bl_[kRing][NT];
    auto load_b = [&](const _Float16* sh, int ks) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            bh_[ks % kRing][nt] = ld_frag(sh, Sh::kB + nt * 4 + ks, lane);
            if (EXACT)
                bl_[ks % kRing][nt] = ld_frag(sh, Sh::kBl + nt * 4 + ks, lane);
        }
    };

    double seg_sum = 0.0;
    for (int ch = ch0; ch < ch1; ++ch) {
        const int t0 = ch * Q;
        const _Float16* sh = shared0 + ch * Sh::kHalfs;
#pragma unroll
        for (int k = 0; k < kTouch; ++k)
            asm volatile("" ::"v"(touched[k]));
        touch(min(ch + 1, ch1 - 1));
        // x into the tile, the chunk's factors beside it
#pragma unroll
        for (int k = 0; k < Tl::kPerRow; ++k)
            *reinterpret_cast<u4*>(xt + (urow + k * Tl::kRowStep) * Tl::kPitch + ucol) = xu[k];
        const float th = __shfl(st_h, 63), tl = __shfl(st_l, 63);
        const float total = th + tl;
        seg_sum += static_cast<double>(th) + static_cast<double>(tl);
        fF[lane] = st_d * st_b;
        fW[lane] = __builtin_amdgcn_exp2f((th - st_h) + (tl - st_l));
        if (OUT) {
            fS[lane] = st_c;
            fK[lane] = skip * inverse_pow2(st_c);
            fH[lane] = st_h;
            fL[lane] = st_l;
        }
        wave_sync();
        if (!OUT) {
            load_b(sh, 0);
            load_b(sh, 1);
        }
        phase();

        // conv; the largest of X' and of X'' in this row
        float xc[32];
        float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float raw[7];
#pragma unroll
            for (int e = 0; e < 7; ++e) {
                const int row = 8 * r + e - 3;
                if (r == 0 && e < 3) {
                    const Act v = xt[(row + 4) * Tl::kPitch + c];   // in the tile for the upper half
                    raw[e] = widen(hi ? v : before[e]);
                } else {
                    raw[e] = widen(xt[(row + 4 * hi) * Tl::kPitch + c]);
                }
            }
            const float4 F = *reinterpret_cast<const float4*>(fF + 8 * r + 4 * hi);
            const float4 W = *reinterpret_cast<const float4*>(fW + 8 * r + 4 * hi);
            const float ff[4] = {F.x, F.y, F.z, F.w}, ww[4] = {W.x, W.y, W.z, W.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float win[4] = {raw[i], raw[i + 1], raw[i + 2], raw[i + 3]};
                const float v = conv_bias_silu(wf, win, bf);
                xc[4 * r + i] = v;
                const float xp = v * ff[i];
                m1 = fmaxf(m1, fabsf(xp));
                m2 = fmaxf(m2, fabsf(xp * ww[i]));
                pin(xc[4 * r + i]);
            }
            pin(m1);
            pin(m2);
            if (r % 2)
                phase();
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)   // the tile's last three rows
            before[k] = xt[(Q - 3 + k) * Tl::kPitch + c];
        load_chunk(min(ch + 1, ch1 - 1));
        m1 = fmaxf(m1, __shfl_xor(m1, 32));
        m2 = fmaxf(m2, __shfl_xor(m2, 32));
        // the row's largest state entry
        float ms = 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                ms = fmaxf(ms, fabsf(S[nt][v]));
        ms = fmaxf(ms, __shfl_xor(ms, 32));
        // a common unit of the state's part and the chunk's is kept small enough for both
        const float state_max = ms * inverse_pow2(unit);
        const float room = fminf(pow2_to<60, kMostS>(state_max), unit * 0x1p60f);
        const float s2 = fminf(pow2_to<8, kMostS>(m2), room);   // the unit of S1
        const float sx = pow2_to<8, kMostX>(fmaxf(m1, state_max));

        // X'' and X' as fragments; Y starts from D x
        h8 wh[4], wl[4], xh[4], xl[4];
        f16v Y[2];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            float v[8], u[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 F = *reinterpret_cast<const float4*>(fF + 16 * ks + 8 * q + 4 * hi);
                const float4 W = *reinterpret_cast<const float4*>(fW + 16 * ks + 8 * q + 4 * hi);
                const float ff[4] = {F.x, F.y, F.z, F.w}, ww[4] = {W.x, W.y, W.z, W.w};
                float kk[4] = {};
                if (OUT) {
                    const float4 K = *reinterpret_cast<const float4*>(fK + 16 * ks + 8 * q + 4 * hi);
                    kk[0] = K.x, kk[1] = K.y, kk[2] = K.z, kk[3] = K.w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = xc[8 * ks + 4 * q + i];
                    const float xp = x * ff[i];
                    v[4 * q + i] = xp * (ww[i] * s2);
                    if (OUT) {
                        u[4 * q + i] = xp * sx;
                        Y[ks / 2][8 * (ks % 2) + 4 * q + i] = (x * sx) * kk[i];
                    }
                }
            }
            parts8<EXACT>(v, wh[ks], wl[ks]);
            pin(wh[ks]);
            if (EXACT)
                pin(wl[ks]);
            if (OUT) {
                parts8<FINE>(u, xh[ks], xl[ks]);
                pin(xh[ks]);
                if (FINE)
                    pin(xl[ks]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float y = Y[ks / 2][8 * (ks % 2) + e];
                    pin(y);
                    Y[ks / 2][8 * (ks % 2) + e] = y;
                }
            }
            phase();
        }

        if (OUT) {
            // this wave's part of the left factor: M . G, then 2^c C; four fragments in flight
            for (int f0 = wave; f0 < AF; f0 += 4 * waves) {
                h8 fh[4], fl[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int f = min(f0 + k * waves, AF - 1);
                    const int at = f < Sh::GF ? Sh::kG + f : Sh::kC + f - Sh::GF;
                    fh[k] = ld_frag(sh, at, lane);
                    if (FINE)
                        fl[k] = ld_frag(sh, f < Sh::GF ? Sh::kGl + f : Sh::kCl + f - Sh::GF, lane);
                }
                phase();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int f = f0 + k * waves;
                    if (f >= AF)
                        break;
                    h8 mh, ml;
                    if (f < Sh::GF) {
                        const int it = f >= 2, ks = it ? f - 2 : f;
                        const float ci = fH[32 * it + c];
                        const float li = FINE ? fL[32 * it + c] : 0.0f;
                        float m[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int j = 16 * ks + kperm(hi, e);
                            float arg = ci - fH[j];
                            float gv = static_cast<float>(fh[k][e]);
                            if (FINE) {
                                arg += li - fL[j];
                                gv += static_cast<float>(fl[k][e]);
                            }
                            m[e] = j <= 32 * it + c ? gv * __builtin_amdgcn_exp2f(arg) : 0.0f;
                        }
                        parts8<FINE>(m, mh, ml);
                    } else {
                        const int row = f - Sh::GF < KS ? c : 32 + c;
                        const float e2 = __builtin_amdgcn_exp2f(fH[row] + fL[row]);
                        if (FINE) {
                            float m[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                m[e] = (static_cast<float>(fh[k][e]) + static_cast<float>(fl[k][e])) * e2;
                            split8(m, mh, ml);
                        } else {
                            mh = fh[k] * static_cast<_Float16>(e2);
                        }
                    }
                    st_frag(L, f, lane, mh);
                    if (FINE)
                        st_frag(L, AF + f, lane, ml);
                }
            }
            phase();
            __syncthreads();
        }
        // B's fragments and z come while the outputs are formed
        const bool update = !OUT || !split || ch + 1 < ch1;
        if (OUT && update)
            load_b(sh, 0);
        if (OUT) {
            const float sscale = sx * inverse_pow2(unit);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = S[ks / 2][8 * (ks % 2) + e] * sscale;
                h8 bh, bl;
                parts8<FINE>(v, bh, bl);
#pragma unroll
                for (int it = 0; it < 2; ++it) {
                    const h8 ah = ld_frag(L, Sh::GF + it * KS + ks, lane);
                    Y[it] = mma(ah, bh, Y[it]);
                    if (FINE) {
                        Y[it] = mma(ah, bl, Y[it]);
                        Y[it] = mma(ld_frag(L, AF + Sh::GF + it * KS + ks, lane), bh, Y[it]);
                    }
                }
                if (ks % 4 == 3)
                    phase();
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int it = ks / 2; it < 2; ++it) {
                    const int f = Sh::g_frag(it, ks);
                    const h8 ah = ld_frag(L, f, lane);
                    Y[it] = mma(ah, xh[ks], Y[it]);
                    if (FINE) {
                        Y[it] = mma(ah, xl[ks], Y[it]);
                        Y[it] = mma(ld_frag(L, AF + f, lane), xh[ks], Y[it]);
                    }
                }
            const float back = inverse_pow2(sx);
            const size_t yrow = static_cast<size_t>(a.H) * a.P;
            const size_t y0 = (static_cast<size_t>(seq) * a.T + t0) * yrow + col0 + ucol;
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                constexpr int kHalf = Tl::kPerRow / 2;
                union Unit {
                    u4 raw;
                    Act v[Tl::kUnit];
                } zu[kHalf], yu;
                if (a.p.z) {
#pragma unroll
                    for (int k = 0; k < kHalf; ++k) {
                        const int r = min(32 * it + urow + k * Tl::kRowStep, len - 1 - t0);
                        zu[k].raw = *reinterpret_cast<const u4*>(static_cast<const Act*>(a.p.z) + y0 + r * yrow);
                    }
                }
                phase();
                wave_sync();   // what was in the tile is read
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 Sc = *reinterpret_cast<const float4*>(fS + 32 * it + 8 * q + 4 * hi);
                    const float sc[4] = {Sc.x, Sc.y, Sc.z, Sc.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        yt[(8 * q + 4 * hi + i) * Tl::kPitch + c] = Y[it][4 * q + i] * (sc[i] * back);
                }
                wave_sync();
#pragma unroll
                for (int k = 0; k < kHalf; ++k) {
                    const int r = urow + k * Tl::kRowStep;
                    float o[Tl::kUnit];
#pragma unroll
                    for (int q = 0; q < Tl::kUnit / 4; ++q) {
                        const float4 v = *reinterpret_cast<const float4*>(yt + r * Tl::kPitch + ucol + 4 * q);
                        o[4 * q] = v.x;
                        o[4 * q + 1] = v.y;
                        o[4 * q + 2] = v.z;
                        o[4 * q + 3] = v.w;
                    }
                    if (a.p.z) {
#pragma unroll
                        for (int e = 0; e < Tl::kUnit; ++e)
                            o[e] *= silu(widen(zu[k].v[e]));
                    }
#pragma unroll
                    for (int e = 0; e < Tl::kUnit; ++e)
                        narrow(o[e], yu.v[e]);
                    if (t0 + 32 * it + r < len)
                        *reinterpret_cast<u4*>(static_cast<Act*>(a.p.y) + y0 + (32 * it + r) * yrow) = yu.raw;
                }
            }
        }

        phase();
        if (update) {
            const float keep = __builtin_amdgcn_exp2f(total) * (s2 * inverse_pow2(unit));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    S[nt][v] *= keep;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks + kAhead < 4)
                    load_b(sh, ks + kAhead);
                phase();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const h8 ah = bh_[ks % kRing][nt];
                    S[nt] = mma(ah, wh[ks], S[nt]);
                    if (EXACT) {
                        S[nt] = mma(ah, wl[ks], S[nt]);
                        S[nt] = mma(bl_[ks % kRing][nt], wh[ks], S[nt]);
                    }
                }
            }
            unit = s2;
        }
        if (OUT)
            __syncthreads();   // the left factor is rewritten by the next chunk
        wave_sync();           // and so are tile and factors
    }
    if (OUT && split)
        return;   // join has written the state
    float* to = split ? seg_row : state_row;
    const float out = inverse_pow2(unit);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(to + 32 * nt + 8 * q) =
                make_float4(S[nt][4 * q] * out, S[nt][4 * q + 1] * out, S[nt][4 * q + 2] * out, S[nt][4 * q + 3] * out);
    if (split && wave == 0 && lane == 0)
        a.seg_decay[head * a.segs + seg] = static_cast<float>(seg_sum);
}

// Each segment's own state becomes the state that enters it; the state itself
// goes to the end of the prompt.  One thread per four entries.
__global__ __launch_bounds__(256) void ssm_join_kernel(ChunkArgs a, int quads) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t head = i / quads;
    const int64_t q = i % quads;
    const int seq = static_cast<int>(head / a.H);
    if (seq >= a.B)
        return;
    const int len = a.lengths ? a.lengths[seq] : a.T;
    if (len < 1 || len > a.T)
        return;
    const int n = ((len + Q - 1) / Q + a.chunks_per_seg - 1) / a.chunks_per_seg;
    float4* st = reinterpret_cast<float4*>(a.p.state) + head * quads + q;
    float4* sg = reinterpret_cast<float4*>(a.seg_state) + head * a.segs * quads + q;
    const float* dec = a.seg_decay + head * a.segs;
    float4 s = *st;
    for (int k = 0; k < n; ++k) {
        const float4 own = sg[static_cast<int64_t>(k) * quads];
        sg[static_cast<int64_t>(k) * quads] = s;
        const float d = __builtin_amdgcn_exp2f(dec[k]);
        s = make_float4(__builtin_fmaf(d, s.x, own.x), __builtin_fmaf(d, s.y, own.y), __builtin_fmaf(d, s.z, own.z),
                        __builtin_fmaf(d, s.w, own.w));
    }
    *st = s;
}

// Segments: waves wanted, and chunks a segment has at least.
constexpr int kWaves = 4096;
constexpr int kSegChunks = 4;

static void segments(const SsmGeo& g, int T, int& segs, int& per) {
    const int nc = (T + Q - 1) / Q;
    const int64_t waves = static_cast<int64_t>(g.B) * g.H * (g.P / 32);
    const int64_t want = (kWaves + waves - 1) / waves;
    const int most = std::max(1, nc / kSegChunks);
    segs = static_cast<int>(std::min<int64_t>(want, most));
    per = (nc + segs - 1) / segs;
    segs = (nc + per - 1) / per;
}

static size_t shared_halfs(const SsmGeo& g) {
    const bool fine = !g.bf16;
    switch (g.N) {
        case 32: return fine ? Shared<32, true>::kHalfs : Shared<32, false>::kHalfs;
        case 64: return fine ? Shared<64, true>::kHalfs : Shared<64, false>::kHalfs;
        case 128: return fine ? Shared<128, true>::kHalfs : Shared<128, false>::kHalfs;
        default: return fine ? Shared<256, true>::kHalfs : Shared<256, false>::kHalfs;
    }
}

static size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

size_t chunked_ws_bytes(const SsmGeo& g, int T) {
    int segs, per;
    segments(g, T, segs, per);
    const size_t nc = (T + Q - 1) / Q;
    size_t n = up256(static_cast<size_t>(g.B) * g.G * nc * shared_halfs(g) * sizeof(_Float16)) +
               static_cast<size_t>(g.B) * g.H * nc * (3 * Q) * sizeof(float);
    if (segs > 1)
        n += up256(static_cast<size_t>(g.B) * g.H * segs * g.P * g.N * 4) + up256(static_cast<size_t>(g.B) * g.H * segs * 4);
    return n;
}

// A launch that may need more than 64 KB of LDS.
static hipError_t launch_lds(void (*kernel)(ChunkArgs), dim3 grid, dim3 block, size_t lds, hipStream_t s,
                             const ChunkArgs& a) {
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(kernel, grid, block, lds, s, a);
    return hipGetLastError();
}

template <int N, typename Act, bool FINE>
static hipError_t chunked_cfg(const SsmGeo& g, const SsmArgs& p, int T, const int32_t* lengths, void* ws,
                              hipStream_t s) {
    int segs, per;
    segments(g, T, segs, per);
    const int nc = (T + Q - 1) / Q;
    char* base = static_cast<char*>(ws);
    _Float16* shared = reinterpret_cast<_Float16*>(base);
    base += up256(static_cast<size_t>(g.B) * g.G * nc * Shared<N, FINE>::kHalfs * sizeof(_Float16));
    float* steps = reinterpret_cast<float*>(base);
    base += static_cast<size_t>(g.B) * g.H * nc * (3 * Q) * sizeof(float);
    float* seg_state = reinterpret_cast<float*>(base);
    float* seg_decay = reinterpret_cast<float*>(base + up256(static_cast<size_t>(g.B) * g.H * segs * g.P * g.N * 4));
    constexpr size_t lds = (static_cast<size_t>(Q) * (2 * N + 1) + 2 * Q) * sizeof(float);
    auto prep = ssm_prep_kernel<N, Act, FINE>;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(prep),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(prep, dim3(static_cast<unsigned>(static_cast<int64_t>(g.B) * g.G * nc)), dim3(512), lds, s,
                       static_cast<const Act*>(p.x), static_cast<const Act*>(p.tail_in), static_cast<const Act*>(p.w),
                       static_cast<const Act*>(p.bias), lengths, T, g.H, g.G, g.P, g.C, nc, shared);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int64_t step_waves = static_cast<int64_t>(g.B) * g.H * nc;
    hipLaunchKernelGGL(ssm_steps_kernel, dim3(static_cast<unsigned>((step_waves + 3) / 4)), dim3(256), 0, s, p.dt,
                       p.dt_bias, p.A, lengths, T, g.H, nc, step_waves, steps);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    // by XCD where the sets of heads come out even over the eight, or nearly
    const int64_t sets = static_cast<int64_t>(g.B) * g.G * segs;
    const bool by_xcd = sets % 8 == 0 || sets >= 64;
    const ChunkArgs a{p,   lengths, shared, steps, seg_state, seg_decay, T,   g.B,
                      g.H, g.G,     g.P,    g.C,   nc,        segs,      per, by_xcd};
    const int waves = g.P / 32;
    const int64_t wgs = (by_xcd ? (sets + 7) / 8 * 8 : sets) * (g.H / g.G);
    const dim3 grid(static_cast<unsigned>(wgs)), block(64 * waves);
    constexpr int kTile = Tile<Act>::kBytes;
    const size_t lds_state = waves * (kTile + 2 * Q * 4);
    const size_t lds_out = waves * (kTile + 6 * Q * 4) +
                           (FINE ? 2 : 1) * (Shared<N, FINE>::GF + Shared<N, FINE>::CF) * 1024;
    if (segs == 1)
        return launch_lds(ssm_chunk_kernel<N, Act, FINE, true, true>, grid, block, lds_out, s, a);
    if ((e = launch_lds(ssm_chunk_kernel<N, Act, FINE, false, true>, grid, block, lds_state, s, a)) != hipSuccess)
        return e;
    const int quads = g.P * N / 4;
    const int64_t threads = static_cast<int64_t>(g.B) * g.H * quads;
    hipLaunchKernelGGL(ssm_join_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, s, a, quads);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    return launch_lds(ssm_chunk_kernel<N, Act, FINE, true, FINE>, grid, block, lds_out, s, a);
}

hipError_t launch_ssm_chunked(const SsmGeo& g, const SsmArgs& p, int T, const int32_t* lengths, void* ws,
                              hipStream_t s) {
    switch (g.N) {
        case 32: return g.bf16 ? chunked_cfg<32, uint16_t, false>(g, p, T, lengths, ws, s)
                               : chunked_cfg<32, float, true>(g, p, T, lengths, ws, s);
        case 64: return g.bf16 ? chunked_cfg<64, uint16_t, false>(g, p, T, lengths, ws, s)
                               : chunked_cfg<64, float, true>(g, p, T, lengths, ws, s);
        case 128: return g.bf16 ? chunked_cfg<128, uint16_t, false>(g, p, T, lengths, ws, s)
                                : chunked_cfg<128, float, true>(g, p, T, lengths, ws, s);
        default: return g.bf16 ? chunked_cfg<256, uint16_t, false>(g, p, T, lengths, ws, s)
                               : chunked_cfg<256, float, true>(g, p, T, lengths, ws, s);
    }
}

}  // namespace ssm
}  // namespace gdn
